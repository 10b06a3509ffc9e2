"""Model check of the scored extend kernel's synchronisation protocol (host only).

The kernel (csrc/extend_scored.cu) runs in one CTA around mbarriers: loader
warps fill a five-slot ring with K and V tiles in turn; two softmax groups
write their Q tile, read their S, rescale their O and write their P over their
S; one warp issues the tensor-core MMAs, S_t = Q_t K^T and O_t += P_t V
(t = 0, 1), which finish in the order of their issue.  This model replays each
role's waits, arrivals, commits and buffer accesses, in the kernel's order,
under random interleavings, with the parities the kernel waits for, and checks:

- a wait passes only on the completion it means (parities do not alias);
- no buffer is overwritten while an MMA issued earlier may use it, and every
  read sees what it expects;
- every interleaving finishes.
"""
import random

import pytest

SLOTS = 5


class Barrier:
    def __init__(self, count=1):
        self.count, self.pending, self.done = count, count, 0

    def arrive(self):
        self.pending -= 1
        if self.pending == 0:
            self.done, self.pending = self.done + 1, self.count


def loader(n):
    slot, parity, reuse = 0, 1, False
    for item in range(2 * n):
        if reuse:
            yield ("wait", f"empty{slot}", parity, item // SLOTS - 1)
        yield ("write", f"ring{slot}", ("K", "V")[item % 2] + str(item // 2))
        yield ("arrive", f"full{slot}")
        slot += 1
        if slot == SLOTS:
            slot, parity, reuse = 0, parity ^ 1, True


def softmax(n, t):
    yield ("write", f"Q{t}", "Q")
    yield ("arrive", "q_full")
    for i in range(n):
        yield ("wait", f"s_full{t}", i & 1, i)
        yield ("read", f"S{t}", f"S{i}")
        if i > 0:
            yield ("read", f"O{t}", f"O{i - 1}")       # the rescale of O
            yield ("write", f"O{t}", f"O{i - 1}")
        yield ("write", f"S{t}", f"P{i}")
        yield ("arrive", f"p_full{t}")
    yield ("wait", f"s_full{t}", n & 1, n)
    yield ("read", f"O{t}", f"O{n - 1}")


def mma(n, drop=()):
    item, at, parity, items = 0, 0, 0, 2 * n

    def done():
        nonlocal item, at, parity
        got = [("commit", f"empty{at}")] if item + SLOTS < items else []
        item += 1
        at += 1
        if at == SLOTS:
            at, parity = 0, parity ^ 1
        return got

    def wait(*a):
        return [] if a[0][:4] in drop else [("wait",) + a]

    def scores(t, slot, i):
        return [("issue", [(f"Q{t}", "Q"), (f"ring{slot}", f"K{i}")], f"S{t}", None, f"S{i}"), ("commit", f"s_full{t}")]

    yield from wait("q_full", 0, 0)
    yield from wait(f"full{at}", parity, item // SLOTS)
    yield from scores(0, 0, 0)
    yield from scores(1, 0, 0)
    yield from done()
    for i in range(n):
        more, v_at, k_at = i + 1 < n, at, (at + 1) % SLOTS
        yield from wait(f"full{at}", parity, item // SLOTS)
        if more:
            yield from wait(f"full{k_at}", parity ^ 1 if k_at == 0 else parity, (item + 1) // SLOTS)
        for t in range(2):
            yield from wait(f"p_full{t}", i & 1, i)
            yield ("issue", [(f"S{t}", f"P{i}"), (f"ring{v_at}", f"V{i}")], f"O{t}", f"O{i - 1}" if i else None, f"O{i}")
            if t == 1:
                yield from done()
            if more:
                yield from scores(t, k_at, i + 1)
            else:
                yield ("commit", f"s_full{t}")
            if t == 1 and more:
                yield from done()
    yield ("commit", "drain")
    yield ("wait", "drain", 0, 0)


def run(n, seed, drop=()):
    rng = random.Random(seed)
    bars = {"q_full": Barrier(2), "drain": Barrier()}
    bars |= {f"{k}{s}": Barrier() for k in ("full", "empty") for s in range(SLOTS)}
    bars |= {f"{k}{t}": Barrier() for k in ("s_full", "p_full") for t in range(2)}
    roles = {"loader": list(loader(n)), "mma": list(mma(n, drop)), "softmax0": list(softmax(n, 0)),
             "softmax1": list(softmax(n, 1))}
    pc = {r: 0 for r in roles}
    holds, busy, inflight = {}, {}, []      # buffer -> contents; buffer -> MMAs in flight that use it
    while True:
        ready = ["tensor"] if inflight else []
        for r, prog in roles.items():
            if pc[r] < len(prog):
                a = prog[pc[r]]
                # an mbarrier test passes when the phase of that parity is not the current one
                if a[0] != "wait" or (bars[a[1]].done & 1) != a[2]:
                    ready.append(r)
        if not ready:
            break
        r = rng.choice(ready)
        if r == "tensor":                   # the oldest issued operation finishes
            kind, *rest = inflight.pop(0)
            if kind == "commit":
                bars[rest[0]].arrive()
                continue
            reads, out, before, after = rest
            for buf, want in reads:
                assert holds.get(buf) == want, f"{buf} holds {holds.get(buf)}, not {want}"
                busy[buf] -= 1
            if before is not None:
                assert holds.get(out) == before
            holds[out] = after
            busy[out] -= 1
            continue
        a = roles[r][pc[r]]
        pc[r] += 1
        if a[0] == "wait":
            assert bars[a[1]].done == a[3] + 1, f"{r}: {a} passed after {bars[a[1]].done} completions"
        elif a[0] == "arrive":
            bars[a[1]].arrive()
        elif a[0] == "commit":
            inflight.append(("commit", a[1]))
        elif a[0] == "issue":
            inflight.append(("mma",) + a[1:])
            for buf in [b for b, _ in a[1]] + [a[2]]:
                busy[buf] = busy.get(buf, 0) + 1
        elif a[0] == "read":
            assert holds.get(a[1]) == a[2] and not busy.get(a[1]), f"{r} reads {a[1]}: {holds.get(a[1])}, not {a[2]}"
        else:
            # an MMA of the other operand kind may be queued behind: it must not use the buffer yet
            assert not busy.get(a[1]), f"{r} overwrites {a[1]} while an MMA uses it"
            holds[a[1]] = a[2]
    assert all(pc[r] == len(prog) for r, prog in roles.items()), f"stuck at {pc}"


@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 6, 11, 24])
def test_every_interleaving_is_safe(n):
    for seed in range(60):
        run(n, seed)


@pytest.mark.parametrize("dropped", ["full", "p_fu", "q_fu"])
def test_the_model_sees_a_missing_wait(dropped):
    with pytest.raises(AssertionError):
        for seed in range(200):
            run(12, seed, drop=(dropped,))
