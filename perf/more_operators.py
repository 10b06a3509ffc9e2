"""Workloads of a decode step's other parts, with a plain form of each.

Around the cache's decode a server plans where new tokens go, prepares their queries and keys, and, for long
contexts, picks the pages worth reading.  Six operators over the NVFP4 paged cache:

  plan       page tables, slots, positions and workspace rows of a step's new tokens, from the requests' lengths
             and a stack of free pages                                             (nvfp4kv_plan_append)
  norm_rope  root-mean-square norms of queries and keys for each head, the position rotation, and the quantised
             append of keys and values, in one pass                                (nvfp4kv_norm_rope_append)
  digest     upper and lower bounds of each page's keys, per channel               (nvfp4kv_page_digest)
  scores     for each page an upper bound of its tokens' scores, from the bounds   (nvfp4kv_page_scores)
  select     the first, the latest and the best scored pages of each KV head       (nvfp4kv_select_pages)
  attend     one new token per sequence over the selected pages alone              (nvfp4kv_decode_attention_selected)

`run` computes an operator with elementary torch operations in 32 bits, or, with `own` set, by the library's
calls.  `exact` restates the definitions in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False

PAGE, DIM, PAGE_HEAD, DIGEST = 16, 128, 2304, 272
EPS = 1e-6
K_SCALE, V_SCALE = 0.0043, 0.0031   # calibrated global scales of keys and values of ordinary size

# the most that one pass may cost: cached (token, KV head) pairs, and (new token, head) rows
MOST_CACHED = 4 * 131073 * 8
MOST_ROWS = 4 * 4099 * 80


def _plan(name, batch, low, high, new, short=False):
    return {"name": name, "op": "plan", "batch": batch, "low": low, "high": high, "new": new, "short": short}


def _norm_rope(name, batch, high, new, hq, hkv, rot=DIM, interleaved=False, norm=True, fp8=False):
    return {"name": name, "op": "norm_rope", "batch": batch, "high": high, "new": new, "hq": hq, "hkv": hkv, "rot": rot,
            "interleaved": interleaved, "norm": norm, "fp8": fp8}


def _cached(name, op, batch, low, high, hq, hkv, budget=0, first=0, recent=0, new=0):
    return {"name": name, "op": op, "batch": batch, "low": low, "high": high, "hq": hq, "hkv": hkv, "budget": budget,
            "first": first, "recent": recent, "new": new}


def listed():
    return [
        # a decode step of a large continuous batch: one token each, a page for every sixteenth
        _plan("plan_decode_256", 256, 1, 8192, 1),
        # a step that takes the next chunk of sixteen prompts, of unequal lengths
        _plan("plan_chunks", 16, 1, 16384, 2048),
        # the new tokens of a decode batch: what counts is the launch
        _norm_rope("norm_rope_decode_32", 32, 8193, 1, 64, 8),
        # long prompts' first chunks, whose keys and values also go to the FP8 workspace
        _norm_rope("norm_rope_prefill_4x4k", 4, 4099, 4099, 64, 8, fp8=True),
        # after a decode step's append: each sequence's last page is bounded again
        _cached("digest_step_32", "digest", 32, 8193, 8193, 64, 8, new=1),
        # after a long prompt's prefill: every page
        _cached("digest_prompt_128k", "digest", 4, 100003, 131073, 64, 8),
        # the pages of a batch at 8K, scored for its new tokens
        _cached("scores_8k", "scores", 32, 8193, 8193, 64, 8),
        # long contexts
        _cached("scores_128k", "scores", 4, 100003, 131073, 64, 8),
        # 64 pages of each KV head in a continuous batch of very unequal lengths
        _cached("select_ragged", "select", 96, 512, 32768, 32, 8, budget=64, first=1, recent=4),
        # an eighth of long contexts
        _cached("select_128k", "select", 4, 100003, 131073, 64, 8, budget=1024, first=1, recent=16),
        # a decode step of a batch at 8K that reads an eighth of it
        _cached("attend_8k", "attend", 32, 8193, 8193, 64, 8, budget=64, first=1, recent=4),
        # of long contexts
        _cached("attend_128k", "attend", 4, 100003, 131073, 64, 8, budget=1024, first=1, recent=16),
    ]


def _log_int(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["plan", "norm_rope", "digest", "scores", "select", "attend"])
    if op == "plan":
        batch, high = _log_int(rng, 1, 1024), _log_int(rng, 1, 131073)
        new = rng.choice([1, 1, _log_int(rng, 1, max(1, 32768 // batch))])
        return _nameless(_plan("", batch, max(1, high // rng.choice([1, 8, 64])), high, new, rng.random() < 0.2))
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 4, 5, 8])
    if op == "norm_rope":
        rows = hq + 2 * hkv
        new = rng.choice([1, _log_int(rng, 1, 8192)])
        batch = max(1, min(_log_int(rng, 1, 256), MOST_ROWS // (rows * new)))
        new = max(1, min(new, MOST_ROWS // (rows * batch)))
        return _nameless(_norm_rope("", batch, max(new, _log_int(rng, 1, 65536)), new, hq, hkv, rng.choice([32, 64, 96, 128, 128]),
                                    rng.random() < 0.4, rng.random() < 0.8, rng.random() < 0.4))
    high = _log_int(rng, 1 if op != "select" else 100, 131073)   # a selection has something to choose from
    low = max(1, high // rng.choice([1, 1, 2, 8, 64]))
    batch = max(1, min(_log_int(rng, 1, 96), MOST_CACHED // (hkv * high)))
    pages = -(-high // PAGE)
    budget = max(1, pages // rng.choice([1 if op != "select" else 3, 2, 4, 8, 16]))
    if op == "attend":
        budget = max(1, min(budget, 4 * 8 * 1024 // (batch * hkv)))
    first = min(budget // 4, rng.choice([0, 1, 4]))
    recent = min(budget // 4, rng.choice([0, 1, 8, budget // 8]))
    return _nameless(_cached("", op, batch, low, high, hq, hkv, budget, first, recent,
                             rng.choice([0, 1, _log_int(rng, 1, low)]) if op == "digest" else 0))


def _nameless(case):
    return {k: v for k, v in case.items() if k != "name"}


def _lengths(case):
    """Cached tokens of each sequence: spread evenly over their logarithm, in mixed order."""
    n, low, high = case["batch"], case["low"], case["high"]
    got = [int(round(low * (high / low) ** (i / (n - 1)))) if n > 1 else high for i in range(n)]
    random.Random(n * 1000003 + high).shuffle(got)
    return got


def _new_tokens(case):
    """New tokens of each request of a plan or a norm_rope: the first has all, later ones down to four tenths."""
    n = case["batch"]
    return [max(1, int(case["new"] * (1.0 - 0.6 * i / n))) for i in range(n)]


def _pages(tokens):
    return [-(-n // PAGE) for n in tokens]


def _plan_need(case):
    """New pages of each request of a plan, and the free pages that it finds."""
    cached, new = _lengths(case), _new_tokens(case)
    need = [a - b for a, b in zip(_pages([c + n for c, n in zip(cached, new)]), _pages(cached))]
    return need, sum(need) * 2 // 3 if case["short"] else sum(need) + 37


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _nvfp4_rows(x):
    """E2M1 codes [n, 128] and E4M3 scale bytes [n, 8] of fp32 rows, near enough for inputs."""
    b = x.view(-1, DIM // 16, 16)
    s = (b.abs().amax(-1) / 6.0).to(torch.float8_e4m3fn)
    y = b / s.float().clamp_min(2.0 ** -9)[..., None]
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=x.device)
    code = torch.bucketize(y.abs(), edges, out_int32=True).to(torch.uint8) | (y < 0).to(torch.uint8) << 3
    return code.view(-1, DIM), s.view(torch.uint8)


def _pool(pages, hkv, gen):
    """A cache pool [pages, hkv, 2304] of keys and values as models make them: channels of unequal size, a few tokens
    that draw attention."""
    pool = torch.empty((pages, hkv, PAGE_HEAD), dtype=torch.uint8, device="cuda")
    channel = torch.exp2(torch.rand(2, DIM, generator=gen, device="cuda") * 3.0 - 1.5)
    for at in range(0, pages, 1 << 15):
        part = pool[at:at + (1 << 15)]
        n = part.shape[0] * hkv * PAGE
        loud = 1.0 + 2.0 * (torch.rand(n, 1, generator=gen, device="cuda") < 0.01)
        k, ks = _nvfp4_rows(torch.randn(n, DIM, generator=gen, device="cuda") * channel[0] * loud)
        v, vs = _nvfp4_rows(torch.randn(n, DIM, generator=gen, device="cuda") * channel[1])
        heads = (part.shape[0], hkv)
        part[..., :1024] = (k[:, 0::2] | k[:, 1::2] << 4).view(*heads, 1024)
        part[..., 1024:1152] = ks.reshape(*heads, 128)
        pairs = v.view(*heads, PAGE // 2, 2, DIM)
        part[..., 1152:2176] = (pairs[..., 0, :] | pairs[..., 1, :] << 4).reshape(*heads, 1024)
        part[..., 2176:] = vs.view(*heads, PAGE, 8).transpose(-1, -2).reshape(*heads, 128)
    return pool


def _digests(pages, hkv, gen):
    """Digests [pages, hkv, 272] of such pages: bounds some two deviations from zero, and the power of two."""
    n = pages * hkv
    channel = torch.exp2(torch.rand(DIM, generator=gen, device="cuda") * 3.0 - 1.5)
    draws = torch.randn(2, n, DIM, generator=gen, device="cuda")
    loud = 1.0 + 2.0 * (torch.rand(n, 1, generator=gen, device="cuda") < 0.1)
    hi, lo = (1.8 + 0.5 * draws[0]) * channel * loud, (-1.8 + 0.5 * draws[1]) * channel * loud
    hi, lo = torch.maximum(hi, lo), torch.minimum(hi, lo)
    scale = _power(torch.frexp(torch.maximum(hi.abs(), lo.abs()).amax(-1, keepdim=True)).exponent - 8)
    d = torch.zeros((n, DIGEST), dtype=torch.uint8, device="cuda")
    d[:, :128] = (hi / scale).to(torch.float8_e4m3fn).view(torch.uint8)
    d[:, 128:256] = (lo / scale).to(torch.float8_e4m3fn).view(torch.uint8)
    d[:, 256:260] = scale.view(torch.uint8)
    return d.view(pages, hkv, DIGEST)


def _page_table(counts, gen, width=None, spare=0):
    """Pages of each sequence: shuffled ids, the rows padded with the first one; and `spare` ids of no sequence."""
    ids = torch.randperm(sum(counts) + spare, generator=gen, device="cuda").to(torch.int32)
    n = torch.tensor(counts, device="cuda")[:, None]
    col = torch.arange(width or max(counts), device="cuda")
    at = torch.cumsum(n, 0) - n + col
    return torch.where(col < n, ids[at.clamp_max(sum(counts) - 1)], ids[0]), ids[sum(counts):]


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _prepare_plan(case, gen):
    cached, new = _lengths(case), _new_tokens(case)
    need, free = _plan_need(case)
    width = max(_pages([c + n for c, n in zip(cached, new)])) + 3
    table, stack = _page_table(_pages(cached), gen, width, spare=sum(need) + 64)
    # room of a step's fixed size for the new tokens, as a captured step has it
    tokens, batch = -(-sum(new) // 64) * 64, case["batch"]
    int64 = lambda n: torch.empty(n, dtype=torch.int64, device="cuda")  # noqa: E731
    return {"table": table, "cached": _int32(cached), "new": _int32(new), "free": stack, "free_count": _int32([free]),
            "num_pages": sum(_pages(cached)) + stack.numel(), "free_left": _int32([0]), "lens": _int32([0] * batch),
            "slots": int64(tokens), "positions": torch.empty(tokens, dtype=torch.int32, device="cuda"),
            "rows": int64(tokens), "cu_q": int64(batch + 1), "cu_rows": int64(batch + 1)}


def _prepare_norm_rope(case, gen):
    s = {k: case[k] for k in ("hq", "hkv", "rot", "interleaved", "norm", "fp8")}
    hq, hkv, new = case["hq"], case["hkv"], _new_tokens(case)
    total = sum(new)
    start = [case["high"] - n if i % 2 == 0 else (case["high"] - n) // 2 for i, n in enumerate(new)]
    pos = np.concatenate([np.arange(p, p + n) for p, n in zip(start, new)])
    # the pages that the new tokens fall into
    counts = [(p + n - 1) // PAGE - p // PAGE + 1 for p, n in zip(start, new)]
    table, _ = _page_table(counts, gen)
    seq = np.repeat(np.arange(len(new)), new)
    local = torch.from_numpy(pos // PAGE - np.array(start)[seq] // PAGE).cuda()
    page = table[torch.from_numpy(seq).cuda(), local].long()
    s["slots"] = page * PAGE + torch.from_numpy(pos % PAGE).cuda()
    s["positions"] = torch.from_numpy(pos.astype(np.int32)).cuda()
    # queries, keys and values side by side, as one projection makes them
    rows = hq + 2 * hkv
    channel = torch.exp2(torch.rand(rows, DIM, generator=gen, device="cuda") * 3.0 - 1.5)
    size = torch.exp2(torch.rand(total, 1, 1, generator=gen, device="cuda") * 4.0 - 2.0)
    s["qkv"] = (torch.randn(total, rows, DIM, generator=gen, device="cuda") * channel * size).to(torch.bfloat16)
    weights = (1.0 + 0.3 * torch.randn(2, DIM, generator=gen, device="cuda")).to(torch.bfloat16)
    s["q_weight"], s["k_weight"] = (weights[0], weights[1]) if case["norm"] else (None, None)
    half = case["rot"] // 2
    rate = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
    angle = torch.arange(int(pos.max()) + 1, dtype=torch.float64, device="cuda")[:, None] * rate
    s["cos_sin"] = torch.cat((angle.cos(), angle.sin()), -1).float()
    s["pool"] = torch.zeros((sum(counts), hkv, PAGE_HEAD), dtype=torch.uint8, device="cuda")
    s["q_out"] = torch.empty((total, hq, DIM), dtype=torch.bfloat16, device="cuda")
    s["ws_k"] = s["ws_v"] = s["ws_rows"] = None
    if case["fp8"]:
        s["ws_rows"] = torch.randperm(total, generator=gen, device="cuda")
        s["ws_k"] = torch.zeros((total, hkv, DIM), dtype=torch.uint8, device="cuda")
        s["ws_v"] = torch.zeros((total, hkv, DIM), dtype=torch.uint8, device="cuda")
    return s


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    if op in ("plan", "norm_rope"):
        return {"op": op, **(_prepare_plan if op == "plan" else _prepare_norm_rope)(case, gen)}
    batch, hq, hkv = case["batch"], case["hq"], case["hkv"]
    lens = _lengths(case)
    pages = _pages(lens)
    s = {"op": op, "hq": hq, "hkv": hkv, "lens": _int32(lens), "max_pages": max(pages), "scale": 1.0 / math.sqrt(DIM)}
    s |= {k: case[k] for k in ("budget", "first", "recent")}
    if op == "select":
        # bounds of some hundred tokens' scores, many of them near one another, a few equal
        x = torch.randn((batch, hkv, max(pages)), generator=gen, device="cuda") * 1.5 + 4.0
        s["scores"] = torch.where(torch.rand(x.shape, generator=gen, device="cuda") < 0.05, torch.round(x * 4.0) / 4.0, x)
        s["selected"] = torch.empty((batch, hkv, case["budget"]), dtype=torch.int32, device="cuda")
        return s
    s["table"], _ = _page_table(pages, gen)
    if op == "scores":
        s["pool"] = torch.empty((sum(pages), hkv, PAGE_HEAD), dtype=torch.uint8, device="cuda")   # not read
        s["digest"] = _digests(sum(pages), hkv, gen)
        s["q"] = torch.randn(batch, hq, DIM, generator=gen, device="cuda").to(torch.bfloat16)
        s["scores"] = torch.zeros((batch, hkv, max(pages)), device="cuda")
        return s
    s["pool"] = _pool(sum(pages), hkv, gen)
    if op == "digest":
        s["digest"] = torch.zeros((sum(pages), hkv, DIGEST), dtype=torch.uint8, device="cuda")
        s["from"] = _int32([n - case["new"] for n in lens]) if case["new"] else None
        return s
    s["q"] = torch.randn(batch, hq, DIM, generator=gen, device="cuda").to(torch.bfloat16)
    # what a selection leaves: the first pages, the last ones, others between; ascending, then -1
    at = torch.arange(max(pages), device="cuda")
    n = _int32(pages)[:, None, None]
    rank = torch.rand((batch, hkv, max(pages)), generator=gen, device="cuda")
    rank = torch.where((at < case["first"]) | (at >= n - case["recent"]), 2.0, rank)
    width = min(case["budget"], max(pages))
    order = torch.sort(torch.where(at < n, rank, -1.0), dim=-1, descending=True, stable=True).indices[..., :width]
    used = torch.arange(width, device="cuda") < n
    order = torch.sort(torch.where(used, order, max(pages)), dim=-1).values
    s["selected"] = torch.full((batch, hkv, case["budget"]), -1, dtype=torch.int32, device="cuda")
    s["selected"][..., :width] = torch.where(used, order, -1).to(torch.int32)
    s["out"] = torch.empty((batch, hq, DIM), dtype=torch.bfloat16, device="cuda")
    s["lse"] = torch.empty((batch, hq), device="cuda")
    return s


# --------------------------------------------------------------------------
# plain forms
# --------------------------------------------------------------------------

def _plain_plan(s):
    free = s["free_count"].long()
    room = s["table"].shape[1] * PAGE
    cached = s["cached"].long().clamp(0, room)
    new = torch.minimum(s["new"].long().clamp_min(0), room - cached)
    have = (cached + PAGE - 1) // PAGE
    need = (cached + new + PAGE - 1) // PAGE - have
    tokens = s["slots"].shape[0]
    served = (torch.cumsum(need, 0) <= free) & (torch.cumsum(new, 0) <= tokens)
    new, need = torch.where(served, new, 0), torch.where(served, need, 0)
    cu_q, cu_rows = s["cu_q"].zero_(), s["cu_rows"].zero_()
    cu_q[1:] = torch.cumsum(new, 0)
    cu_rows[1:] = torch.cumsum(cached + new, 0)
    s["lens"].copy_(cached + new)
    # the new pages, off the top of the stack
    col = torch.arange(s["table"].shape[1], device="cuda")
    nth = (torch.cumsum(need, 0) - need)[:, None] + col - have[:, None]
    fresh = (col >= have[:, None]) & (col < (have + need)[:, None])
    taken = s["free"][(free - 1 - nth).clamp(0, s["free"].shape[0] - 1)]
    s["table"].copy_(torch.where(fresh, taken, s["table"]))
    s["free_left"].copy_(free - need.sum())
    # the new tokens
    t = torch.arange(tokens, device="cuda")
    live = t < cu_q[-1]
    b = torch.searchsorted(cu_q[1:], t, right=True).clamp_max(new.shape[0] - 1)
    pos = torch.where(live, cached[b] + t - cu_q[b], 0)
    page = s["table"][b, pos // PAGE].long()
    s["slots"].copy_(torch.where(live, page * PAGE + pos % PAGE, -1))
    s["positions"].copy_(pos)
    s["rows"].copy_(torch.where(live, cu_rows[b] + pos, -1))
    return _planned(s)


def _planned(s):
    return {k: s[k] for k in ("table", "lens", "slots", "positions", "rows", "cu_q", "cu_rows", "free_left")}


def _pairs(x):
    return x[..., 0::2] + x[..., 1::2]


def _normed(x, weight):
    """x / rms(x) * weight over the last axis, each step rounded to 32 bits, the sum as a tree of neighbours."""
    if weight is None:
        return x
    total = _pairs(_pairs(_pairs(_pairs(_pairs(_pairs(_pairs(x * x)))))))
    one = torch.ones((), device="cuda")
    return x * (one / (total * (1.0 / DIM) + EPS).sqrt()) * weight.float()


def _rotated(x, s):
    half = s["rot"] // 2
    cos, sin = s["cos_sin"][s["positions"].long()][:, None].split(half, -1)
    a, b = (x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if s["interleaved"] else (x[..., :half], x[..., half:2 * half])
    ra, rb = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack((ra, rb), -1).flatten(-2) if s["interleaved"] else torch.cat((ra, rb), -1)
    return torch.cat((turned, x[..., 2 * half:]), -1)


def _quantised(x, g):
    """E2M1 codes [..., 128] and E4M3 scale bytes [..., 8] of bf16 rows, step by step in 32 bits, ties to even."""
    b = x.float().unflatten(-1, (8, 16))
    g = torch.full((), g, device="cuda")
    s = (b.abs().amax(-1) / (6.0 * g)).clamp_max(448.0).to(torch.float8_e4m3fn)
    den = (s.float() * g)[..., None]
    y = torch.where(den == 0, 0.0, (b / den).abs())
    up = lambda m, tie: ((y >= m) if tie else (y > m)).to(torch.uint8)  # noqa: E731
    code = up(0.25, False) + up(0.75, True) + up(1.25, False) + up(1.75, True) + up(2.5, False) + up(3.5, True) + up(5.0, False)
    return (code | torch.signbit(b).to(torch.uint8) << 3).flatten(-2), s.view(torch.uint8)


def _plain_norm_rope(s):
    hq, hkv = s["hq"], s["hkv"]
    q, k, v = s["qkv"].split((hq, hkv, hkv), 1)
    s["q_out"].copy_(_rotated(_normed(q.float(), s["q_weight"]), s).to(torch.bfloat16))
    k = _rotated(_normed(k.float(), s["k_weight"]), s).to(torch.bfloat16)
    page, row = s["slots"] // PAGE, s["slots"] % PAGE
    pool = s["pool"]
    code, scale = _quantised(k, K_SCALE)
    pool[..., :1024].unflatten(-1, (PAGE, 64))[page, :, row] = code[..., 0::2] | code[..., 1::2] << 4
    pool[..., 1024:1152].unflatten(-1, (PAGE, 8))[page, :, row] = scale
    # the two tokens of a byte of the values go in one after the other
    code, scale = _quantised(v, V_SCALE)
    pairs = pool[..., 1152:2176].unflatten(-1, (PAGE // 2, DIM))
    even = (row % 2 == 0)[:, None, None]
    spare = torch.zeros((PAGE * pool.shape[0], hkv, DIM), dtype=torch.uint8, device="cuda")
    spare[s["slots"]] = code
    there = torch.zeros(PAGE * pool.shape[0], dtype=torch.bool, device="cuda")
    there[s["slots"]] = True
    mate = s["slots"] ^ 1
    old = pairs[page, :, row // 2]
    low = torch.where(even, code, torch.where(there[mate][:, None, None], spare[mate], old & 15))
    high = torch.where(even, torch.where(there[mate][:, None, None], spare[mate], old >> 4), code)
    pairs[page, :, row // 2] = low | high << 4
    pool[..., 2176:].unflatten(-1, (8, PAGE)).transpose(-1, -2)[page, :, row] = scale
    if s["fp8"]:
        s["ws_k"][s["ws_rows"]] = k.float().clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
        s["ws_v"][s["ws_rows"]] = v.float().clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    return _appended(s)


def _appended(s):
    # every step of the quantisation is one rounded operation, so the packed codes are determined byte by byte and
    # come back as they lie (their values would take another kernel to unpack); the 8-bit rows as values
    got = {"q": s["q_out"], "pages": s["pool"]}
    if s["fp8"]:
        got |= {"ws_k": s["ws_k"].view(torch.float8_e4m3fn), "ws_v": s["ws_v"].view(torch.float8_e4m3fn)}
    return got


def _e2m1(codes):
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0],
                         device=codes.device)
    return table[codes.to(torch.int32)]


def _keys(heads):
    """Keys [..., 16, 128] of page-heads [..., 2304], without the global scale."""
    lead = heads.shape[:-1]
    kd = heads[..., :1024].reshape(*lead, PAGE, DIM // 2)
    k = _e2m1(torch.stack((kd & 15, kd >> 4), -1)).view(*lead, PAGE, 8, 16)
    return (k * heads[..., 1024:1152].contiguous().view(torch.float8_e4m3fn).float().view(*lead, PAGE, 8, 1)).flatten(-2)


def _values(heads):
    lead = heads.shape[:-1]
    vd = heads[..., 1152:2176].reshape(*lead, PAGE // 2, DIM)
    v = _e2m1(torch.stack((vd & 15, vd >> 4), -2)).view(*lead, PAGE, 8, 16)
    vs = heads[..., 2176:].contiguous().view(torch.float8_e4m3fn).float().view(*lead, 8, PAGE)
    return (v * vs.transpose(-1, -2)[..., None]).flatten(-2)


def _power(e):
    """2^e of int32 exponents, to the bit."""
    return (e + 127 << 23).view(torch.float32)


def _outward(x, up):
    """x rounded to E4M3, up or down (|x| <= 256): to a whole number of its binade's steps."""
    step = _power(torch.frexp(x.abs().clamp_min(2.0 ** -6)).exponent - 4)
    return (torch.ceil(x / step) if up else torch.floor(x / step)) * step


def _plain_digest(s):
    at = torch.arange(s["max_pages"], device="cuda")
    lens = s["lens"].long()[:, None]
    live = at * PAGE < lens
    if s["from"] is not None:
        live = live & (at >= s["from"].long().clamp_min(0)[:, None] // PAGE)
    b, page = live.nonzero(as_tuple=True)
    ids = s["table"][b, page].long()
    k = _keys(s["pool"][ids])                                        # [n, Hkv, 16, 128]
    valid = (page * PAGE)[:, None] + torch.arange(PAGE, device="cuda") < lens[b]
    valid = valid[:, None, :, None]
    hi = torch.where(valid, k, -math.inf).amax(-2)
    lo = torch.where(valid, k, math.inf).amin(-2)
    top = torch.maximum(hi.abs(), lo.abs()).amax(-1, keepdim=True)
    # frexp: top = m 2^e with m in [0.5, 1)
    e = torch.frexp(torch.where(top > 0, top, 1.0)).exponent - 1
    scale = torch.where(top > 0, _power(e - 7), 1.0)
    d = torch.zeros((*hi.shape[:-1], DIGEST), dtype=torch.uint8, device="cuda")
    d[..., :128] = (_outward(hi / scale, True) + 0.0).to(torch.float8_e4m3fn).view(torch.uint8)
    d[..., 128:256] = (_outward(lo / scale, False) + 0.0).to(torch.float8_e4m3fn).view(torch.uint8)
    d[..., 256:260] = scale.contiguous().view(torch.uint8)
    s["digest"][ids] = d
    return _digested(s)


def _digested(s):
    d = s["digest"]
    return {"hi": d[..., :128].view(torch.float8_e4m3fn), "lo": d[..., 128:256].view(torch.float8_e4m3fn),
            "scale": d[..., 256:260].view(torch.float32), "rest": d[..., 260:]}


def _plain_scores(s):
    b, hkv = s["q"].shape[0], s["hkv"]
    d = s["digest"][s["table"].long()].transpose(1, 2)               # [B, Hkv, pages, 272]
    hi = d[..., :128].contiguous().view(torch.float8_e4m3fn).float()
    lo = d[..., 128:256].contiguous().view(torch.float8_e4m3fn).float()
    q = s["q"].float().view(b, hkv, -1, DIM)
    u = torch.matmul(q.clamp_min(0), hi.transpose(-1, -2)) + torch.matmul(q.clamp_max(0), lo.transpose(-1, -2))
    u = u.amax(2) * d[..., 256:260].contiguous().view(torch.float32)[..., 0] * (s["scale"] * K_SCALE)
    live = torch.arange(s["max_pages"], device="cuda") * PAGE < s["lens"].long()[:, None, None]
    s["scores"].copy_(torch.where(live, u, s["scores"]))
    return s["scores"]


def _plain_select(s):
    at = torch.arange(s["max_pages"], device="cuda")
    n = ((s["lens"].long() + PAGE - 1) // PAGE)[:, None, None]
    always = (at < s["first"]) | (at >= n - s["recent"])
    rank = torch.where(at < n, torch.where(always, math.inf, s["scores"]), -math.inf)
    width = min(s["budget"], s["max_pages"])
    order = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., :width]
    used = torch.arange(width, device="cuda") < n
    order = torch.sort(torch.where(used, order, s["max_pages"]), dim=-1).values
    s["selected"].fill_(-1)
    s["selected"][..., :width] = torch.where(used, order, -1).to(torch.int32)
    return s["selected"]


def _plain_attend(s):
    b, hkv, group = s["q"].shape[0], s["hkv"], s["hq"] // s["hkv"]
    page = s["selected"].long()                                      # [B, Hkv, n]
    chosen = page >= 0
    ids = s["table"].long().gather(1, page.clamp_min(0).view(b, -1)).view(page.shape)
    heads = s["pool"][ids, torch.arange(hkv, device="cuda")[:, None]]
    k, v = _keys(heads).flatten(2, 3) * K_SCALE, _values(heads).flatten(2, 3) * V_SCALE
    pos = (page * PAGE)[..., None] + torch.arange(PAGE, device="cuda")
    visible = (chosen[..., None] & (pos < s["lens"].long()[:, None, None, None])).flatten(2)[:, :, None]
    q = s["q"].float().view(b, hkv, group, DIM)
    x = (torch.matmul(q, k.transpose(-1, -2)) * s["scale"]).masked_fill(~visible, -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    e = (x - top).exp()
    total = e.sum(-1, keepdim=True)
    s["lse"].copy_((top + total.log()).view(b, -1))
    s["out"].copy_((torch.matmul(e, v) / torch.where(total > 0, total, torch.ones_like(total))).view(b, s["hq"], DIM))
    return {"out": s["out"], "lse": s["lse"]}


# --------------------------------------------------------------------------
# the library's calls
# --------------------------------------------------------------------------

def _own(s):
    import nvfp4_quantized_paged_quantize_gb300 as kv

    op = s["op"]
    if op == "plan":
        kv.nvfp4kv_plan_append(s["table"], s["cached"], s["new"], s["free"], s["free_count"], s["num_pages"], s["lens"],
                               s["slots"], s["free_left"], positions=s["positions"], cu_q=s["cu_q"], ws_rows=s["rows"],
                               cu_prefix=s["cu_rows"])
        return _planned(s)
    if op == "norm_rope":
        hq, hkv = s["hq"], s["hkv"]
        cache = kv.Cache(s["pool"], s["pool"].shape[0], hkv, K_SCALE, V_SCALE)
        q, k, v = s["qkv"].split((hq, hkv, hkv), 1)
        kv.nvfp4kv_norm_rope_append(cache, q, k, v, s["slots"], s["positions"], s["cos_sin"], s["q_out"],
                                    q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS, interleaved=s["interleaved"],
                                    ws_rows=s["ws_rows"], ws_k=s["ws_k"], ws_v=s["ws_v"])
        return _appended(s)
    if op == "select":
        kv.nvfp4kv_select_pages(s["scores"], s["lens"], s["budget"], s["first"], s["recent"], s["selected"])
        return s["selected"]
    cache = kv.Cache(s["pool"], s["pool"].shape[0], s["hkv"], K_SCALE, V_SCALE)
    if op == "digest":
        kv.nvfp4kv_page_digest(cache, s["table"], s["lens"], s["digest"], first_tokens=s["from"])
        return _digested(s)
    if op == "scores":
        kv.nvfp4kv_page_scores(cache, s["digest"], s["q"], s["table"], s["lens"], s["scale"], s["scores"])
        return s["scores"]
    if "workspace" not in s:  # scratch of the batch's shape, as a program keeps it between steps
        n = kv.nvfp4kv_decode_workspace_size(cache, s["q"].shape[0], s["hq"])
        s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    kv.nvfp4kv_decode_attention_selected(cache, s["q"], s["out"], s["table"], s["lens"], s["scale"], s["selected"],
                                         s["workspace"], lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


_PLAIN = {"plan": _plain_plan, "norm_rope": _plain_norm_rope, "digest": _plain_digest, "scores": _plain_scores,
          "select": _plain_select, "attend": _plain_attend}


def run(state):
    return _own(state) if own else _PLAIN[state["op"]](state)


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------

def work(case):
    op, batch = case["op"], case["batch"]
    if op == "plan":
        need, free = _plan_need(case)
        new = _new_tokens(case)
        tokens = -(-sum(new) // 64) * 64
        # lengths in and out, the sums; stack entries read and table entries written; slots, positions and rows
        return {"bytes": batch * (12.0 + 16.0) + 8.0 * min(sum(need), free) + 20.0 * tokens, "flops": 0}
    if op == "norm_rope":
        total, hq, hkv = sum(_new_tokens(case)), case["hq"], case["hkv"]
        row = hq * 4.0 * DIM + 2 * hkv * (2.0 * DIM + 72 + (DIM if case["fp8"] else 0)) + 4.0 * case["rot"] + 12
        return {"bytes": total * row, "flops": total * (hq + hkv) * DIM * 7.0}
    lens = _lengths(case)
    pages, hq, hkv = _pages(lens), case["hq"], case["hkv"]
    if op == "digest":
        done = sum(p - max(0, n - case["new"]) // PAGE for p, n in zip(pages, lens)) if case["new"] else sum(pages)
        return {"bytes": done * hkv * (1152.0 + DIGEST), "flops": done * hkv * PAGE * DIM * 3.0}
    if op == "scores":
        return {"bytes": sum(pages) * hkv * (DIGEST + 4.0) + batch * hq * 2.0 * DIM, "flops": sum(pages) * hq * 4.0 * DIM}
    if op == "select":
        return {"bytes": hkv * (4.0 * sum(pages) + 4.0 * batch * case["budget"]), "flops": 0}
    read = sum(min(p, case["budget"]) for p in pages) * hkv
    return {"bytes": read * (PAGE_HEAD + 4.0) + batch * hq * (4.0 * DIM + 4), "flops": read * (hq // hkv) * PAGE * DIM * 4.0}


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------

_E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def _byte_values():
    """The 16 E2M1 codes and the 256 E4M3 bytes as 64-bit numbers, from the formats' fields."""
    e2m1 = np.concatenate([_E2M1, -_E2M1])
    byte = np.arange(256)
    exponent, mantissa = byte >> 3 & 15, byte & 7
    e4m3 = np.where(exponent > 0, (1 + mantissa / 8.0) * 2.0 ** (exponent - 7.0), mantissa / 8.0 * 2.0 ** -6)
    e4m3 = np.where(byte & 128, -e4m3, e4m3)
    return torch.tensor(e2m1, device="cuda"), torch.tensor(e4m3, device="cuda")


def _exact_rows(pool, ids, head, t):
    """Keys and values [n, 128] of the tokens t of one sequence and KV head in 64 bits, row by row of the page layout."""
    e2m1, e4m3 = _byte_values()
    raw = pool[ids.long()[t // PAGE], head]                          # [n, 2304]: each token's page-head
    row, d = (t % PAGE)[:, None], torch.arange(DIM, device="cuda")[None]
    kb = raw.gather(1, row * 64 + d // 2).long()
    k = e2m1[torch.where(d % 2 == 0, kb & 15, kb >> 4)] * e4m3[raw.gather(1, 1024 + row * 8 + d // 16).long()]
    vb = raw.gather(1, 1152 + row // 2 * 128 + d).long()
    v = e2m1[torch.where(row % 2 == 0, vb & 15, vb >> 4)] * e4m3[raw.gather(1, 2176 + d // 16 * 16 + row).long()]
    return k, v


def _exact_norm_rope(s):
    x = s["qkv"].double()
    hq, hkv, half = s["hq"], s["hkv"], s["rot"] // 2
    angle = s["cos_sin"].double()[s["positions"].long()]
    turn = torch.complex(angle[:, :half], angle[:, half:])[:, None]

    def made(rows, weight):
        if weight is not None:
            rows = rows * torch.rsqrt(rows.square().mean(-1, keepdim=True) + EPS) * weight.double()
        i = torch.arange(half, device="cuda")
        a, b = (2 * i, 2 * i + 1) if s["interleaved"] else (i, i + half)
        z = torch.complex(rows[..., a], rows[..., b]) * turn
        rows = rows.clone()
        rows[..., a], rows[..., b] = z.real, z.imag
        return rows

    got = {"q": made(x[:, :hq], s["q_weight"]), "pages": None}
    if s["fp8"]:
        for name, rows in (("ws_k", made(x[:, hq:hq + hkv], s["k_weight"])), ("ws_v", x[:, hq + hkv:])):
            got[name] = torch.empty_like(rows)
            got[name][s["ws_rows"]] = rows
    return got


def _exact_digest(s):
    d = s["digest"]
    hi, lo = (torch.zeros((*d.shape[:2], DIM), dtype=torch.float64, device="cuda") for _ in range(2))
    scale = torch.zeros((*d.shape[:2], 1), dtype=torch.float64, device="cuda")
    grid = _byte_values()[1][:127]                                   # ascending magnitudes, 0 .. 448

    def outward(x, up):
        at = torch.searchsorted(grid, x.abs())                       # the first magnitude that is not smaller
        above = grid[at]
        below = torch.where(above == x.abs(), above, grid[(at - 1).clamp_min(0)])
        away = (x >= 0) if up else (x < 0)
        return torch.sign(x) * torch.where(away, above, below)

    for b, n in enumerate(s["lens"].tolist()):
        start = max(0, int(s["from"][b])) // PAGE if s["from"] is not None else 0
        t = torch.arange(start * PAGE, n, device="cuda")
        pad = -len(t) % PAGE
        ids = s["table"][b, start:-(-n // PAGE)].long()
        for h in range(s["hkv"]):
            k, _ = _exact_rows(s["pool"], s["table"][b], h, t)
            k = torch.cat((k, k[-1:].expand(pad, DIM))).view(-1, PAGE, DIM)
            top, bottom = k.max(1).values, k.min(1).values
            most = k.abs().amax((1, 2))[:, None]
            log = torch.floor(torch.log2(torch.where(most > 0, most, 1.0))).long() - 7
            unit = torch.where(most > 0, (log + 1023 << 52).view(torch.float64), 1.0)
            hi[ids, h], lo[ids, h], scale[ids, h] = outward(top / unit, True), outward(bottom / unit, False), unit
    return {"hi": hi, "lo": lo, "scale": scale, "rest": None}


def _exact_scores(s):
    _, e4m3 = _byte_values()
    group = s["hq"] // s["hkv"]
    got = s["scores"].double()
    for b, n in enumerate(s["lens"].tolist()):
        pages = -(-n // PAGE)
        for h in range(s["hkv"]):
            raw = s["digest"][s["table"][b, :pages].long(), h]
            hi, lo = e4m3[raw[:, :128].long()], e4m3[raw[:, 128:256].long()]
            unit = raw[:, 256:260].contiguous().view(torch.float32)[:, 0].double()
            q = s["q"][b, h * group:(h + 1) * group].double()
            u = torch.stack([torch.maximum(x * hi, x * lo).sum(-1) for x in q]).amax(0)
            got[b, h, :pages] = u * unit * s["scale"] * float(np.float32(K_SCALE))
    return got


def _exact_attend(s):
    group = s["hq"] // s["hkv"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["lens"].tolist()):
        for h in range(s["hkv"]):
            pages = s["selected"][b, h]
            t = (pages[pages >= 0].long()[:, None] * PAGE + torch.arange(PAGE, device="cuda")).flatten()
            k, v = _exact_rows(s["pool"], s["table"][b], h, t[t < n])
            x = s["q"][b, h * group:(h + 1) * group].double() @ k.T * (s["scale"] * float(np.float32(K_SCALE)))
            lse[b, h * group:(h + 1) * group] = torch.logsumexp(x, 1)
            out[b, h * group:(h + 1) * group] = torch.softmax(x, 1) @ v * float(np.float32(V_SCALE))
    return {"out": out, "lse": lse}


def exact(case, seed):
    op = case["op"]
    if op in ("plan", "select"):
        return None   # whole numbers
    s = prepare(case, seed)
    return {"norm_rope": _exact_norm_rope, "digest": _exact_digest, "scores": _exact_scores, "attend": _exact_attend}[op](s)
