"""Extend with scored attention, prefix and document masks against float64
references over the FP8 workspace (tolerances: tests/scored_util.py)."""
import numpy as np
import pytest
import torch

import nvfp4_quantized_paged_quantize_gb300 as kv
from nvfp4_quantized_paged_quantize_gb300 import inputs
from gpu_util import dev, status_word
from scored_util import SCALE, attend, check, extend_seen, on_gpu, random_q

pytestmark = pytest.mark.gpu

SLOPES = lambda hq: 2.0 ** (-8.0 * (np.arange(hq) + 1) / hq)  # noqa: E731


def e4m3(x):
    return torch.from_numpy(np.ascontiguousarray(x)).view(torch.float8_e4m3fn).double().numpy()


class Case:
    """A ragged extend batch: sequence b has prefix[b] cached rows and chunk[b] new ones, 5 unused rows behind each
    (filled with NaN bytes: nothing may read them into a result)."""

    def __init__(self, prefix, chunk, hq, hkv, seed, q_size=1.0, sk=1.0, sv=1.0, k_exp=(3, 8)):
        rng = np.random.default_rng(seed)
        self.prefix, self.chunk, self.hq, self.hkv = list(prefix), list(chunk), hq, hkv
        self.sk, self.sv = sk, sv
        rows = [p + c + 5 for p, c in zip(prefix, chunk)]
        self.first = np.concatenate([[0], np.cumsum(rows)]).astype(np.int64)
        self.cu_q = np.concatenate([[0], np.cumsum(chunk)]).astype(np.int64)
        shape = (int(self.first[-1]), hkv, 128)
        self.wk = inputs.fp8_bytes_by_field(rng, shape, *k_exp)
        self.wv = inputs.fp8_bytes_by_field(rng, shape, 3, 8)
        for b in range(len(prefix)):
            end = self.first[b + 1]
            self.wk[end - 5:end] = 0x7F
            self.wv[end - 5:end] = 0x7F
        n = int(self.cu_q[-1])
        self.q, self.q64 = random_q((n, hq, 128), seed + 1, q_size)
        self.out = torch.full((n, hq, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((n, hq), float("nan"), device="cuda")
        self.status = status_word()
        self.gpu = [dev(a) for a in (self.cu_q, self.wk, self.wv, self.first[:-1], np.asarray(prefix, np.int32))]

    def run(self, scoring, full=None, docs=None, max_q_len=None, **kw):
        cu_q, wk, wv, first, prefix = self.gpu
        i32 = lambda a: None if a is None else dev(np.asarray(a, np.int32))  # noqa: E731
        kv.nvfp4kv_extend_attention_scored(self.q, cu_q, max_q_len or max(self.chunk), wk, wv, first, prefix, self.out,
                                           SCALE, self.sk, self.sv, scoring=None if scoring is None else on_gpu(scoring),
                                           full_lens=i32(full), doc_starts=i32(docs), lse=self.lse,
                                           device_status=self.status, **kw)

    def check(self, scoring, full=None, docs=None, rows=None):
        torch.cuda.synchronize()
        assert self.status.item() == 0
        scoring = scoring or kv.Scoring()
        out, lse = self.out.double().cpu().numpy(), self.lse.double().cpu().numpy()
        group = self.hq // self.hkv
        for b, (P, C) in enumerate(zip(self.prefix, self.chunk)):
            r0 = self.first[b]
            K, V = (e4m3(w[r0:r0 + P + C]) for w in (self.wk, self.wv))
            for t in range(C):
                i = int(self.cu_q[b]) + t
                if rows is not None and i not in rows:
                    continue
                seen = extend_seen(P, C, t, scoring, None if full is None else full[b],
                                   None if docs is None else docs[i])
                dist = np.abs(P + t - np.arange(P + C)).astype(float)
                for h in range(self.hq):
                    slope = 0.0 if scoring.slopes is None else float(scoring.slopes[h])
                    r = attend(self.q64[i, h], K[:, h // group] * self.sk, V[:, h // group] * self.sv, seen, dist, SCALE,
                               scoring.softcap, slope)
                    check(out[i, h], r["out"], r["tol_out"], f"out {i} {h}")
                    if seen.any():
                        check(lse[i, h], r["lse"], r["tol_lse"], f"lse {i} {h}")
                    else:
                        assert lse[i, h] == -np.inf


SCORINGS = {
    "plain": lambda hq: kv.Scoring(),
    "cap": lambda hq: kv.Scoring(softcap=20.0),
    "cap_tight": lambda hq: kv.Scoring(softcap=1.5),
    "bias": lambda hq: kv.Scoring(slopes=SLOPES(hq)),
    "window_1": lambda hq: kv.Scoring(window=1),
    "window_20": lambda hq: kv.Scoring(window=20, sinks=4),
    "window_130": lambda hq: kv.Scoring(window=130, sinks=150),
    "all": lambda hq: kv.Scoring(softcap=30.0, window=90, sinks=5, slopes=SLOPES(hq)),
}


@pytest.mark.parametrize("name", list(SCORINGS))
@pytest.mark.parametrize("hq,hkv", [(8, 2), (2, 2)])
def test_scored_extend(cuda_lib, name, hq, hkv):
    case = Case([0, 37, 300, 128, 5], [17, 64, 1, 129, 0], hq, hkv, seed=len(name) + hq, q_size=2.0, sk=0.5, sv=1.25)
    scoring = SCORINGS[name](hq)
    case.run(scoring)
    case.check(scoring)


@pytest.mark.parametrize("group", [1, 16, 128])
def test_group_sizes(cuda_lib, group):
    case = Case([70, 0], [5, 9], 2 * group, 2, seed=group)
    scoring = kv.Scoring(softcap=25.0, window=33, sinks=2, slopes=SLOPES(2 * group))
    case.run(scoring)
    case.check(scoring)


@pytest.mark.parametrize("name", ["plain", "bias", "window_20", "all"])
def test_prefix_mask(cuda_lib, name):
    # shared positions: none, past the chunk's end, inside the prefix, inside the chunk
    case = Case([10, 50, 200, 30], [40, 60, 20, 300], 4, 1, seed=21)
    full = [-3, 1000, 100, 170]
    scoring = SCORINGS[name](4)
    case.run(scoring, full=full)
    case.check(scoring, full=full)


@pytest.mark.parametrize("name", ["plain", "cap", "window_20", "window_130", "all"])
def test_document_mask(cuda_lib, name):
    case = Case([0, 90], [400, 60], 4, 2, seed=22)
    rng = np.random.default_rng(5)
    docs = []
    for P, C in zip(case.prefix, case.chunk):
        start, left = 0, 0
        for pos in range(P + C):
            if left == 0:
                start, left = pos, int(rng.integers(1, 120))
            left -= 1
            if pos >= P:
                docs.append(start)
    docs[3] = -7                                                 # hides nothing
    scoring = SCORINGS[name](4)
    case.run(scoring, docs=docs)
    case.check(scoring, docs=docs)


def test_prefix_and_document_masks_together(cuda_lib):
    case = Case([20], [200], 4, 1, seed=23)
    docs = [0] * 60 + [80] * 140
    full = [150]
    scoring = kv.Scoring(window=30, sinks=3, slopes=SLOPES(4))
    case.run(scoring, full=full, docs=docs)
    case.check(scoring, full=full, docs=docs)


def test_rows_that_see_nothing(cuda_lib):
    # documents that start behind their own token: single rows, and whole blocks of rows
    case = Case([10, 300], [70, 300], 8, 2, seed=24)
    docs = np.zeros(370, np.int64)
    docs[5] = 16                                                 # position 15
    docs[40:70] = 2 ** 31 - 1
    docs[70:] = 5000                                             # sequence 1: every row
    docs[200] = 0
    for scoring in (None, kv.Scoring(softcap=9.0, window=64, sinks=2), kv.Scoring(slopes=SLOPES(8))):
        case.out.fill_(float("nan"))
        case.run(scoring, docs=docs)
        case.check(scoring, docs=docs)


def test_sharp_scores_move_the_running_maximum(cuda_lib):
    case = Case([300, 64], [40, 3], 16, 2, seed=25, k_exp=(6, 13))
    for scoring in (None, kv.Scoring(slopes=np.full(16, 0.01)), kv.Scoring(softcap=500.0)):
        case.run(scoring, max_q_len=200)                         # a generous bound: extra tiles leave
        case.check(scoring)


def test_windows_over_long_prefixes(cuda_lib):
    case = Case([5000, 1111], [70, 200], 4, 1, seed=26)
    rows = set(range(0, 270, 23)) | {0, 69, 70, 269}
    for scoring in (kv.Scoring(window=700, sinks=260), kv.Scoring(softcap=15.0),
                    kv.Scoring(slopes=SLOPES(4), window=4000, sinks=1)):
        case.run(scoring)
        case.check(scoring, rows=rows)


def test_plain_scoring_equals_the_plain_extend(cuda_lib):
    case = Case([100, 7], [50, 33], 8, 2, seed=27)
    case.run(None)
    cu_q, wk, wv, first, prefix = case.gpu
    out32 = torch.empty(tuple(case.out.shape), dtype=torch.float32, device="cuda")
    kv.nvfp4kv_extend_attention(case.q, cu_q, 50, wk, wv, first, prefix, out32, SCALE)
    torch.cuda.synchronize()
    # both within P's f16 rounding of the same sums, one of them rounded to bf16 as well
    a, b = case.out.float(), out32
    assert ((a - b).abs() <= 2.0 ** -8 * b.abs() + 2.0 ** -9 * b.norm(dim=-1, keepdim=True)).all()


def test_rows_outside_the_workspace_and_bad_lengths_are_flagged(cuda_lib):
    case = Case([40, 60], [20, 30], 4, 1, seed=28)
    good = list(case.gpu)
    case.gpu[3] = dev(np.array([case.first[0], 10 ** 12], np.int64))
    case.run(kv.Scoring(softcap=8.0))
    torch.cuda.synchronize()
    assert case.status.item() == kv.NVFP4KV_DEVERR_ROW
    case.status.zero_()
    case.check(kv.Scoring(softcap=8.0), rows=set(range(20)))     # the other sequence is right
    case.gpu = good
    case.status.zero_()
    case.run(None, max_q_len=25)                                 # sequence 1's chunk is cut
    torch.cuda.synchronize()
    assert case.status.item() == kv.NVFP4KV_DEVERR_LENGTH
    case.status.zero_()
    case.check(None, rows=set(range(20)))


def test_capture_and_another_stream(cuda_lib):
    case = Case([64], [100], 8, 2, seed=29)
    scoring = kv.Scoring(softcap=10.0, window=50, sinks=4)
    ds = on_gpu(scoring)
    cu_q, wk, wv, first, prefix = case.gpu
    call = lambda: kv.nvfp4kv_extend_attention_scored(case.q, cu_q, 100, wk, wv, first, prefix, case.out, SCALE,  # noqa: E731
                                                      scoring=ds, lse=case.lse, device_status=case.status)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    case.check(scoring)
    want = case.out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    case.out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(case.out, want)


def test_rows_out_of_sight_may_hold_anything(cuda_lib):
    # rows that no query sees (between the sinks and the window, before the
    # documents) are NaN bytes, in tiles that others make visible
    case = Case([600, 300], [9, 40], 4, 1, seed=30)
    scoring = kv.Scoring(window=50, sinks=4)
    docs = [0] * 9 + [170] * 40
    r0, r1 = int(case.first[0]), int(case.first[1])
    hidden = np.r_[r0 + 4:r0 + 600 - 49, r1:r1 + 170, r1 + 174:r1 + 300 - 49]
    case.gpu[1][dev(hidden)] = 0x7F
    case.gpu[2][dev(hidden)] = 0x7F
    for sc in (scoring, kv.Scoring(window=50, sinks=4, softcap=20.0), kv.Scoring(window=50, sinks=4, slopes=SLOPES(4))):
        case.out.fill_(float("nan"))
        case.run(sc, docs=docs)
        case.check(sc, docs=docs)


@pytest.mark.parametrize("softcap", [2.0 ** -20, 2.0 ** -6, 1.0, 6.0, 2.0 ** 20])
def test_caps_of_every_size(cuda_lib, softcap):
    # all scores far beyond the cap, around it (each form of the cap), far inside it
    case = Case([200], [70], 4, 2, seed=31, q_size=2.0)
    case.run(kv.Scoring(softcap=softcap))
    case.check(kv.Scoring(softcap=softcap))


UNSEEN = {
    # two documents in a block of rows: the first one's middle is behind its window
    "two_documents": ([600], [40], [[0] * 20 + [620] * 20], dict(window=50, sinks=4)),
    # padding between documents, hidden from itself too by a start behind every token
    "padding": ([30], [90], [[0] * 25 + [2 ** 31 - 1] * 15 + [70] * 50], {}),
    "padding_window": ([300], [90], [[0] * 25 + [5000] * 15 + [340] * 50], dict(window=20, sinks=3)),
    # starts in no order, sinks that cross a tile's edge, documents that see ahead
    "any_order": ([2000, 700], [37, 50], [([1800] * 9 + [3] * 9 + [900] * 9 + [120] * 10), [640, 10, 250, 9000, 380] * 10],
                  dict(window=8, sinks=20)),
    "many_documents": ([500], [250], [[max(0, 3 * (t // 3) - 200) * (t % 2) + 500 * (t % 7 == 0) for t in range(250)]],
                       dict(window=5, sinks=2)),
}


@pytest.mark.parametrize("name", list(UNSEEN))
@pytest.mark.parametrize("kind", ["plain", "cap", "bias"])
@pytest.mark.parametrize("hq,hkv,full", [(4, 1, False), (2, 2, False), (8, 1, True)])
def test_rows_that_no_document_shows_may_hold_anything(cuda_lib, name, kind, hq, hkv, full):
    prefix, chunk, docs, mask = UNSEEN[name]
    case = Case(prefix, chunk, hq, hkv, seed=40 + len(name))
    scoring = kv.Scoring(softcap=20.0 if kind == "cap" else 0.0, slopes=SLOPES(hq) if kind == "bias" else None, **mask)
    full = [P // 3 for P in prefix] if full else None
    hidden = []
    for b, (P, C) in enumerate(zip(prefix, chunk)):
        seen = np.zeros(P + C, bool)
        for t in range(C):
            seen |= extend_seen(P, C, t, scoring, None if full is None else full[b], docs[b][t])
        assert not seen.all()
        hidden.append(int(case.first[b]) + np.flatnonzero(~seen))
    hidden = dev(np.concatenate(hidden))
    case.gpu[1][hidden] = 0x7F
    case.gpu[2][hidden] = 0x7F
    flat = np.concatenate(docs)
    case.run(scoring, full=full, docs=flat)
    case.check(scoring, full=full, docs=flat)


@pytest.mark.parametrize("mask", ["none", "window", "bias"])
@pytest.mark.parametrize("softcap", [500.0, 2.0 ** 14, 2.0 ** 20])
def test_small_scores_beside_one_at_its_cap(cuda_lib, softcap, mask):
    # one query whose scores pass its cap among queries with scores of a few units:
    # theirs stay as accurate.  (The keys' scale keeps every query inside f16's range.)
    case = Case([120], [40], 4, 1, seed=33, k_exp=(9, 12), sk=32.0)
    size = torch.full((40, 1, 1), 2.0 ** -10)
    size[11] = 2.0 ** -10 * softcap                              # in the same warp as queries 8 .. 15
    q = (torch.from_numpy(case.q64).float() * size).to(torch.bfloat16)
    case.q, case.q64 = q.cuda(), q.double().numpy()
    scoring = kv.Scoring(softcap=softcap, window=100 if mask == "window" else 0, sinks=2,
                         slopes=SLOPES(4) if mask == "bias" else None)
    case.run(scoring)
    case.check(scoring)


@pytest.mark.parametrize("softcap", [0.0, 20.0])
def test_the_steepest_slopes(cuda_lib, softcap):
    # log2(e) times the slope is past fp32's range: the nearest key alone is left
    case = Case([70, 0], [40, 9], 4, 1, seed=34)
    scoring = kv.Scoring(softcap=softcap, slopes=np.array([float(np.finfo(np.float32).max), 0.5, 2.5e38, 3e38]))
    case.run(scoring)
    case.check(scoring)
