"""Decode with scored attention, and with accumulated weights, against float64
references over the dequantised cache (tolerances: tests/scored_util.py)."""
import numpy as np
import pytest
import torch

import nvfp4_quantized_paged_quantize_gb300 as kv
from gpu_util import dev, status_word
from scored_util import (SCALE, check, decode_ref, on_gpu, page_tables, random_cache, random_q, sequence_rows)

pytestmark = pytest.mark.gpu

SLOPES = lambda hq: 2.0 ** (-8.0 * (np.arange(hq) + 1) / hq)  # noqa: E731


class Batch:
    """A batch over a random cache, its GPU tensors and the references."""

    def __init__(self, lens, hq, hkv, seed, gk=1.0, gv=1.0, q_size=1.0, extra_cols=0, spare_pages=2):
        self.lens, self.hq, self.hkv = list(lens), hq, hkv
        self.table, used = page_tables(lens, seed, extra_cols=extra_cols)
        self.cache, self.oracle = random_cache(used + spare_pages, hkv, seed, gk, gv)
        self.q, self.q64 = random_q((len(lens), hq, 128), seed + 1, q_size)
        self.pt, self.sl = dev(self.table), dev(np.asarray(lens, np.int32))
        self.out = torch.full((len(lens), hq, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((len(lens), hq), float("nan"), device="cuda")
        self.status = status_word()

    def decode(self, scoring, **kw):
        ws = torch.empty(kv.nvfp4kv_decode_workspace_size(self.cache, len(self.lens), self.hq), dtype=torch.uint8,
                         device="cuda")
        kv.nvfp4kv_decode_attention_scored(self.cache, self.q, self.out, self.pt, self.sl, SCALE, ws,
                                           scoring=None if scoring is None else on_gpu(scoring), lse=self.lse,
                                           device_status=self.status, **kw)

    def weighted(self, scoring, weights, decay=1.0, max_total_pages=None, **kw):
        n = kv.nvfp4kv_decode_weights_workspace_size(self.cache, len(self.lens), self.hq,
                                                     max_total_pages or self.cache.num_pages)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda").fill_(0xFF)      # scratch needs no initialisation
        kv.nvfp4kv_decode_attention_weights(self.cache, self.q, self.out, self.pt, self.sl, SCALE, weights, ws,
                                            scoring=None if scoring is None else on_gpu(scoring), decay=decay,
                                            lse=self.lse, max_total_pages=max_total_pages,
                                            device_status=self.status, **kw)

    def refs(self, scoring):
        scoring = scoring or kv.Scoring()
        group = self.hq // self.hkv
        for b, L in enumerate(self.lens):
            for h in range(self.hkv):
                K, V = sequence_rows(self.oracle, self.table[b], h, L)
                yield b, h, [decode_ref(K, V, self.q64[b, h * group + g], L, scoring, head=h * group + g)
                             for g in range(group)]

    def check(self, scoring, weights=None, before=None, decay=1.0):
        torch.cuda.synchronize()
        assert self.status.item() == 0
        out, lse = self.out.double().cpu().numpy(), self.lse.double().cpu().numpy()
        w = None if weights is None else weights.double().cpu().numpy()
        group = self.hq // self.hkv
        for b, h, refs in self.refs(scoring):
            for g, r in enumerate(refs):
                i = h * group + g
                check(out[b, i], r["out"], r["tol_out"], f"out {b} {i}")
                if self.lens[b] == 0:
                    assert lse[b, i] == -np.inf
                else:
                    check(lse[b, i], r["lse"], r["tol_lse"], f"lse {b} {i}")
            if w is not None:
                L = self.lens[b]
                old = before[b, h].astype(np.float64)
                want = decay * old[:L] + sum(r["p"] for r in refs)
                tol = sum(r["tol_p"] for r in refs) + 2.0 ** -22 * np.abs(want)
                check(w[b, h, :L], want, tol, f"weights {b} {h}")
                assert np.array_equal(w[b, h, L:], old[L:]), "entries past the sequence were touched"


SCORINGS = {
    "plain": lambda hq: kv.Scoring(),
    "cap": lambda hq: kv.Scoring(softcap=20.0),
    "cap_tight": lambda hq: kv.Scoring(softcap=1.5),            # most scores beyond it: tanh's outer form
    "bias": lambda hq: kv.Scoring(slopes=SLOPES(hq)),
    "bias_steep": lambda hq: kv.Scoring(slopes=np.full(hq, 3.0)),
    "window_1": lambda hq: kv.Scoring(window=1),
    "window_16": lambda hq: kv.Scoring(window=16, sinks=4),
    "window_17": lambda hq: kv.Scoring(window=17, sinks=16),
    "window_100": lambda hq: kv.Scoring(window=100, sinks=37),
    "window_joins_sinks": lambda hq: kv.Scoring(window=40, sinks=2000),
    "all": lambda hq: kv.Scoring(softcap=30.0, window=90, sinks=5, slopes=SLOPES(hq)),
}
LENS = [0, 1, 15, 16, 17, 33, 100, 129, 257, 500]


@pytest.mark.parametrize("name", list(SCORINGS))
@pytest.mark.parametrize("hq,hkv", [(8, 2), (1, 1), (10, 2), (16, 2)])
def test_scored_decode(cuda_lib, name, hq, hkv):
    batch = Batch(LENS, hq, hkv, seed=hq * 31 + len(name), gk=0.75, gv=1.5, q_size=2.0)
    scoring = SCORINGS[name](hq)
    batch.decode(scoring)
    batch.check(scoring)


@pytest.mark.parametrize("name", ["plain", "cap", "bias", "window_17", "all"])
@pytest.mark.parametrize("hq,hkv,decay", [(8, 2, 1.0), (2, 2, 0.5), (6, 1, 0.0), (10, 2, 0.25), (16, 2, 1.0)])
def test_accumulated_weights(cuda_lib, name, hq, hkv, decay):
    batch = Batch(LENS, hq, hkv, seed=hq * 37 + len(name), q_size=2.0)
    scoring = SCORINGS[name](hq)
    before = np.random.default_rng(3).random((len(LENS), hkv, 517), dtype=np.float32)   # an odd stride
    if decay == 0.0:
        for b, L in enumerate(LENS):
            before[b, :, :L] = np.nan                            # not read: NaN must not come through
    weights = dev(before)
    batch.weighted(scoring, weights, decay)
    batch.check(scoring, weights, np.where(np.isnan(before), 0.0, before), decay)


def test_no_scoring_is_the_plain_decode(cuda_lib):
    batch = Batch([300, 77], 8, 2, seed=5)
    batch.decode(None)
    batch.check(None)
    out32 = torch.empty((2, 8, 128), dtype=torch.float32, device="cuda")
    ws = torch.empty(kv.nvfp4kv_decode_workspace_size(batch.cache, 2, 8), dtype=torch.uint8, device="cuda")
    kv.nvfp4kv_decode_attention(batch.cache, batch.q, out32, batch.pt, batch.sl, SCALE, ws)
    assert torch.equal(out32.to(torch.bfloat16), batch.out)     # the same kernel, rounded once


@pytest.mark.parametrize("batch_size", [129, 1100])             # the length scan in blocks, the combine's prefix
def test_many_sequences(cuda_lib, batch_size):
    lens = np.random.default_rng(batch_size).integers(0, 40, batch_size)
    lens[-1] = 0                                                  # an empty one at the end
    batch = Batch(lens, 2, 1, seed=batch_size)
    scoring = kv.Scoring(window=20, sinks=3)
    before = np.ones((batch_size, 1, 48), np.float32)
    weights = dev(before)
    batch.weighted(scoring, weights, 0.5)
    batch.check(scoring, weights, before, 0.5)


def test_all_sequences_empty(cuda_lib):
    batch = Batch([0, 0, 0], 4, 1, seed=8)
    weights = torch.ones((3, 1, 16), device="cuda")
    batch.weighted(kv.Scoring(softcap=5.0), weights)
    batch.check(None, weights, np.ones((3, 1, 16), np.float32))


@pytest.mark.parametrize("name", ["plain", "cap", "all"])
def test_pairs_cut_over_many_warps(cuda_lib, name):
    lens = [9001, 40]
    batch = Batch(lens, 8, 1, seed=11, q_size=1.5)
    scoring = SCORINGS[name](8)
    if name == "all":
        scoring = kv.Scoring(softcap=30.0, window=5000, sinks=100, slopes=SLOPES(8))
    before = np.random.default_rng(4).random((2, 1, 9001), dtype=np.float32)
    weights = dev(before)
    batch.weighted(scoring, weights, 0.875)
    batch.check(scoring, weights, before, 0.875)


def test_repeated_steps_accumulate(cuda_lib):
    batch = Batch([70, 200], 8, 2, seed=12)
    weights = torch.zeros((2, 2, 208), device="cuda")
    for _ in range(3):
        batch.weighted(None, weights)
    torch.cuda.synchronize()
    w = weights.double().cpu().numpy()
    for b, L in enumerate(batch.lens):
        # each step adds the group's four softmaxes: 12 per KV head in the end
        # (each weight within 2^-11 relative by far, the sums of at most 200 terms too)
        np.testing.assert_allclose(w[b, :, :L].sum(-1), 12.0, rtol=2.0 ** -11)
        assert not w[b, :, L:].any()


def test_pages_out_of_sight_are_not_touched(cuda_lib):
    # the page-table entries between the sinks and the window are stale ids
    # (here: out of range), and the rows out of sight in partly visible pages are NaN scales
    lens = [400]
    batch = Batch(lens, 4, 1, seed=13)
    scoring = kv.Scoring(window=50, sinks=20)                    # sees 0 .. 19 and 350 .. 399
    first, last = 2, 350 // 16                                   # pages 0, 1 and 21 .. 24 are visited
    table = batch.table.copy()
    table[0, first:last] = 1 << 30
    want = list(batch.refs(scoring))
    batch.pt = dev(table)
    for t in list(range(20, 32)) + list(range(last * 16, 350)):
        page, row = int(batch.table[0, t // 16]), t % 16
        batch.cache.k_scale[page, 0, row] = 0x7F
        batch.cache.v_scale[page, 0, row] = 0x7F
    before = np.ones((1, 1, 400), np.float32)
    weights = dev(before)
    batch.weighted(scoring, weights, 0.5)
    torch.cuda.synchronize()
    assert batch.status.item() == 0
    for b, h, refs in want:
        for g, r in enumerate(refs):
            check(batch.out[b, g].double().cpu(), r["out"], r["tol_out"], "out")
        p = sum(r["p"] for r in refs)
        check(weights[0, 0].cpu(), 0.5 + p, sum(r["tol_p"] for r in refs) + 2.0 ** -20, "weights")


def test_bad_indices_are_flagged(cuda_lib):
    batch = Batch([64, 64], 4, 1, seed=14)
    good, table = batch.table.copy(), batch.table.copy()
    table[1, :] = -5                                             # nothing of sequence 1 can be read
    batch.pt = dev(table)
    weights = torch.ones((2, 1, 64), device="cuda")
    batch.weighted(kv.Scoring(softcap=10.0), weights, 0.5)
    torch.cuda.synchronize()
    assert batch.status.item() == kv.NVFP4KV_DEVERR_PAGE
    assert not batch.out[1].any() and (batch.lse[1] == -float("inf")).all()
    assert (weights[1] == 0.5).all()                             # decayed, nothing added
    # a length past the page table is clamped and flagged; weights too short for a sequence are, too
    batch.pt, batch.sl = dev(good), dev(np.array([64, 80], np.int32))
    batch.status.zero_()
    batch.decode(None)
    torch.cuda.synchronize()
    assert batch.status.item() == kv.NVFP4KV_DEVERR_LENGTH
    batch.sl = dev(np.array([64, 64], np.int32))
    batch.status.zero_()
    guard = torch.full((2, 1, 60), 7.0, device="cuda")
    batch.weighted(None, guard[:1].expand(2, 1, 60).contiguous(), 1.0)
    torch.cuda.synchronize()
    assert batch.status.item() == kv.NVFP4KV_DEVERR_LENGTH


def test_more_pages_than_the_workspace_holds(cuda_lib):
    batch = Batch([64, 200], 4, 1, seed=15)
    weights = torch.full((2, 1, 208), 3.0, device="cuda")
    batch.weighted(None, weights, 0.5, max_total_pages=16)       # 4 + 13 pages
    torch.cuda.synchronize()
    assert batch.status.item() == kv.NVFP4KV_DEVERR_LENGTH
    assert (weights == 3.0).all()
    batch.status.zero_()
    batch.check(None)
    batch.weighted(None, weights, 0.5, max_total_pages=17)
    batch.check(None, weights, np.full((2, 1, 208), 3.0, np.float32), 0.5)


def test_capture_and_another_stream(cuda_lib):
    batch = Batch([300, 45], 8, 2, seed=16)
    scoring = kv.Scoring(softcap=10.0, window=100, sinks=4)
    dev_scoring = on_gpu(scoring)
    weights = torch.zeros((2, 2, 304), device="cuda")
    n = kv.nvfp4kv_decode_weights_workspace_size(batch.cache, 2, 8, batch.cache.num_pages)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    call = lambda: kv.nvfp4kv_decode_attention_weights(batch.cache, batch.q, batch.out, batch.pt, batch.sl, SCALE,  # noqa: E731
                                                       weights, ws, scoring=dev_scoring, lse=batch.lse,
                                                       device_status=batch.status)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    batch.check(scoring, weights, np.zeros((2, 2, 304), np.float32))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    weights.zero_()
    batch.out.zero_()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    w2 = weights.clone()
    weights.zero_()
    call()
    call()
    torch.cuda.synchronize()
    assert torch.equal(w2, weights)                              # bit-identical, graph or not
    q2, batch.q64 = random_q((2, 8, 128), 99)
    batch.q.copy_(q2)                                            # new inputs at the captured addresses
    weights.zero_()
    graph.replay()
    batch.check(scoring, weights, np.zeros((2, 2, 304), np.float32))


@pytest.mark.parametrize("softcap", [2.0 ** -20, 2.0 ** -6, 1.0, 6.0, 2.0 ** 20])
def test_caps_of_every_size(cuda_lib, softcap):
    batch = Batch([40, 300], 8, 2, seed=17, q_size=2.0)
    batch.decode(kv.Scoring(softcap=softcap))
    batch.check(kv.Scoring(softcap=softcap))


def test_outputs_stay_inside_their_buffers(cuda_lib):
    from test_gpu_canary import Guarded

    batch = Batch([0, 33, 400, 17], 10, 2, seed=18)
    out, lse = Guarded((4, 10, 128), torch.bfloat16), Guarded((4, 10), torch.float32)
    weights = Guarded((4, 2, 401), torch.float32)
    weights.t.zero_()
    n = kv.nvfp4kv_decode_weights_workspace_size(batch.cache, 4, 10, batch.cache.num_pages)
    ws = Guarded((n,), torch.uint8)
    scoring = kv.Scoring(softcap=10.0, window=40, sinks=3)
    kv.nvfp4kv_decode_attention_weights(batch.cache, batch.q, out.t, batch.pt, batch.sl, SCALE, weights.t, ws.t,
                                        scoring=scoring, decay=0.5, lse=lse.t, device_status=batch.status)
    batch.out, batch.lse = out.t, lse.t
    batch.check(scoring, weights.t, np.zeros((4, 2, 401), np.float32), 0.5)
    for g in (out, lse, weights, ws):
        assert g.intact()


@pytest.mark.parametrize("kept", [False, True])
def test_a_bias_that_leaves_fp32_hides_its_head_alone(cuda_lib, kept):
    # a head whose bias is -inf in fp32 on all but its nearest keys, beside heads
    # whose maximum moves; several pages of a pair to a warp
    lens = [300] * 500 + [17, 1, 0]
    batch = Batch(lens, 4, 1, seed=19, q_size=2.0)
    scoring = kv.Scoring(slopes=np.array([1e37, 0.01, 1e35, 0.0]))
    if kept:
        before = np.ones((len(lens), 1, 304), np.float32)
        weights = dev(before)
        batch.weighted(scoring, weights, 0.5)
        batch.check(scoring, weights, before, 0.5)
    else:
        batch.decode(scoring)
        batch.check(scoring)


def test_the_steepest_slopes(cuda_lib):
    # log2(e) times the slope is past fp32's range: the nearest key alone is left
    batch = Batch([300, 17, 1], 4, 1, seed=21, q_size=2.0)
    scoring = kv.Scoring(slopes=np.array([float(np.finfo(np.float32).max), 0.5, 2.5e38, 3e38]))
    batch.decode(scoring)
    batch.check(scoring)


@pytest.mark.parametrize("exponent", [24, 40, 90])
def test_caps_with_large_global_scales(cuda_lib, exponent):
    # scores of a few units from keys of 2^exponent and queries as small: the factor inside the tanh is large
    batch = Batch([40, 300], 8, 2, seed=20, gk=2.0 ** exponent, q_size=2.0 ** (1 - exponent))
    for softcap in (1.0, 2.0 ** -20):
        batch.decode(kv.Scoring(softcap=softcap))
        batch.check(kv.Scoring(softcap=softcap))


@pytest.mark.parametrize("window", [0, 50])
@pytest.mark.parametrize("stride", [1, 60, 64, 399])
def test_sums_shorter_than_a_sequence(cuda_lib, window, stride):
    # tokens below the stride get their sums, the others none, and nothing past them is touched
    from test_gpu_canary import Guarded

    lens = [64, 400, 33]
    batch = Batch(lens, 8, 2, seed=22)
    scoring = kv.Scoring(window=window, sinks=4)
    weights = Guarded((3, 2, stride), torch.float32)
    before = np.random.default_rng(6).random((3, 2, stride), dtype=np.float32)
    weights.t.copy_(dev(before))
    batch.weighted(scoring, weights.t, 0.5)
    torch.cuda.synchronize()
    assert batch.status.item() == kv.NVFP4KV_DEVERR_LENGTH and weights.intact()
    w = weights.t.double().cpu().numpy()
    for b, h, refs in batch.refs(scoring):
        n = min(stride, lens[b])
        old = before[b, h].astype(np.float64)
        want, tol = sum(r["p"] for r in refs)[:n], sum(r["tol_p"] for r in refs)[:n]
        want = 0.5 * old[:n] + want
        check(w[b, h, :n], want, tol + 2.0 ** -22 * want, f"weights {b} {h}")
        assert np.array_equal(w[b, h, n:], old[n:])
