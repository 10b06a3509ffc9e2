"""Cache eviction: the kept tokens, their sums and their bytes, exactly; and a
decode that accumulates, evicts, appends and goes on over the packed cache."""
import numpy as np
import pytest
import torch

import oracle
import nvfp4_quantized_paged_quantize_gb300 as kv
from gpu_util import bf16_dev, dev, pool_host, status_word
from nvfp4_quantized_paged_quantize_gb300 import inputs
from scored_util import SCALE, check, decode_ref, evict_ref, page_tables, random_cache, random_q, sequence_rows
from test_gpu_canary import Guarded

pytestmark = pytest.mark.gpu


def heavy_tailed(shape, seed):
    rng = np.random.default_rng(seed)
    w = np.exp(rng.standard_normal(shape) * 2.5 - 4.0).astype(np.float32)
    return np.where(rng.random(shape) < 0.1, np.float32(0.0), w)


class Eviction:
    def __init__(self, lens, hkv, budget, first, recent, weights, seed=1, kept_extra=0):
        self.lens, self.hkv, self.budget, self.first, self.recent = list(lens), hkv, budget, first, recent
        self.w = weights
        kept_lens = [min(n, budget) for n in lens]
        self.table, used = page_tables(lens, seed)
        dst, more = page_tables([budget] * len(lens), seed + 1, first=used)
        self.dst = dst
        for b, n in enumerate(kept_lens):
            self.dst[b, (n + 15) // 16:] = -1                    # not written, so not looked at
        self.cache, self.oracle = random_cache(used + more, hkv, seed)
        self.cache.pages[used:] = 0xA5
        self.before = self.cache.pages.clone()
        B = len(lens)
        self.kept = Guarded((B, hkv, budget), torch.int32)
        self.kept_weights = Guarded((B, hkv, budget + kept_extra), torch.float32)
        self.new_lens = Guarded((B,), torch.int32)
        self.status = status_word()
        self.pt, self.sl, self.dpt, self.dw = dev(self.table), dev(np.asarray(lens, np.int32)), dev(self.dst), dev(weights)

    def run(self):
        kv.nvfp4kv_evict(self.cache, self.pt, self.sl, self.dw, self.budget, self.first, self.recent, self.dpt,
                         self.kept.t, self.kept_weights.t, self.new_lens.t, device_status=self.status)
        torch.cuda.synchronize()

    def check(self):
        assert self.status.item() == 0
        for g in (self.kept, self.kept_weights, self.new_lens):
            assert g.intact()
        kept, kw = self.kept.t.cpu().numpy(), self.kept_weights.t.cpu().numpy()
        after, pages = pool_host(self.cache), self.cache.pages
        src = [self.oracle.k_data, self.oracle.v_data, self.oracle.k_scale, self.oracle.v_scale]
        written = torch.zeros(self.cache.num_pages, dtype=torch.bool)
        for b, L in enumerate(self.lens):
            n = min(L, self.budget)
            assert self.new_lens.t[b].item() == n
            for h in range(self.hkv):
                want = evict_ref(self.w[b, h], L, self.budget, self.first, self.recent)
                assert np.array_equal(kept[b, h, :n], want), (b, h)
                assert (kept[b, h, n:] == -1).all()
                assert np.array_equal(kw[b, h, :n].view(np.uint32), self.w[b, h, want].view(np.uint32))
                assert not kw[b, h, n:self.budget].any()
                row = lambda table, t: (table[b, t // 16].astype(np.int64) * self.hkv + h) * 16 + t % 16  # noqa: E731
                slots = np.arange((n + 15) // 16 * 16)
                for got, was in zip(after, src):
                    rows = got[row(self.dst, slots)]
                    assert np.array_equal(rows[:n], was[row(self.table, want)]), (b, h)
                    assert not rows[n:].any()                    # the last page's rows behind the sequence
            written[self.dst[b, :(n + 15) // 16].astype(np.int64)] = True
        assert torch.equal(pages.cpu()[~written], self.before.cpu()[~written])   # every other page as it was


@pytest.mark.parametrize("budget,first,recent", [(64, 4, 16), (50, 0, 0), (33, 16, 17), (1, 0, 0), (1, 0, 1), (96, 96, 0),
                                                 (17, 1, 1)])
def test_eviction(cuda_lib, budget, first, recent):
    lens = [0, 1, 15, budget - 1, budget, budget + 1, 100, 257, 1000]
    w = heavy_tailed((len(lens), 3, 1003), budget)
    e = Eviction(lens, 3, budget, first, recent, w, seed=budget, kept_extra=5)
    e.run()
    e.check()


def test_ties_and_special_values(cuda_lib):
    n = 700
    rows = [np.zeros(n), np.full(n, -1.0), np.tile([1.0, 2.0], n // 2), np.where(np.arange(n) % 7 == 0, np.inf, 1.0),
            np.where(np.arange(n) % 5 == 0, np.nan, np.arange(n)), np.where(np.arange(n) % 2 == 0, 0.0, -0.0),
            np.linspace(-3, 3, n), np.full(n, 2.0 ** -149), -np.full(n, np.inf)]
    w = np.stack(rows).astype(np.float32)[:, None]
    w[4, 0, 3] = np.array([0xFFC00001], np.uint32).view(np.float32)[0]         # a negative NaN
    for budget in (100, 333, 650):
        e = Eviction([n] * len(rows), 1, budget, 3, 40, w, seed=budget)
        e.run()
        e.check()


@pytest.mark.parametrize("L,hkv", [(20000, 2), (20481, 1), (50000, 1), (170000, 1)])
def test_long_sequences(cuda_lib, L, hkv):
    # one CTA, clusters of several, and more keys than a full cluster holds at once
    lens = [L, L // 3]
    w = heavy_tailed((2, hkv, L), L)
    w = np.where(w > 0, np.float32(2.0) ** np.round(np.log2(np.maximum(w, 1e-9))), w).astype(np.float32)  # many ties
    e = Eviction(lens, hkv, L // 8 + 3, 5, L // 100, w, seed=L)
    e.run()
    e.check()


def test_many_pairs(cuda_lib):
    lens = np.random.default_rng(2).integers(0, 300, 150).tolist()
    e = Eviction(lens, 8, 100, 4, 20, heavy_tailed((150, 8, 300), 3), seed=7)
    e.run()
    e.check()


def test_optional_outputs_and_lengths_in_place(cuda_lib):
    lens = [300, 40]
    w = heavy_tailed((2, 2, 304), 4)
    e = Eviction(lens, 2, 64, 4, 16, w, seed=8)
    kv.nvfp4kv_evict(e.cache, e.pt, e.sl, e.dw, 64, 4, 16, e.dpt, e.kept.t, new_lens=e.sl, device_status=e.status)
    torch.cuda.synchronize()
    assert e.sl.tolist() == [64, 40]
    e.new_lens.t.copy_(e.sl)
    for b in range(2):
        for h in range(2):
            n = min(lens[b], 64)
            at = e.kept.t[b, h, :n].long()
            e.kept_weights.t[b, h, :n] = e.dw[b, h][at]
            e.kept_weights.t[b, h, n:] = 0
    e.check()


def test_bad_pages_and_lengths_are_flagged(cuda_lib):
    w = heavy_tailed((2, 1, 320), 5)
    e = Eviction([300, 300], 1, 64, 4, 16, w, seed=9)
    table, dst = e.table.copy(), e.dst.copy()
    table[1, 0] = 1 << 30                                        # the first tokens' page: zeros
    dst[0, 1] = -2                                               # not written
    e.pt, e.dpt = dev(table), dev(dst)
    e.run()
    assert e.status.item() == kv.NVFP4KV_DEVERR_PAGE
    got = pool_host(e.cache)
    assert not got[0][e.dst[1, 0] * 16: e.dst[1, 0] * 16 + 4].any()
    assert (e.cache.pages[int(e.dst[0, 1])] == 0xA5).all()
    assert (e.cache.pages[int(e.dst[0, 0])] != 0xA5).any()
    # lengths outside the table or the sums are cut
    for lens, want in (([-4, 400], [0, 64]), ([300, 321], [64, 64])):
        e = Eviction([300, 300], 1, 64, 4, 16, w, seed=9)
        e.sl = dev(np.asarray(lens, np.int32))
        e.run()
        assert e.status.item() == kv.NVFP4KV_DEVERR_LENGTH
        assert e.new_lens.t.tolist() == want


def test_capture(cuda_lib):
    w = heavy_tailed((2, 2, 30000), 6)
    e = Eviction([30000, 500], 2, 200, 4, 16, w, seed=10)
    e.run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kv.nvfp4kv_evict(e.cache, e.pt, e.sl, e.dw, 200, 4, 16, e.dpt, e.kept.t, e.kept_weights.t, e.new_lens.t,
                         device_status=e.status)
    w2 = heavy_tailed((2, 2, 30000), 61)
    e.dw.copy_(dev(w2))
    e.kept.t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    e.w = w2
    e.check()


def test_decode_evict_append_decode(cuda_lib):
    """As a server would use them: decode steps that accumulate weights, an eviction into fresh pages, the next
    token appended behind the survivors, and a decode over the packed cache."""
    lens, hq, hkv, budget = [333, 50], 8, 2, 96
    table, used = page_tables(lens, 20)
    dst, more = page_tables([budget + 16] * 2, 21, first=used)
    cache, o = random_cache(used + more, hkv, 20)
    pt, sl = dev(table), dev(np.asarray(lens, np.int32))
    weights = torch.zeros((2, hkv, 352), device="cuda")
    status = status_word()
    ws = torch.empty(kv.nvfp4kv_decode_weights_workspace_size(cache, 2, hq, used + more), dtype=torch.uint8, device="cuda")
    out = torch.empty((2, hq, 128), dtype=torch.bfloat16, device="cuda")
    scoring = kv.Scoring(softcap=30.0)
    want = np.zeros((2, hkv, 352))
    for step in range(3):
        q, q64 = random_q((2, hq, 128), 30 + step, 2.0)
        kv.nvfp4kv_decode_attention_weights(cache, q, out, pt, sl, SCALE, weights, ws, scoring=scoring,
                                            device_status=status)
        for b in range(2):
            for i in range(hq):
                K, V = sequence_rows(o, table[b], i // 4, lens[b])
                want[b, i // 4, :lens[b]] += decode_ref(K, V, q64[b, i], lens[b], scoring)["p"]
    kept = torch.empty((2, hkv, budget), dtype=torch.int32, device="cuda")
    left = torch.zeros((2, hkv, budget + 16), device="cuda")
    kv.nvfp4kv_evict(cache, pt, sl, weights, budget, 4, 32, dev(dst), kept, left, sl, device_status=status)
    torch.cuda.synchronize()
    w = weights.cpu().numpy()
    np.testing.assert_allclose(w, want, rtol=2.0 ** -10, atol=2.0 ** -40)
    assert sl.tolist() == [budget, 50]
    # the next token
    rng = np.random.default_rng(40)
    k, v = (inputs.bf16_bits(rng.standard_normal((2, hkv, 128)).astype(np.float32)) for _ in range(2))
    slots = np.array([dst[b, n // 16].astype(np.int64) * 16 + n % 16 for b, n in enumerate([budget, 50])])
    kv.nvfp4kv_quantize_append(cache, bf16_dev(k), bf16_dev(v), dev(slots), device_status=status)
    sl += 1
    q, q64 = random_q((2, hq, 128), 50, 2.0)
    dws = torch.empty(kv.nvfp4kv_decode_weights_workspace_size(cache, 2, hq, used + more), dtype=torch.uint8,
                      device="cuda")
    before = left.cpu().numpy().astype(np.float64)
    kv.nvfp4kv_decode_attention_weights(cache, q, out, dev(dst), sl, SCALE, left, dws, scoring=scoring,
                                        device_status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    fresh = oracle.Cache(2, hkv, 128, 16)
    assert oracle.quantize_append(fresh, k, v, np.array([0, 16])) == 0
    got, after = out.double().cpu().numpy(), left.double().cpu().numpy()
    for b, n in enumerate([budget, 50]):
        for h in range(hkv):
            idx = evict_ref(w[b, h], lens[b], budget, 4, 32)
            assert np.array_equal(kept[b, h, :n].cpu().numpy(), idx)
            K, V = sequence_rows(o, table[b], h, lens[b])
            row = [(b * hkv + h) * 16]
            K = np.concatenate([K[idx], oracle.dequantize_rows(fresh, "k", row)])
            V = np.concatenate([V[idx], oracle.dequantize_rows(fresh, "v", row)])
            refs = [decode_ref(K, V, q64[b, h * 4 + g], n + 1, scoring) for g in range(4)]
            for g, r in enumerate(refs):
                check(got[b, h * 4 + g], r["out"], r["tol_out"], f"{b} {h} {g}")
            total = before[b, h, :n + 1] + sum(r["p"] for r in refs)
            check(after[b, h, :n + 1], total, sum(r["tol_p"] for r in refs) + 2.0 ** -22 * total, "sums")
