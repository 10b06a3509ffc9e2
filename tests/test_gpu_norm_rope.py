"""The normed and rotated append: queries, cache bytes and workspace bytes, bit
for bit, and against 64 bits."""
import numpy as np
import pytest
import torch

import oracle
import nvfp4_quantized_paged_quantize_gb300 as kv
from gpu_util import dev, pool_host, status_word
from step_util import bf16_round, bits, norm_rope_exact, norm_rope_steps, same
from test_gpu_canary import Guarded

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
EPS = 1e-5
PARTS = ("k_data", "v_data", "k_scale", "v_scale")


def table_of(max_position, rot):
    half = rot // 2
    angle = np.arange(max_position)[:, None] * 10000.0 ** (-np.arange(half) / half)
    return np.concatenate([np.cos(angle), np.sin(angle)], -1).astype(np.float32)


class Append:
    def __init__(self, n, hq, hkv, rot=128, interleaved=False, norms=(True, True), fp8=True, packed=True, seed=1, pages=None,
                 slots=None, ws=(1.0, 1.0), g=(0.0043, 0.0031), size=1.0):
        rng = np.random.default_rng(seed)
        self.n, self.hq, self.hkv, self.inter, self.ws, self.size = n, hq, hkv, interleaved, ws, size
        x = rng.standard_normal((n, hq + 2 * hkv, 128)) * 2.0 ** rng.integers(-4, 5, (n, hq + 2 * hkv, 1)) * size
        x[rng.random(x.shape) < 0.02] = 0.0
        if n > 1:
            x[1] = 0.0                                        # a token of zeros, its norm eps alone
        x[0, :, 16:32] = 0.0                                  # and a block of them
        x[0, :, 32:48] = -0.0
        self.x = bf16_round(x)
        wide = hq + 2 * hkv + (1 if packed else 0)            # a gap between tokens
        self.qkv = torch.full((n, wide, 128), float("nan"), dtype=BF16, device="cuda")
        self.qkv[:, :hq + 2 * hkv] = torch.from_numpy(self.x).to(BF16).cuda()
        parts = self.qkv[:, :hq], self.qkv[:, hq:hq + hkv], self.qkv[:, hq + hkv:hq + 2 * hkv]
        self.q, self.k, self.v = parts if packed else (t.contiguous() for t in parts)
        self.weights = [bf16_round(1 + 0.4 * rng.standard_normal(128)) if on else None for on in norms]
        self.dw = [None if w is None else torch.from_numpy(w).to(BF16).cuda() for w in self.weights]
        self.max_position = 700
        self.cs = table_of(self.max_position, rot) if rot else None
        self.pos = rng.integers(0, self.max_position, n).astype(np.int32)
        self.pages = pages or (n + 15) // 16 + 1
        self.slots = rng.permutation(self.pages * 16)[:n].astype(np.int64) if slots is None else np.asarray(slots, np.int64)
        self.g = tuple(float(np.float32(v)) for v in g)
        self.pool = Guarded((self.pages, hkv, kv.NVFP4KV_PAGE_HEAD_BYTES), torch.uint8)
        self.pool.t.random_(0, 256, generator=torch.Generator("cuda").manual_seed(seed))
        self.cache = kv.Cache(self.pool.t, self.pages, hkv, *self.g)
        self.before = [a.copy() for a in pool_host(self.cache)]
        self.q_out = Guarded((n, hq, 128), BF16)
        self.fp8 = fp8
        self.total = n + 5
        self.ws_rows = rng.permutation(self.total)[:n].astype(np.int64)
        self.wk, self.wv = (Guarded((self.total, hkv, 128), torch.uint8) for _ in range(2))
        self.wk.t.fill_(0x55)
        self.wv.t.fill_(0x55)
        self.status = status_word()

    def run(self, q_out=None):
        kv.nvfp4kv_norm_rope_append(self.cache, self.q, self.k, self.v, dev(self.slots), dev(self.pos),
                                    None if self.cs is None else dev(self.cs), self.q_out.t if q_out is None else q_out,
                                    q_weight=self.dw[0], k_weight=self.dw[1], eps=EPS, interleaved=self.inter,
                                    ws_rows=dev(self.ws_rows) if self.fp8 else None, ws_k=self.wk.t, ws_v=self.wv.t,
                                    k_ws_scale=self.ws[0], v_ws_scale=self.ws[1], device_status=self.status)
        torch.cuda.synchronize()

    def check(self, flags=0, q_out=None):
        assert self.status.item() == flags
        for g in (self.pool, self.q_out, self.wk, self.wv):
            assert g.intact()
        hq, hkv = self.hq, self.hkv
        qx, kx, vx = self.x[:, :hq], self.x[:, hq:hq + hkv], self.x[:, hq + hkv:]
        made = [bf16_round(norm_rope_steps(a, w, EPS, self.cs, self.pos, self.inter)) for a, w in zip((qx, kx), self.weights)]
        got = (self.q_out.t if q_out is None else q_out).float().cpu().numpy()
        same(bits(got), bits(made[0]), "queries")
        ok = (self.pos >= 0) & (self.pos < self.max_position)
        want, tol = norm_rope_exact(qx[ok], self.weights[0], EPS, self.cs, self.pos[ok], self.inter)
        assert (np.abs(got[ok] - want) <= tol).all()
        # the cache, as quantising those rows would leave it
        ref = oracle.Cache(self.pages, hkv, 128, 16, *self.g, arrays=[a.copy() for a in self.before])
        oracle.quantize_append(ref, bits(made[1]), bits(vx), self.slots)
        for name, a, b in zip(PARTS, pool_host(self.cache), (ref.k_data, ref.v_data, ref.k_scale, ref.v_scale)):
            same(a, b, name)
        wk, wv = (np.full((self.total, hkv, 128), 0x55, np.uint8) for _ in range(2))
        if self.fp8:
            oracle.bf16_to_fp8_workspace(bits(made[1]), bits(vx), self.ws_rows, wk, wv, *self.ws)
        same(self.wk.t.cpu().numpy(), wk, "workspace keys")
        same(self.wv.t.cpu().numpy(), wv, "workspace values")


@pytest.mark.parametrize("n,hq,hkv", [(1, 8, 1), (1, 1, 1), (2, 8, 2), (3, 5, 5), (17, 6, 3), (33, 64, 8), (130, 10, 2)])
def test_append(cuda_lib, n, hq, hkv):
    a = Append(n, hq, hkv, seed=n + hq)
    a.run()
    a.check()


@pytest.mark.parametrize("rot", [0, 32, 64, 96, 128])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norms", [(True, True), (False, True), (True, False), (False, False)])
def test_rotations_and_norms(cuda_lib, rot, interleaved, norms):
    a = Append(21, 4, 2, rot, interleaved, norms, fp8=rot % 64 == 0, packed=interleaved, seed=rot + 2 * interleaved)
    a.run()
    a.check()


def test_several_rows_to_a_group(cuda_lib):
    # enough rows that every 8-lane group takes two or four, tokens ending inside one; in-order slots pair up values
    for n, hq, hkv, start in ((2100, 7, 1, 0), (3001, 8, 1, 1), (801, 64, 8, 5)):
        a = Append(n, hq, hkv, seed=n, slots=np.arange(start, start + n), pages=(start + n) // 16 + 1)
        a.run()
        a.check()


def test_values_of_every_size(cuda_lib):
    # far below eps, subnormal squares, and large; workspace scales other than one; scales that flush blocks to zero
    for size in (2.0 ** -60, 2.0 ** -20, 2.0 ** 40):
        a = Append(12, 4, 2, size=size, norms=(True, True), seed=7, ws=(0.37, 2.0 ** -9), g=(0.01, 1e30 if size < 1 else 2.0 ** 35))
        a.run()
        a.check()


def test_padding_and_bad_indices(cuda_lib):
    a = Append(40, 8, 2, seed=11)
    a.slots[[0, 7, 8, 39]] = -1
    a.slots[20] = a.pages * 16
    a.slots[21] = 1 << 40
    a.ws_rows[[3, 39]] = -1
    a.ws_rows[4] = a.total
    a.pos[5], a.pos[6] = -1, a.max_position
    a.run()
    a.check(kv.NVFP4KV_DEVERR_SLOT | kv.NVFP4KV_DEVERR_ROW | kv.NVFP4KV_DEVERR_POSITION)


def test_queries_in_place(cuda_lib):
    for packed in (True, False):
        a = Append(300, 9, 3, packed=packed, seed=12)
        a.run(q_out=a.q)
        a.check(q_out=a.q)
        if packed:                                            # the gap between tokens is as it was
            assert torch.isnan(a.qkv[:, -1]).all()


def test_nothing_to_do(cuda_lib):
    a = Append(4, 8, 2, seed=13)
    empty = a.q[:0]
    kv.nvfp4kv_norm_rope_append(a.cache, empty, a.k[:0], a.v[:0], dev(a.slots[:0]), dev(a.pos[:0]), dev(a.cs), empty,
                                q_weight=a.dw[0], k_weight=a.dw[1], device_status=a.status)
    torch.cuda.synchronize()
    assert a.status.item() == 0
    for name, x, y in zip(PARTS, pool_host(a.cache), a.before):
        same(x, y, name)


def test_the_parts_are_those_of_the_other_calls(cuda_lib):
    # no norm, no rotation: the queries as they are, the cache as nvfp4kv_quantize_append leaves it
    a = Append(100, 8, 4, rot=0, norms=(False, False), fp8=False, packed=False, seed=14)
    a.run()
    a.check()
    other = kv.Cache.empty(a.pages, a.hkv, k_global_scale=a.g[0], v_global_scale=a.g[1])
    other.pages.random_(0, 256, generator=torch.Generator("cuda").manual_seed(14))
    kv.nvfp4kv_quantize_append(other, a.k, a.v, dev(a.slots))
    assert torch.equal(other.pages, a.cache.pages) and torch.equal(a.q_out.t, a.q)


def test_capture_on_another_stream(cuda_lib):
    a = Append(50, 8, 2, seed=15)
    slots, pos, cs = dev(a.slots), dev(a.pos), dev(a.cs)
    rows = dev(a.ws_rows)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        kv.nvfp4kv_norm_rope_append(a.cache, a.q, a.k, a.v, slots, pos, cs, a.q_out.t, q_weight=a.dw[0], k_weight=a.dw[1],
                                    eps=EPS, ws_rows=rows, ws_k=a.wk.t, ws_v=a.wv.t, device_status=a.status)
    graph.replay()
    graph.replay()                                            # writing the same bytes again changes nothing
    torch.cuda.synchronize()
    a.check()


def test_tokens_far_apart(cuda_lib):
    # rows whose offsets pass 2^31 elements, of the queries, keys and values and of the result
    a = Append(3, 2, 1, packed=False, seed=16)
    far = (1 << 30) + 128
    big = torch.empty(2 * far + 512, dtype=BF16, device="cuda")
    rows = big.as_strided((3, 4, 128), (far, 128, 1))
    for h, part in ((0, a.q), (2, a.k), (3, a.v)):
        rows[:, h:h + part.shape[1]] = part
    a.q, a.k, a.v = rows[:, :2], rows[:, 2:3], rows[:, 3:4]
    a.run(q_out=a.q)
    a.check(q_out=a.q)
