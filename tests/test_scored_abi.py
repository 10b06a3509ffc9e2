"""Host-side refusals of the scored attention calls and the eviction (no GPU:
every check here returns before anything touches CUDA), and the references the
GPU tests use, pinned to torch's own attention."""
import ctypes

import numpy as np
import pytest
import torch

import nvfp4_quantized_paged_quantize_gb300 as kv

INVALID, UNSUPPORTED, OK = kv.NVFP4KV_ERR_INVALID_ARGUMENT, kv.NVFP4KV_ERR_UNSUPPORTED, kv.NVFP4KV_OK


@pytest.fixture(scope="module")
def lib():
    return kv.load()


def _cache(**kw):
    c = kv.Cache(0x10000, 4, 2)
    for k, v in kw.items():
        setattr(c, k, v)
    return c.c_struct()


def _call(fn, good):
    def call(**kw):
        a = list(good)
        for k, v in kw.items():
            a[int(k[1:])] = v
        return fn(*a)
    return call


BAD_SCORINGS = [dict(softcap=-1.0), dict(softcap=float("nan")), dict(softcap=float("inf")), dict(softcap=1e-9),
                dict(softcap=2e6), dict(window=-1), dict(sinks=-1, window=5), dict(slopes=0x1001)]


def test_scored_decode_refusals(lib):
    cs = ctypes.byref(_cache())
    sc = kv.Scoring(softcap=1.0).c_struct()
    # (cache, q, out, lse, page_table, max_pages, seq_lens, batch, hq, scale, scoring, ws, ws_bytes, status, stream)
    call = _call(lib.nvfp4kv_decode_attention_scored,
                 [cs, 16, 16, 4, 4, 1, 4, 0, 8, 0.1, ctypes.byref(sc), 256, 1 << 20, None, None])
    assert call() == OK                                                        # an empty batch
    for bad in BAD_SCORINGS:
        assert call(a10=ctypes.byref(kv.Scoring(**bad).c_struct())) == INVALID, bad
    assert call(a0=None) == INVALID and call(a3=6) == INVALID and call(a8=7) == INVALID
    assert call(a8=18) == UNSUPPORTED                                          # nine query heads per KV head
    assert call(a9=float("nan")) == INVALID and call(a7=-1) == INVALID
    assert call(a7=1, a1=None) == INVALID and call(a7=1, a2=24) == INVALID     # null q, misaligned out
    assert call(a0=ctypes.byref(_cache(head_dim=64))) == UNSUPPORTED
    assert call(a10=None) == OK                                                # no scoring


def test_weights_refusals(lib):
    cs = ctypes.byref(_cache())
    # (..., scale, scoring, weights, stride, decay, max_total_pages, ws, ws_bytes, status, stream)
    call = _call(lib.nvfp4kv_decode_attention_weights,
                 [cs, 16, 16, None, 4, 1, 4, 0, 8, 0.1, None, 4, 16, 1.0, 4, 256, 1 << 20, None, None])
    assert call() == OK
    assert call(a12=0) == INVALID and call(a13=-0.5) == INVALID and call(a13=float("nan")) == INVALID
    assert call(a13=float("inf")) == INVALID and call(a14=-1) == INVALID
    n = ctypes.c_size_t()
    size = lib.nvfp4kv_decode_weights_workspace_size
    assert size(cs, 1, 8, 4, None) == INVALID and size(None, 1, 8, 4, ctypes.byref(n)) == INVALID
    assert size(cs, -1, 8, 4, ctypes.byref(n)) == INVALID and size(cs, 1, 7, 4, ctypes.byref(n)) == INVALID
    assert size(cs, 1, 8, -1, ctypes.byref(n)) == INVALID and size(cs, 1, 18, 4, ctypes.byref(n)) == UNSUPPORTED
    assert size(cs, 1, 8, 1 << 40, ctypes.byref(n)) == UNSUPPORTED


def test_scored_extend_refusals(lib):
    good = [16, 8, 4, 16, 16, 8, 4, 2, 100, 8, 2, 128, 1.0, 1.0, 0.1, None, None, None, 16, None, None, None]
    call = _call(lib.nvfp4kv_extend_attention_scored, good)
    for bad in BAD_SCORINGS:
        assert call(a15=ctypes.byref(kv.Scoring(**bad).c_struct())) == INVALID, bad
    assert call(a9=6) == UNSUPPORTED and call(a9=7) == INVALID and call(a11=64) == UNSUPPORTED
    assert call(a16=6) == INVALID and call(a17=2) == INVALID and call(a19=1) == INVALID   # misaligned masks, lse
    assert call(a18=None) == INVALID and call(a18=24) == INVALID
    assert call(a7=0) == OK and call(a2=0) == OK


def test_eviction_refusals(lib):
    cs = ctypes.byref(_cache())
    # (cache, pt, max_pages, lens, batch, weights, stride, budget, first, recent, dst_pt, dst_max, kept, kw, kw_stride,
    #  new_lens, status, stream)
    call = _call(lib.nvfp4kv_evict, [cs, 4, 8, 4, 0, 4, 128, 64, 4, 16, 4, 4, 4, 4, 64, 4, None, None])
    assert call() == OK
    assert call(a7=0) == INVALID and call(a8=-1) == INVALID and call(a9=-1) == INVALID
    assert call(a8=49) == INVALID                                              # first + recent > budget
    assert call(a8=2 ** 31 - 1, a9=2 ** 31 - 1) == INVALID                     # whose sum passes 32 bits
    assert call(a11=3) == INVALID                                              # too few destination pages
    assert call(a14=63) == INVALID and call(a13=None, a14=0) == OK
    assert call(a2=0) == INVALID and call(a6=0) == INVALID and call(a4=-1) == INVALID
    assert call(a4=1, a12=None) == INVALID and call(a4=1, a10=None) == INVALID and call(a4=1, a5=6) == INVALID
    assert call(a4=1, a2=1 << 27) == UNSUPPORTED                               # tokens past 32 bits
    assert call(a4=1, a1=64, a10=64) == INVALID                                # packed into the old pages
    assert call(a4=1, a5=4096, a13=4096, a10=64) == INVALID                    # kept sums over the old ones
    assert call(a4=1, a5=4096, a13=4096 + 4 * (2 * 128 - 1), a10=64) == INVALID
    assert call(a4=1, a5=4096, a13=4096 - 4 * (2 * 64 - 1), a10=64) == INVALID
    assert call(a0=ctypes.byref(_cache(page_size=32))) == UNSUPPORTED


def test_bindings_refuse_wrong_tensors():
    # tensors that are not on the GPU, or of another type or shape, never reach the library
    c = kv.Cache(torch.zeros((4, 2, 2304), dtype=torch.uint8), 4, 2)
    q = torch.zeros((1, 8, 128), dtype=torch.bfloat16)
    table, lens = torch.zeros((1, 4), dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    out, ws = torch.zeros_like(q), torch.zeros(1 << 10, dtype=torch.uint8)
    for args in ((q, out, table, lens), (q.float(), out, table, lens), (q, out.float(), table, lens),
                 (q, out, table.long(), lens), (q[:, ::2], out[:, ::2], table, lens)):
        with pytest.raises(ValueError):
            kv.nvfp4kv_decode_attention_scored(c, *args, 0.1, ws)
        with pytest.raises(ValueError):
            kv.nvfp4kv_decode_attention_weights(c, *args, 0.1, torch.zeros((1, 2, 64)), ws)
    with pytest.raises(ValueError):
        kv.nvfp4kv_evict(c, table, lens, torch.zeros((1, 2, 64)), 16, 0, 0, table, torch.zeros((1, 2, 16), dtype=torch.int32))
    with pytest.raises(ValueError):
        mx = kv.Cache(torch.zeros((4, 2, 2176), dtype=torch.uint8), 4, 2, mxfp4=True)
        kv.nvfp4kv_decode_attention_scored(mx, q, out, table, lens, 0.1, ws)


def test_reference_attention_matches_torch():
    from scored_util import attend, extend_seen

    rng = np.random.default_rng(1)
    K, V, q = rng.standard_normal((50, 128)), rng.standard_normal((50, 128)), rng.standard_normal(128)
    for scoring, kw in ((kv.Scoring(), {}), (kv.Scoring(window=7, sinks=3), {}), (kv.Scoring(), dict(full=45)),
                        (kv.Scoring(window=9, sinks=2), dict(doc=20))):
        seen = extend_seen(30, 20, 5, scoring, **kw)
        p = 35
        want = [j for j in range(50) if j <= max(p, kw.get("full", 0) - 1) and j >= kw.get("doc", 0) and
                (not scoring.window or p - j < scoring.window or j < kw.get("doc", 0) + scoring.sinks)]
        assert np.flatnonzero(seen).tolist() == want
        bias = -0.25 * np.abs(p - np.arange(50.0))
        got = attend(q, K, V, seen, np.abs(p - np.arange(50.0)), 0.1, slope=0.25)
        mask = torch.from_numpy(np.where(seen, bias, -np.inf))[None]
        ref = torch.nn.functional.scaled_dot_product_attention(
            torch.from_numpy(q)[None, None], torch.from_numpy(K)[None], torch.from_numpy(V)[None], attn_mask=mask, scale=0.1)
        np.testing.assert_allclose(got["out"], ref[0, 0].numpy(), rtol=1e-10, atol=1e-12)
        x = np.where(seen, 0.1 * (K @ q) + bias, -np.inf)
        np.testing.assert_allclose(got["lse"], torch.logsumexp(torch.from_numpy(x), 0).item(), rtol=1e-12)
    # the cap, and a row that sees nothing
    got = attend(q, K, V, np.ones(50, bool), np.zeros(50), 0.1, softcap=2.0)
    x = 2.0 * np.tanh(0.1 * (K @ q) / 2.0)
    np.testing.assert_allclose(got["out"], torch.softmax(torch.from_numpy(x), 0).numpy() @ V, rtol=1e-10, atol=1e-12)
    empty = attend(q, K, V, np.zeros(50, bool), np.zeros(50), 0.1)
    assert not empty["out"].any() and empty["lse"] == -np.inf


def test_eviction_refuses_lengths_at_an_offset(lib):
    cs = ctypes.byref(_cache())
    call = _call(lib.nvfp4kv_evict,
                 [cs, 64, 8, 4096, 3, 1 << 20, 128, 64, 4, 16, 128, 4, 4, None, 0, 4, None, None])
    assert call(a15=4100) == INVALID and call(a15=4096 - 8) == INVALID


def test_bindings_refuse_tensors_of_another_gpu(monkeypatch):
    class OnGpu:
        """What the checks look at of a tensor, on GPU `gpu`."""
        is_cuda = True

        def __init__(self, dtype, shape, gpu):
            self.dtype, self.shape, self.gpu, self.device = dtype, shape, gpu, f"cuda:{gpu}"

        def dim(self):
            return len(self.shape)

        def is_contiguous(self):
            return True

        def get_device(self):
            return self.gpu

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    c = kv.Cache(0x10000, 4, 2)
    i32, bf16, f32 = torch.int32, torch.bfloat16, torch.float32
    decode = [(bf16, (1, 8, 128)), (bf16, (1, 8, 128)), (i32, (1, 4)), (i32, (1,))]
    evict = [(i32, (1, 4)), (i32, (1,)), (f32, (1, 2, 64)), (i32, (1, 4)), (i32, (1, 2, 16))]
    for k in range(4):
        t = [OnGpu(*a, gpu=int(i == k)) for i, a in enumerate(decode)]
        with pytest.raises(ValueError, match="got .* on cuda:1"):
            kv.nvfp4kv_decode_attention_scored(c, *t, 0.1, None, workspace_bytes=0)
    for k in range(5):
        t = [OnGpu(*a, gpu=int(i == k)) for i, a in enumerate(evict)]
        with pytest.raises(ValueError, match="got .* on cuda:1"):
            kv.nvfp4kv_evict(c, t[0], t[1], t[2], 16, 0, 0, t[3], t[4])
    # the pool and the workspace
    other, t = OnGpu(torch.uint8, (4, 2, 2304), 1), [OnGpu(*a, gpu=0) for a in decode]
    with pytest.raises(ValueError, match="cache.pages: .* got cuda:1"):
        kv.nvfp4kv_decode_attention_scored(kv.Cache(other, 4, 2), *t, 0.1, None, workspace_bytes=0)
    with pytest.raises(ValueError, match="workspace: .* got cuda:1"):
        kv.nvfp4kv_decode_attention_scored(c, *t, 0.1, other, workspace_bytes=0)


def test_eviction_refuses_budgets_that_its_loops_cannot_count(lib):
    # a cluster's loops over a budget step by up to 4096 in 32 bits
    cs = ctypes.byref(_cache())
    pages = 1 << 27
    call = _call(lib.nvfp4kv_evict,
                 [cs, 64, 8, 4096, 1, 1 << 20, 128, 2 ** 31 - 1, 4, 16, 128, pages, 4, None, 0, None, None, None])
    for over in (2 ** 31 - 1, 2 ** 31 - 4095):
        assert call(a7=over, a12=None) == UNSUPPORTED, over
    assert call(a7=2 ** 31 - 4096, a12=None) == INVALID        # only the missing list is refused


class OnGpu:
    """What the bindings' checks look at of a tensor, on GPU `gpu` (-1: on the CPU)."""

    def __init__(self, dtype, shape, gpu=0):
        self.dtype, self.shape, self.gpu = dtype, shape, gpu
        self.device, self.is_cuda = f"cuda:{gpu}" if gpu >= 0 else "cpu", gpu >= 0

    def dim(self):
        return len(self.shape)

    def is_contiguous(self):
        return True

    def get_device(self):
        return self.gpu


@pytest.mark.parametrize("gpu", [1, -1])
def test_bindings_refuse_a_status_word_elsewhere(monkeypatch, gpu):
    # the kernels write it, so it has to be memory of the current GPU too
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    c, status = kv.Cache(0x10000, 4, 2), OnGpu(torch.int32, (1,), gpu)
    i32, i64, bf16, f32, u8 = torch.int32, torch.int64, torch.bfloat16, torch.float32, torch.uint8
    q, out, table, lens, sums = (OnGpu(*a) for a in ((bf16, (1, 8, 128)), (bf16, (1, 8, 128)), (i32, (1, 4)), (i32, (1,)),
                                                     (f32, (1, 2, 64))))
    ws = OnGpu(u8, (5, 2, 128))
    calls = [
        lambda: kv.nvfp4kv_decode_attention_scored(c, q, out, table, lens, 0.1, None, workspace_bytes=0,
                                                   device_status=status),
        lambda: kv.nvfp4kv_decode_attention_weights(c, q, out, table, lens, 0.1, sums, None, workspace_bytes=0,
                                                    device_status=status),
        lambda: kv.nvfp4kv_extend_attention_scored(q, OnGpu(i64, (2,)), 1, ws, ws, OnGpu(i64, (2,)), lens, out, 0.1,
                                                   device_status=status),
        lambda: kv.nvfp4kv_evict(c, table, lens, sums, 16, 0, 0, OnGpu(i32, (1, 4)), OnGpu(i32, (1, 2, 16)),
                                 device_status=status),
    ]
    for call in calls:
        with pytest.raises(ValueError, match="device_status: "):
            call()


def test_streams_and_devices_without_torchs_private_calls(monkeypatch):
    # the bindings take a shortcut where torch has it; the public calls do without
    class Stream:
        cuda_stream = 0x1234

    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    monkeypatch.delattr(torch._C, "_cuda_getDevice", raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: Stream)
    assert kv._stream(None) == 0x1234 and kv._stream(Stream) == 0x1234 and kv._stream(7) == 7
    assert kv._current_gpu(OnGpu(torch.int32, (1,))) == 3
