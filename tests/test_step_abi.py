"""Host-side refusals of the step plan, the normed and rotated append and the
page selection (no GPU: every check here returns before anything touches CUDA),
and their references, pinned on the CPU."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
import nvfp4_quantized_paged_quantize_gb300 as kv
import step_util as su

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


def test_plan_refusals(lib):
    # (table, max_pages, cached, new, batch, free, capacity, count, num_pages, tokens, lens, slots, positions, cu_q, rows,
    #  cu_prefix, left, status, stream); a null free count is refused last but for the aliases
    good = [64, 8, 128, 256, 2, 512, 16, None, 100, 64, 1024, 2048, 4096, 8, 8, 8, 4, None, None]
    call = _call(lib.nvfp4kv_plan_append, good)
    assert call() == INVALID                                                   # no free count
    for bad in (dict(a1=0), dict(a4=-1), dict(a6=-1), dict(a8=0), dict(a9=-1)):
        assert call(a7=4, **bad) == INVALID, bad
    for big in (dict(a1=1 << 27), dict(a9=(1 << 31) - 1), dict(a9=(1 << 31) - (1 << 18)), dict(a8=1 << 27), dict(a4=1 << 30),
                dict(a6=(1 << 30) + 1)):
        assert call(a7=4, **big) == UNSUPPORTED, big
    for missing in (0, 2, 3, 5, 10, 11, 16):
        assert call(a7=4, **{f"a{missing}": None}) == INVALID, missing
    for odd in (0, 2, 3, 5, 7, 10, 12, 16):
        assert call(**{"a7": 4, f"a{odd}": 6}) == INVALID, odd
    for odd in (11, 13, 14, 15):
        assert call(**{"a7": 4, f"a{odd}": 12}) == INVALID, odd
    # lengths on top of one another, but not in place
    assert call(a7=4, a10=132) == INVALID and call(a7=4, a10=124) == INVALID
    assert call(a7=4, a10=256) == INVALID and call(a7=4, a10=260) == INVALID


def test_norm_rope_refusals(lib):
    cs = ctypes.byref(_cache())

    def how(**kw):
        h = kv._CNormRope(16, 16, 1e-6, 128, 0)
        for k, v in kw.items():
            setattr(h, k, v)
        return ctypes.byref(h)

    # (cache, q, q_stride, k, k_stride, v, v_stride, hq, n, slots, positions, cos_sin, max_pos, how, q_out, q_out_stride,
    #  ws_rows, rows, k_ws, v_ws, ws_k, ws_v, status, stream)
    good = [cs, 16, 1536, 16, 1536, 16, 1536, 8, 0, 8, 4, 16, 100, how(), 1 << 20, 1024, None, 0, 1.0, 1.0, None, None,
            None, None]
    call = _call(lib.nvfp4kv_norm_rope_append, good)
    assert call() == OK                                                        # no tokens
    assert call(a0=None) == INVALID and call(a13=None) == INVALID and call(a7=0) == INVALID and call(a8=-1) == INVALID
    for rot in (-32, 16, 48, 127, 160):
        assert call(a13=how(rotary_dim=rot)) == UNSUPPORTED, rot
    for eps in (0.0, -1e-6, float("nan"), float("inf")):
        assert call(a13=how(eps=eps)) == INVALID, eps
    assert call(a13=how(eps=0.0, q_weight=None, k_weight=None)) == OK          # no norms, no eps
    assert call(a13=how(q_weight=8)) == INVALID and call(a13=how(k_weight=24)) == INVALID
    assert call(a12=0) == INVALID and call(a12=0, a13=how(rotary_dim=0)) == OK
    for k, low in ((2, 1024), (15, 1024), (4, 256), (6, 256)):                  # tokens that run into one another; odd strides
        assert call(**{f"a{k}": low}) == OK
        assert call(**{f"a{k}": low - 8}) == INVALID and call(**{f"a{k}": low + 4}) == INVALID, k
    assert call(a16=8, a18=0.0) == INVALID and call(a16=8, a19=float("nan")) == INVALID and call(a16=8, a17=-1) == INVALID
    # with tokens, up to the last check before the GPU is asked (the queries' overlap)
    some = _call(lib.nvfp4kv_norm_rope_append, good[:8] + [3, *good[9:15], 1024, *good[16:]])
    assert some(a8=1 << 28) == UNSUPPORTED and some(a2=(1 << 40) + 8) == UNSUPPORTED
    for missing in (1, 3, 5, 9, 10, 11, 14):
        assert some(**{f"a{missing}": None}) == INVALID, missing
    for odd in (1, 3, 5, 11, 14):
        assert some(**{f"a{odd}": 24}) == INVALID, odd
    assert some(a9=4) == INVALID and some(a10=2) == INVALID
    assert some(a16=8) == INVALID and some(a16=8, a17=5, a20=16, a21=24) == INVALID and some(a16=4, a17=5, a20=16, a21=16) == INVALID
    assert some(a14=16) == INVALID                                             # in place, with another stride
    assert some(a14=16 + 2 * 1024) == INVALID                                  # across the next token's
    assert some(a1=1 << 20, a14=(1 << 20) - 16) == INVALID
    wide = ((1 << 20) + 4) * 128
    assert some(a7=(1 << 20) + 4, a8=1, a2=wide, a15=wide) == UNSUPPORTED      # more heads than offsets in a token count


def test_digest_and_score_refusals(lib):
    cs = ctypes.byref(_cache())
    # (cache, table, max_pages, lens, first, batch, digest, status, stream)
    call = _call(lib.nvfp4kv_page_digest, [cs, 4, 8, 4, None, 0, 16, None, None])
    assert call() == OK
    assert call(a0=None) == INVALID and call(a2=0) == INVALID and call(a5=-1) == INVALID and call(a7=2) == INVALID
    assert call(a4=6) == INVALID
    for missing in (1, 3, 6):
        assert call(**{"a5": 1, f"a{missing}": None}) == INVALID
    assert call(a5=1, a1=6) == INVALID and call(a5=1, a3=6) == INVALID and call(a5=1, a6=24) == INVALID
    assert call(a5=1, a2=1 << 27) == UNSUPPORTED and call(a5=1 << 20, a2=1 << 11) == UNSUPPORTED
    assert call(a0=ctypes.byref(_cache(page_size=32))) == UNSUPPORTED
    # (cache, digest, q, table, max_pages, lens, batch, hq, scale, scores, stride, status, stream)
    call = _call(lib.nvfp4kv_page_scores, [cs, 16, 16, 4, 8, 4, 0, 8, 0.1, 4, 8, None, None])
    assert call() == OK
    assert call(a7=7) == INVALID and call(a7=0) == INVALID and call(a7=18) == UNSUPPORTED and call(a10=0) == INVALID
    assert call(a8=0.0) == INVALID and call(a8=float("inf")) == INVALID
    assert call(a6=1, a2=None) == INVALID and call(a6=1, a9=None) == INVALID and call(a6=1, a2=8) == INVALID
    assert call(a6=1, a9=2) == INVALID and call(a6=1, a10=(1 << 40) + 1) == UNSUPPORTED and call(a6=1, a1=None) == INVALID


def test_selection_refusals(lib):
    # (scores, stride, lens, batch, hkv, budget, first, recent, selected, status, stream)
    call = _call(lib.nvfp4kv_select_pages, [4, 8, 4, 0, 2, 8, 1, 2, 4, None, None])
    assert call() == OK
    for bad in (dict(a1=0), dict(a3=-1), dict(a4=0), dict(a5=0), dict(a6=-1), dict(a7=-1), dict(a6=7), dict(a9=2),
                dict(a6=2 ** 31 - 1, a7=2 ** 31 - 1)):
        assert call(**bad) == INVALID, bad
    assert call(a5=(1 << 27) + 1) == UNSUPPORTED and call(a3=1 << 27) == UNSUPPORTED and call(a1=1 << 41) == UNSUPPORTED
    for missing in (0, 2, 8):
        assert call(**{"a3": 1, f"a{missing}": None}) == INVALID and call(**{"a3": 1, f"a{missing}": 6}) == INVALID
    cs = ctypes.byref(_cache())
    # (cache, q, out, lse, table, max_pages, lens, batch, hq, scale, selected, budget, ws, ws_bytes, status, stream)
    call = _call(lib.nvfp4kv_decode_attention_selected, [cs, 16, 16, 4, 4, 1, 4, 0, 8, 0.1, 4, 8, 256, 1 << 20, None, None])
    assert call() == OK
    assert call(a11=0) == INVALID and call(a11=-3) == INVALID and call(a10=2) == INVALID and call(a3=6) == INVALID
    assert call(a8=18) == UNSUPPORTED and call(a9=float("nan")) == INVALID and call(a7=1, a1=None) == INVALID


class OnGpu:
    """What the bindings' checks look at of a tensor, on GPU `gpu` (-1: on the CPU)."""

    def __init__(self, dtype, shape, gpu=0, strides=None):
        self.dtype, self.shape, self.gpu = dtype, torch.Size(shape), gpu
        self.device, self.is_cuda = f"cuda:{gpu}" if gpu >= 0 else "cpu", gpu >= 0
        self.strides = strides or torch.empty(shape, device="meta").stride()

    def dim(self):
        return len(self.shape)

    def stride(self):
        return self.strides

    def is_contiguous(self):
        return True

    def get_device(self):
        return self.gpu

    def data_ptr(self):
        return 0  # none: the library refuses it


def _calls(cache, **kw):
    """Every binding of this kind as (function, tensors, the rest)."""
    i32, i64, bf16, f32, u8 = torch.int32, torch.int64, torch.bfloat16, torch.float32, torch.uint8
    table, lens, q, sel = (i32, (1, 4)), (i32, (1,)), (bf16, (1, 8, 128)), (i32, (1, 2, 3))
    kvs, digest, scores = (bf16, (1, 2, 128)), (u8, (4, 2, 272)), (f32, (1, 2, 4))
    return [
        (lambda *t: kv.nvfp4kv_plan_append(*t[:5], 4, *t[5:8], positions=t[8], cu_q=t[9], ws_rows=t[10], cu_prefix=t[11], **kw),
         [table, lens, lens, (i32, (9,)), lens, lens, (i64, (3,)), lens, (i32, (3,)), (i64, (2,)), (i64, (3,)), (i64, (2,))]),
        (lambda *t: kv.nvfp4kv_norm_rope_append(cache, *t[:7], q_weight=t[7], k_weight=t[8], ws_rows=t[9], ws_k=t[10],
                                                ws_v=t[11], **kw),
         [q, kvs, kvs, (i64, (1,)), lens, (f32, (50, 64)), q, (bf16, (128,)), (bf16, (128,)), (i64, (1,)),
          (u8, (6, 2, 128)), (u8, (6, 2, 128))]),
        (lambda *t: kv.nvfp4kv_page_digest(cache, *t[:3], first_tokens=t[3], **kw), [table, lens, digest, lens]),
        (lambda *t: kv.nvfp4kv_page_scores(cache, *t[:4], 0.1, t[4], **kw), [digest, q, table, lens, scores]),
        (lambda *t: kv.nvfp4kv_select_pages(*t[:2], 3, 1, 1, t[2], **kw), [scores, lens, sel]),
        (lambda *t: kv.nvfp4kv_decode_attention_selected(cache, *t[:4], 0.1, t[4], None, workspace_bytes=0, **kw),
         [q, q, table, lens, sel]),
    ]


def test_bindings_refuse_wrong_tensors(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    c = kv.Cache(0x10000, 4, 2)
    for n, (fn, tensors) in enumerate(_calls(c)):
        for k, (dtype, shape) in enumerate(tensors):
            good = [OnGpu(*a) for a in tensors]
            # another GPU (all the others are then on another one than the first, or it is), the CPU, another type, a size more
            for other in (OnGpu(dtype, shape, 1), OnGpu(torch.float64, shape), OnGpu(dtype, (*shape, 1))):
                with pytest.raises(ValueError):
                    fn(*good[:k], other, *good[k + 1:])
                    pytest.fail(f"call {n}, tensor {k}")
    for fn, tensors in _calls(c, device_status=OnGpu(torch.int32, (1,), 1)):
        with pytest.raises(ValueError, match="device_status: "):
            fn(*(OnGpu(*a) for a in tensors))
    mx = kv.Cache(0x10000, 4, 2, mxfp4=True)
    for fn, tensors in [_calls(mx)[k] for k in (1, 2, 3, 5)]:
        with pytest.raises(ValueError, match="MXFP4"):
            fn(*(OnGpu(*a) for a in tensors))
    # rows of a token that do not follow one another
    fn, tensors = _calls(c)[1]
    good = [OnGpu(*a) for a in tensors]
    for k in (0, 1, 2, 6):
        dtype, shape = tensors[k]
        for strides in ((4096, 256, 1), (4096, 128, 2)):
            with pytest.raises(ValueError, match="contiguous rows"):
                fn(*good[:k], OnGpu(dtype, shape, 0, strides), *good[k + 1:])


# --- the references -------------------------------------------------------

def test_reference_rows_agree_with_64_bits():
    rng = np.random.default_rng(5)
    x = su.bf16_round(rng.standard_normal((40, 3, 128)) * 2.0 ** rng.integers(-6, 7, (40, 3, 1)))
    w = su.bf16_round(1 + 0.3 * rng.standard_normal(128))
    pos = rng.integers(0, 1000, 40)
    for rot, inter, weight in ((128, False, w), (128, True, w), (64, False, w), (96, True, None), (32, False, None), (0, False, w)):
        angle = np.arange(1000)[:, None] * 10000.0 ** (-np.arange(rot // 2) / max(1, rot // 2))
        cs = np.concatenate([np.cos(angle), np.sin(angle)], -1).astype(np.float32)
        got = su.bf16_round(su.norm_rope_steps(x, weight, 1e-6, cs, pos, inter)).astype(np.float64)
        want, tol = su.norm_rope_exact(x, weight, 1e-6, cs, pos, inter)
        assert (np.abs(got - want) <= tol).all()
        # a rotation keeps lengths, and each pair's
        if weight is None:
            np.testing.assert_allclose(np.linalg.norm(want, axis=-1), np.linalg.norm(x.astype(np.float64), axis=-1), rtol=1e-6)


def test_reference_digest_bounds_and_is_tight():
    rng = np.random.default_rng(6)
    for n in (1, 2, 16):
        K = rng.standard_normal((n, 128)) * 2.0 ** rng.integers(-6, 7, 128)
        K = np.round(K * 64) / 64
        hi, lo, scale = su.digest_ref(K)
        assert (hi * scale >= K.max(0)).all() and (lo * scale <= K.min(0)).all()
        # off by less than one step: an eighth of the value, or the smallest step
        for got, want in ((hi * scale, K.max(0)), (lo * scale, K.min(0))):
            assert (np.abs(got - want) <= np.maximum(np.abs(want) / 8, 2.0 ** -9 * scale)).all()
        q = rng.standard_normal((5, 128))
        top, tol = su.score_ref(q, hi, lo, scale, 0.3)
        assert top + tol >= 0.3 * (q @ K.T).max()
    assert su.digest_ref(np.zeros((3, 128)))[2] == 1.0
    assert oracle.e4m3_value(0x7E) == su.E4M3[-1] == 448.0


def test_reference_plan_hands_out_every_page_once():
    rng = np.random.default_rng(7)
    cached, new = rng.integers(0, 100, 12), rng.integers(0, 60, 12)
    table = np.full((12, 12), -1, np.int32)
    at = 0
    for b, c in enumerate(cached):
        n = -(-c // 16)
        table[b, :n] = range(at, at + n)
        at += n
    free = (np.arange(60) + at).astype(np.int32)
    r = su.plan_ref(table, cached, new, free, 60, at + 60, 800)
    assert r["flags"] == 0 and r["lens"] == (cached + new).tolist() and r["cu_q"][-1] == new.sum()
    used = [p for b in range(12) for p in r["table"][b, :-(-(cached[b] + new[b]) // 16)]]
    assert len(set(used)) == len(used) and r["free_left"][0] == 60 - (len(used) - at)
    slots = [s for s in r["slots"] if s >= 0]
    assert len(set(slots)) == len(slots) == new.sum()
