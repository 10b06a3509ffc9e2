"""Refusals of sizes whose products pass 64 bits (no GPU: the checks return
before anything touches CUDA)."""
import ctypes

import pytest

import nvfp4_quantized_paged_quantize_gb300 as kv

UNSUPPORTED = kv.NVFP4KV_ERR_UNSUPPORTED


@pytest.mark.parametrize("num_pages", [1 << 27, 1 << 40, 1 << 59, 1 << 60, 3 << 60, (1 << 63) - 1])
def test_plan_of_too_many_pages(num_pages):
    # without a free count: refused at the latest
    assert kv.load().nvfp4kv_plan_append(64, 8, 128, 256, 2, 512, 16, None, num_pages, 64, 1024, 2048, 4096, 8, 8, 8, 4, None,
                                         None) == UNSUPPORTED


@pytest.mark.parametrize("which", [2, 4, 6, 15])
@pytest.mark.parametrize("tokens,stride", [(1 << 24, 1 << 40), (1 << 23, 1 << 40), ((1 << 26) + 8, 1 << 38), ((1 << 28) - 1, 1 << 36)])
def test_rows_too_far_apart(which, tokens, stride):
    # without queries: refused at the latest
    cache = kv.Cache(0x10000, 4, 2).c_struct()
    how = kv._CNormRope(16, 16, 1e-6, 128, 0)
    args = [ctypes.byref(cache), None, 512, 16, 512, 16, 512, 4, tokens, 8, 4, 16, 100, ctypes.byref(how), 1 << 20, 512, None, 0, 1.0,
            1.0, None, None, None, None]
    assert kv.load().nvfp4kv_norm_rope_append(*args) == kv.NVFP4KV_ERR_INVALID_ARGUMENT
    args[which] = stride
    assert kv.load().nvfp4kv_norm_rope_append(*args) == UNSUPPORTED
