"""Queries of every finite size: the page scores against their reference, with
tolerances as step_util derives them."""
import numpy as np
import pytest
import torch

import nvfp4_quantized_paged_quantize_gb300 as kv
from gpu_util import dev, status_word
from scored_util import SCALE, page_tables, random_cache, random_q, sequence_rows
from step_util import e4m3_values, score_ref
from test_gpu_page_selection import guarded_digest

pytestmark = pytest.mark.gpu


# near bf16's largest, where the products with the queries' share of the scale would leave fp32 before the pages' units
# bring them back; the smallest normal ones and subnormal ones; scales of the keys that make scores of ordinary size of them
@pytest.mark.parametrize("size,gk,softmax_scale", [(2.0 ** 115, 0.37, SCALE), (2.0 ** 118, 0.37, SCALE), (2.0 ** 124, 2.0 ** -10, SCALE),
                                                   (2.0 ** 124, 2.0 ** -120, SCALE), (2.0 ** 120, 1.0, 2.0 ** -60),
                                                   (2.0 ** -90, 0.37, SCALE), (2.0 ** -110, 2.0 ** 100, SCALE),
                                                   (2.0 ** -124, 2.0 ** 110, SCALE), (2.0 ** -128, 2.0 ** 120, 1.0)])
@pytest.mark.parametrize("small", [False, True])
def test_scores(cuda_lib, size, gk, softmax_scale, small):
    lens, hkv, group = [300, 40, 16], 3, 5
    table, used = page_tables(lens, 50)
    cache, _ = random_cache(used, hkv, 51, gk=gk)
    if small:
        cache.k_scale[::2] = torch.arange(1, 9, dtype=torch.uint8, device="cuda")   # pages of tiny keys, of tiny units
        cache.k_scale[1] = 0                                                        # and of zeros
    pt, sl = dev(table), dev(np.asarray(lens, np.int32))
    d, status = guarded_digest(cache), status_word()
    kv.nvfp4kv_page_digest(cache, pt, sl, d.t)
    q, q64 = random_q((len(lens), hkv * group, 128), 52, size)
    assert np.isfinite(q64).all()
    q[1, 0], q64[1, 0] = 0, 0.0
    q[1, 1, 5:], q64[1, 1, 5:] = 0, 0.0
    scores = torch.full((len(lens), hkv, table.shape[1]), -7.0, device="cuda")
    kv.nvfp4kv_page_scores(cache, d.t, q, pt, sl, softmax_scale, scores, device_status=status)
    assert status.item() == 0
    got, raw = scores.double().cpu().numpy(), d.t.cpu().numpy()
    factor = float(np.float32(softmax_scale) * np.float32(gk))
    for b, n in enumerate(lens):
        for h in range(hkv):
            heads = q64[b, h * group:(h + 1) * group]
            for p in range(-(-n // 16)):
                r = raw[table[b, p], h]
                want, tol = score_ref(heads, e4m3_values(r[:128]), e4m3_values(r[128:256]), r[256:260].view(np.float32)[0], factor)
                assert abs(want) < 2.0 ** 127 and abs(got[b, h, p] - want) <= tol, (b, h, p, got[b, h, p], want)
