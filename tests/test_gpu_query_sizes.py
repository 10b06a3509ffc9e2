"""Queries of every finite size: the page scores and the decodes against their
references, with tolerances as step_util and scored_util derive them."""
import numpy as np
import pytest
import torch

import oracle
import nvfp4_quantized_paged_quantize_gb300 as kv
from gpu_util import dev, pool_host, status_word
from scored_util import SCALE, check, page_tables, random_cache, random_q, sequence_rows
from step_util import e4m3_values, score_ref
from test_gpu_page_selection import attend_ref, guarded_digest, random_lists, run_attend

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


# keys' scales that bring the scores back to ordinary size, where the softmax tells them apart
@pytest.mark.parametrize("size,gk", [(2.0 ** 113, 2.0 ** -113), (2.0 ** 118, 2.0 ** -118), (2.0 ** 124, 2.0 ** -123), (2.0 ** -80, 2.0 ** 80),
                                     (2.0 ** -100, 2.0 ** 100), (2.0 ** -118, 2.0 ** 118)])
def test_decodes(cuda_lib, size, gk):
    lens, hkv, group = [700, 40, 16], 2, 5
    table, used = page_tables(lens, 53)
    cache, o = random_cache(used, hkv, 54, gk=gk, gv=0.25)
    run_attend(cache, o, table, lens, hkv * group, random_lists(lens, hkv, 9, 55), 56, size=size)
    q, q64 = random_q((len(lens), hkv * group, 128), 56, size)
    pt, sl = dev(table), dev(np.asarray(lens, np.int32))
    ws = torch.zeros(kv.nvfp4kv_decode_workspace_size(cache, len(lens), hkv * group), dtype=torch.uint8, device="cuda")
    out, scored = torch.empty(q.shape, device="cuda"), torch.empty_like(q)
    lse = torch.empty(q.shape[:2], device="cuda")
    kv.nvfp4kv_decode_attention(cache, q, out, pt, sl, SCALE, ws)
    kv.nvfp4kv_decode_attention_scored(cache, q, scored, pt, sl, SCALE, ws, lse=lse)
    got = [x.double().cpu().numpy() for x in (out, scored, lse)]
    for b, n in enumerate(lens):
        for i in range(hkv * group):
            r = attend_ref(o, table[b], i // group, n, range(-(-n // 16)), q64[b, i])
            for x in got[:2]:
                check(x[b, i], r["out"], r["tol_out"], f"{b} {i}")
            check(got[2][b, i], r["lse"], r["tol_lse"], f"lse {b} {i}")


def test_keys_of_zeros(cuda_lib):
    # a multiplier past fp32's largest number meets scores of zero: equal weights
    table, used = page_tables([100], 57)
    cache, o = random_cache(used, 1, 58, gk=2.0 ** 20)
    cache.k_scale.zero_()
    o = oracle.Cache(used, 1, 128, 16, 2.0 ** 20, 1.0, arrays=pool_host(cache))
    run_attend(cache, o, table, [100], 8, random_lists([100], 1, 4, 59), 60, size=2.0 ** 120)
    q, _ = random_q((1, 8, 128), 60, 2.0 ** 120)
    out = torch.empty(q.shape, device="cuda")
    ws = torch.zeros(kv.nvfp4kv_decode_workspace_size(cache, 1, 8), dtype=torch.uint8, device="cuda")
    kv.nvfp4kv_decode_attention(cache, q, out, dev(table), dev(np.array([100], np.int32)), SCALE, ws)
    r = attend_ref(o, table[0], 0, 100, range(7), np.zeros(128))
    for i in range(8):
        check(out[0, i].double().cpu().numpy(), r["out"], r["tol_out"], f"{i}")
