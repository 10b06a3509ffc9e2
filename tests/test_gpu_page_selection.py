"""Digests, page scores, selection and the decode over selected pages, each
against its reference, and a whole decode step of them, captured."""
import numpy as np
import pytest
import torch

import oracle
import nvfp4_quantized_paged_quantize_gb300 as kv
from gpu_util import bf16_dev, dev, pool_host, status_word
from nvfp4_quantized_paged_quantize_gb300 import inputs
from scored_util import SCALE, attend, check, evict_ref, page_tables, random_cache, random_q, sequence_rows
from step_util import bf16_round, bits, digest_ref, e4m3_values, norm_rope_steps, same, score_ref
from test_gpu_canary import Guarded
from test_gpu_norm_rope import EPS, PARTS, table_of

pytestmark = pytest.mark.gpu

F32, U8 = torch.float32, torch.uint8


def pages_of(lens):
    return [-(-max(0, n) // 16) for n in lens]


def guarded_digest(cache, fill=0x33):
    d = Guarded((cache.num_pages, cache.num_kv_heads, kv.NVFP4KV_DIGEST_BYTES), U8)
    d.t.fill_(fill)
    return d


def check_digest(d, o, table, lens, first=None):
    """Every page of the sequences from `first` on has its keys' digest, all others the fill byte 0x33."""
    raw = d.t.cpu().numpy()
    touched = np.zeros(raw.shape[0], bool)
    for b, n in enumerate(lens):
        for p in range(max(0, first[b]) // 16 if first is not None else 0, -(-n // 16)):
            page = int(table[b, p])
            touched[page] = True
            for h in range(o.num_kv_heads):
                K, _ = sequence_rows(o, table[b], h, n)
                hi, lo, scale = digest_ref(K[16 * p:16 * p + 16] / o.k_global_scale)
                got = raw[page, h]
                assert np.array_equal(e4m3_values(got[:128]), hi) and np.array_equal(e4m3_values(got[128:256]), lo), (b, p, h)
                assert got[256:260].view(np.float32)[0] == scale and not got[260:].any()
                assert not (got[:256] == 0x80).any()                 # no negative zeros
    assert (raw[~touched] == 0x33).all()
    assert d.intact()


@pytest.mark.parametrize("lens,hkv", [([1], 1), ([16, 17, 0, 5], 2), ([100, 257, 33], 3), ([700, 3], 8)])
def test_digest(cuda_lib, lens, hkv):
    table, used = page_tables(lens, 3, extra_cols=2)
    cache, o = random_cache(used + 2, hkv, 4)
    d, status = guarded_digest(cache), status_word()
    kv.nvfp4kv_page_digest(cache, dev(table), dev(np.asarray(lens, np.int32)), d.t, device_status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    check_digest(d, o, table, lens)


def test_digest_of_many_sequences(cuda_lib):
    # more sequences than a block has threads, many of them empty
    rng = np.random.default_rng(5)
    lens = np.where(rng.random(700) < 0.4, 0, rng.integers(0, 60, 700)).tolist()
    table, used = page_tables(lens, 6)
    cache, o = random_cache(used, 2, 7)
    d = guarded_digest(cache)
    kv.nvfp4kv_page_digest(cache, dev(table), dev(np.asarray(lens, np.int32)), d.t)
    check_digest(d, o, table, lens)


def test_digest_of_the_last_pages(cuda_lib):
    lens, first = [100, 257, 33, 48, 0, 20, 7], [95, 256, 0, 48, 0, -5, 1000]
    table, used = page_tables(lens, 8)
    cache, o = random_cache(used, 2, 9)
    d, status = guarded_digest(cache), status_word()
    kv.nvfp4kv_page_digest(cache, dev(table), dev(np.asarray(lens, np.int32)), d.t, first_tokens=dev(np.asarray(first, np.int32)),
                           device_status=status)
    assert status.item() == 0
    check_digest(d, o, table, lens, first)


def test_digest_of_extreme_keys(cuda_lib):
    # zeros, one sign only, the format's largest and smallest values, scales that underflow to zero
    cache, o = random_cache(6, 1, 10)
    cache.k_scale[0] = 0
    cache.k_data[1] = 0x77                                           # 6.0
    cache.k_data[2] = 0xFF                                           # -6.0
    cache.k_scale[1:3] = 0x7E                                        # 448
    cache.k_data[3] = 0x81                                           # 0.5 and -0
    cache.k_scale[3] = 0x01                                          # 2^-9
    cache.k_data[4] = 0x88                                           # -0 and -0
    cache.k_scale[5] = torch.arange(128, device="cuda").view(1, 16, 8).clamp_max(0x7E).to(U8)   # every scale
    o = oracle.Cache(6, 1, 128, 16, arrays=pool_host(cache))
    table, d = np.arange(6, dtype=np.int32)[None], guarded_digest(cache)
    kv.nvfp4kv_page_digest(cache, dev(table), dev(np.array([96], np.int32)), d.t)
    check_digest(d, o, table, [96])


def test_digest_and_scores_flag_bad_pages_and_lengths(cuda_lib):
    table, used = page_tables([64, 64], 11)
    cache, o = random_cache(used, 2, 12)
    table[0, 1], table[1, 3] = -1, used
    q, q64 = random_q((2, 8, 128), 13)
    for lens, flag in (([64, 64], 0), ([70, -3], kv.NVFP4KV_DEVERR_LENGTH)):
        d, status = guarded_digest(cache, 0x20), status_word()
        kv.nvfp4kv_page_digest(cache, dev(table), dev(np.asarray(lens, np.int32)), d.t, device_status=status)
        assert status.item() == kv.NVFP4KV_DEVERR_PAGE | flag and d.intact()
        status.zero_()
        scores = Guarded((2, 2, 4), F32)
        scores.t.fill_(7.0)
        kv.nvfp4kv_page_scores(cache, d.t, q, dev(table), dev(np.asarray(lens, np.int32)), SCALE, scores.t, device_status=status)
        assert status.item() == kv.NVFP4KV_DEVERR_PAGE | flag and scores.intact()
        got = scores.t.cpu().numpy()
        assert (got[0, :, 1] == -np.inf).all() and np.isfinite(got[0][:, [0, 2, 3]]).all()
        if flag:
            assert (got[1] == 7.0).all()                             # a negative length: none
        else:
            assert (got[1, :, 3] == -np.inf).all()
    # fewer places than pages
    status.zero_()
    scores = Guarded((2, 2, 3), F32)
    kv.nvfp4kv_page_scores(cache, d.t, q, dev(table), dev(np.array([64, 48], np.int32)), SCALE, scores.t, device_status=status)
    assert status.item() == kv.NVFP4KV_DEVERR_PAGE | kv.NVFP4KV_DEVERR_LENGTH and scores.intact()


@pytest.mark.parametrize("lens,hkv,group,size", [([1], 1, 1, 1.0), ([16, 300, 0, 5], 2, 4, 1.0), ([257, 256, 255], 3, 8, 30.0),
                                                 ([1000, 33], 2, 5, 2.0 ** -70), ([500], 8, 7, 2.0 ** 60), ([300, 40], 5, 2, 1.0),
                                                 ([90, 530], 12, 1, 1.0), ([2100], 1, 3, 1.0), ([700, 50], 4, 2, 1.0)])
def test_scores(cuda_lib, lens, hkv, group, size):
    table, used = page_tables(lens, 14, extra_cols=1)
    cache, o = random_cache(used, hkv, 15, gk=0.37)
    pt, sl = dev(table), dev(np.asarray(lens, np.int32))
    d, status = guarded_digest(cache), status_word()
    kv.nvfp4kv_page_digest(cache, pt, sl, d.t)
    q, q64 = random_q((len(lens), hkv * group, 128), 16, size)
    q[0, 0] = 0
    q64[0, 0] = 0.0
    stride = table.shape[1] + 3
    scores = Guarded((len(lens), hkv, stride), F32)
    scores.t.fill_(-7.0)
    kv.nvfp4kv_page_scores(cache, d.t, q, pt, sl, SCALE, scores.t, device_status=status)
    assert status.item() == 0 and scores.intact()
    got, raw = scores.t.double().cpu().numpy(), d.t.cpu().numpy()
    factor = SCALE * o.k_global_scale
    for b, n in enumerate(lens):
        pages = -(-n // 16)
        assert (got[b, :, pages:] == -7.0).all()
        for h in range(hkv):
            K, _ = sequence_rows(o, table[b], h, n)
            heads = q64[b, h * group:(h + 1) * group]
            for p in range(pages):
                r = raw[table[b, p], h]
                want, tol = score_ref(heads, e4m3_values(r[:128]), e4m3_values(r[128:256]), r[256:260].view(np.float32)[0], factor)
                assert abs(got[b, h, p] - want) <= tol, (b, h, p)
                # no token of the page scores more
                assert got[b, h, p] + tol >= (heads @ K[16 * p:16 * p + 16].T * SCALE).max()


def test_scores_of_many_sequences(cuda_lib):
    rng = np.random.default_rng(17)
    lens = np.where(rng.random(300) < 0.3, 0, rng.integers(0, 90, 300)).tolist()
    table, used = page_tables(lens, 18)
    cache, o = random_cache(used, 2, 19)
    pt, sl = dev(table), dev(np.asarray(lens, np.int32))
    d = guarded_digest(cache)
    kv.nvfp4kv_page_digest(cache, pt, sl, d.t)
    q, q64 = random_q((300, 4, 128), 20)
    scores = torch.zeros((300, 2, table.shape[1]), device="cuda")
    kv.nvfp4kv_page_scores(cache, d.t, q, pt, sl, SCALE, scores)
    got, raw = scores.double().cpu().numpy(), d.t.cpu().numpy()
    for b, n in enumerate(lens):
        for h in range(2):
            for p in range(-(-n // 16)):
                r = raw[table[b, p], h]
                want, tol = score_ref(q64[b, 2 * h:2 * h + 2], e4m3_values(r[:128]), e4m3_values(r[128:256]),
                                      r[256:260].view(np.float32)[0], SCALE)
                assert abs(got[b, h, p] - want) <= tol


# --- selection ------------------------------------------------------------

def select(w, lens, budget, first, recent, stride=None):
    B, hkv, n = w.shape
    out, status = Guarded((B, hkv, budget), torch.int32), status_word()
    kv.nvfp4kv_select_pages(dev(w), dev(np.asarray(lens, np.int32)), budget, first, recent, out.t, device_status=status)
    torch.cuda.synchronize()
    assert out.intact()
    return out.t.cpu().numpy(), status.item()


def check_selection(w, lens, budget, first, recent):
    got, status = select(w, lens, budget, first, recent)
    assert status == 0
    for b, n in enumerate(pages_of(lens)):
        for h in range(w.shape[1]):
            want = evict_ref(w[b, h, :n], n, budget, first, recent)
            same(got[b, h, :len(want)].astype(int), want, f"{b} {h}")
            assert (got[b, h, len(want):] == -1).all()


@pytest.mark.parametrize("budget,first,recent", [(4, 0, 0), (4, 1, 1), (4, 4, 0), (4, 0, 4), (1, 0, 0), (33, 2, 7), (63, 1, 16), (200, 1, 4)])
def test_selection(cuda_lib, budget, first, recent):
    lens = [0, 1, 16, 17, budget * 16 - 1, budget * 16, budget * 16 + 1, budget * 16 + 17, 1000, 3210, 4096]
    rng = np.random.default_rng(budget)
    check_selection(rng.standard_normal((len(lens), 3, 256)).astype(np.float32), lens, budget, first, recent)


def test_selection_ties_and_special_values(cuda_lib):
    n = 700
    at = np.arange(n)
    rows = [np.zeros(n), np.full(n, -1.0), np.tile([1.0, 2.0], n // 2), np.where(at % 7 == 0, np.inf, 1.0),
            np.where(at % 5 == 0, np.nan, at), np.where(at % 2 == 0, 0.0, -0.0), np.linspace(-3, 3, n), np.full(n, 2.0 ** -149),
            -np.full(n, np.inf), np.where(at % 3 == 0, -np.inf, at), 1.0 + at * 2.0 ** -23, np.where(at < 350, 1e30, -1e30),
            2.0 ** (at % 250 - 125.0), -(1.0 + (at // 100) * 2.0 ** -20)]
    w = np.stack(rows).astype(np.float32)[:, None]
    w[4, 0, 3] = np.array([0xFFC00001], np.uint32).view(np.float32)[0]         # a negative NaN
    for budget in (1, 5, 100, 333, 650, 699):
        check_selection(w, [16 * n - 3] * len(rows), budget, min(3, budget), min(40, budget - min(3, budget)))


@pytest.mark.parametrize("pages", [1023, 2048, 4097, 8192, 8193, 20000, 70000])
def test_selection_of_long_sequences(cuda_lib, pages):
    rng = np.random.default_rng(pages)
    w = (rng.standard_normal((2, 2, pages)) * 1.5 + 4).astype(np.float32)
    w[1] = np.round(w[1] * 4) / 4                                              # many ties
    for budget in (pages // 8, pages // 2 + 1, 17):
        check_selection(w, [16 * pages, 16 * (pages // 2) + 5], budget, 1, 4)


@pytest.mark.parametrize("pages", [16385, 40000])
def test_selection_of_long_sequences_with_special_values(cuda_lib, pages):
    at = np.arange(pages)
    rng = np.random.default_rng(5)
    rows = [np.zeros(pages), np.where(at % 7 == 0, np.inf, 1.0), np.where(at % 5 == 0, np.nan, at), np.linspace(-3, 3, pages),
            np.where(at % 3 == 0, -np.inf, at), 1.0 + (at % 1000) * 2.0 ** -23, np.where(at < 350, 1e30, -1e30),
            rng.standard_normal(pages), np.where(at == pages - 9, 1e9, rng.random(pages))]
    w = np.stack(rows).astype(np.float32)[:, None]
    for budget in (1, 40, pages // 3, pages - 1):
        check_selection(w, [16 * pages - 3] * len(rows), budget, min(3, budget), min(40, budget - min(3, budget)))
    # lengths of which some parts, or all, have nothing to choose from
    check_selection(w, [0, 1, 16 * 60, 16 * 61, 16 * 100, 16 * 5000, 16 * pages, 16 * 33, 16 * 9000], 60, 7, 21)
    check_selection(np.repeat(w, 5, 1), [16 * pages - 3] * len(rows), 77, 2, 2)


def test_selection_of_many_pairs_and_cut_lengths(cuda_lib):
    rng = np.random.default_rng(21)
    lens = rng.integers(0, 2000, 200)
    check_selection(rng.standard_normal((200, 8, 125)).astype(np.float32), lens, 20, 1, 3)
    # longer than the scores have room for, and negative: cut and flagged
    w = rng.standard_normal((2, 1, 125)).astype(np.float32)
    got, status = select(w, [2001, -1], 20, 1, 3)
    assert status == kv.NVFP4KV_DEVERR_LENGTH
    assert np.array_equal(got[0, 0], evict_ref(w[0, 0], 125, 20, 1, 3)) and (got[1] == -1).all()


# --- the decode over selected pages ---------------------------------------

def attend_ref(o, table_row, h, n, pages, q, softmax_scale=SCALE):
    """One query head over the tokens of the listed pages."""
    K, V = sequence_rows(o, table_row, h, n)
    t = np.concatenate([np.arange(16 * p, min(16 * p + 16, n)) for p in pages]) if len(pages) else np.zeros(0, int)
    return attend(q, K[t], V[t], np.ones(len(t), bool), np.zeros(len(t)), softmax_scale)


def run_attend(cache, o, table, lens, hq, sel, seed, size=1.0, flags=0, skip=()):
    B, hkv, budget = sel.shape
    q, q64 = random_q((B, hq, 128), seed, size)
    out, lse = Guarded((B, hq, 128), torch.bfloat16), Guarded((B, hq), F32)
    ws = Guarded((kv.nvfp4kv_decode_workspace_size(cache, B, hq),), U8)
    ws.t.fill_(0xFF)                                                           # NaN, were any of it read unwritten
    status = status_word()
    kv.nvfp4kv_decode_attention_selected(cache, q, out.t, dev(table), dev(np.asarray(lens, np.int32)), SCALE, dev(sel), ws.t,
                                         lse=lse.t, device_status=status)
    torch.cuda.synchronize()
    assert status.item() == flags
    for g in (out, lse, ws):
        assert g.intact()
    got, gl = out.t.double().cpu().numpy(), lse.t.double().cpu().numpy()
    G = hq // hkv
    table = np.where((table >= 0) & (table < cache.num_pages), table, 0)       # a bad id's page is in `skip`
    for b, n in enumerate(lens):
        for i in range(hq):
            pages = [p for p in sel[b, i // G, :min(budget, -(-n // 16))] if 0 <= p < -(-n // 16) and (b, p) not in skip]
            r = attend_ref(o, table[b], i // G, n, pages, q64[b, i])
            if not pages:
                assert not got[b, i].any() and gl[b, i] == -np.inf
                continue
            check(got[b, i], r["out"], r["tol_out"], f"{b} {i}")
            check(gl[b, i], r["lse"], r["tol_lse"], f"lse {b} {i}")
    return out.t, lse.t


def random_lists(lens, hkv, budget, seed, last=True):
    """Ascending lists of distinct pages, -1 behind them; `last`: the last page among them."""
    rng = np.random.default_rng(seed)
    sel = np.full((len(lens), hkv, budget), -1, np.int32)
    for b, n in enumerate(pages_of(lens)):
        for h in range(hkv):
            m = min(n, budget)
            pick = np.sort(rng.permutation(n)[:m])
            if last and m:
                pick = np.unique(np.append(pick[1:], n - 1)) if n - 1 not in pick else pick
            sel[b, h, :len(pick)] = pick
    return sel


@pytest.mark.parametrize("lens,hkv,group,budget", [([1], 1, 1, 1), ([17, 300, 0, 5], 2, 4, 3), ([1000, 33, 257], 2, 8, 20),
                                                   ([700], 3, 5, 1), ([512, 100], 1, 7, 200), ([5000, 40], 2, 8, 64),
                                                   ([8000, 100], 1, 8, 480)])
def test_selected_decode(cuda_lib, lens, hkv, group, budget):
    table, used = page_tables(lens, 22, extra_cols=1)
    cache, o = random_cache(used, hkv, 23, gk=0.5, gv=0.25)
    run_attend(cache, o, table, lens, hkv * group, random_lists(lens, hkv, budget, 24), 25)


@pytest.mark.parametrize("batch", [20, 70, 150, 200])
def test_selected_decode_of_a_large_batch(cuda_lib, batch):
    # one wave of CTAs (several to a pair, one to a pair), and more pairs than that
    rng = np.random.default_rng(26)
    lens = np.where(rng.random(batch) < 0.2, 0, rng.integers(0, 700, batch)).tolist()
    table, used = page_tables(lens, 27)
    cache, o = random_cache(used, 2, 28)
    run_attend(cache, o, table, lens, 8, random_lists(lens, 2, 9, 29), 30)


@pytest.mark.parametrize("pairs,group", [(12, 7), (41, 5), (47, 8), (55, 3), (70, 7), (90, 8), (120, 6), (200, 8)])
def test_selected_decode_at_every_number_of_parts(cuda_lib, pairs, group):
    # 8, 7, .. 1 CTAs to a pair on this GPU: heads that do not divide among them, lists shorter than the warps
    rng = np.random.default_rng(pairs)
    lens = rng.integers(0, 900, pairs).tolist()
    table, used = page_tables(lens, pairs + 1)
    cache, o = random_cache(used, 1, pairs + 2)
    run_attend(cache, o, table, lens, group, random_lists(lens, 1, 23, pairs + 3), pairs + 4)


def test_lists_in_any_order_with_gaps(cuda_lib):
    lens = [400, 90, 50, 33]
    table, used = page_tables(lens, 31)
    cache, o = random_cache(used, 2, 32)
    sel = np.full((4, 2, 6), -1, np.int32)
    sel[0, 0] = [24, -1, 3, -5, 0, 24 - 1]                                     # the partial last page first
    sel[0, 1] = [-1, -1, -1, -1, -1, 7]
    sel[1, 0] = [-1] * 6                                                       # no page at all
    sel[1, 1] = [5, 4, 3, 2, 1, 0]
    sel[2, 0, :4] = [3, -1, -1, 0]                                             # two tokens of the last page, and a whole one
    sel[2, 1, 4] = 1                                                           # behind what is looked at: four pages
    sel[3, :, 0] = 2                                                           # one token alone
    run_attend(cache, o, table, lens, 8, sel, 33)


def test_every_page_listed_is_the_plain_decode(cuda_lib):
    lens = [333, 1500, 16]
    table, used = page_tables(lens, 34)
    cache, o = random_cache(used, 2, 35)
    n = max(pages_of(lens))
    sel = np.full((3, 2, n), -1, np.int32)
    for b, m in enumerate(pages_of(lens)):
        sel[b, :, :m] = np.arange(m)
    out, lse = run_attend(cache, o, table, lens, 16, sel, 36)
    q, _ = random_q((3, 16, 128), 36)
    ws = torch.empty(kv.nvfp4kv_decode_workspace_size(cache, 3, 16), dtype=U8, device="cuda")
    o2, l2 = torch.empty_like(out), torch.empty_like(lse)
    kv.nvfp4kv_decode_attention_scored(cache, q, o2, dev(table), dev(np.asarray(lens, np.int32)), SCALE, ws, lse=l2)
    q64 = random_q((3, 16, 128), 36)[1]
    for b, m in enumerate(lens):
        for i in range(16):                                                    # both within the same bounds of the same values
            r = attend_ref(o, table[b], i // 8, m, range(pages_of(lens)[b]), q64[b, i])
            check(o2[b, i].double().cpu().numpy(), r["out"], r["tol_out"], f"{b} {i}")
            check(l2[b, i].double().cpu().numpy(), r["lse"], r["tol_lse"], f"lse {b} {i}")


def test_selected_decode_flags_bad_entries(cuda_lib):
    lens = [200, 100]
    table, used = page_tables(lens, 37)
    cache, o = random_cache(used, 2, 38)
    sel = random_lists(lens, 2, 4, 39)
    sel[0, 0, 1], sel[1, 1, 0] = 13, 2 ** 31 - 1                               # past the sequences' 13 and 7 pages
    run_attend(cache, o, table, lens, 8, sel, 40, flags=kv.NVFP4KV_DEVERR_PAGE)
    table[0, sel[0, 1, 0]] = used                                              # a listed page outside the pool
    sel = random_lists(lens, 2, 4, 39)
    run_attend(cache, o, table, lens, 8, sel, 40, flags=kv.NVFP4KV_DEVERR_PAGE, skip={(0, int(sel[0, 1, 0]))})


def test_pages_at_the_end_of_a_large_pool(cuda_lib):
    # byte offsets past 2^32 in the pool and past 2^29 in the digests: the same results as from a small pool
    lens, hkv = [200, 37], 8
    table, used = page_tables(lens, 60)
    small, _ = random_cache(used, hkv, 61)
    many = 280000
    big = kv.Cache.empty(many, hkv)
    big.pages[many - used:] = small.pages
    sl, sel = dev(np.asarray(lens, np.int32)), dev(random_lists(lens, hkv, 5, 62))
    q, _ = random_q((2, 16, 128), 63)
    got = []
    for cache, shift in ((small, 0), (big, many - used)):
        pt = dev(np.where(table >= 0, table + shift, table).astype(np.int32))
        status = status_word()
        d = torch.zeros((cache.num_pages, hkv, kv.NVFP4KV_DIGEST_BYTES), dtype=U8, device="cuda")
        kv.nvfp4kv_page_digest(cache, pt, sl, d, device_status=status)
        scores = torch.zeros((2, hkv, table.shape[1]), device="cuda")
        kv.nvfp4kv_page_scores(cache, d, q, pt, sl, SCALE, scores, device_status=status)
        out, lse = torch.empty_like(q), torch.empty((2, 16), device="cuda")
        ws = torch.empty(kv.nvfp4kv_decode_workspace_size(cache, 2, 16), dtype=U8, device="cuda")
        kv.nvfp4kv_decode_attention_selected(cache, q, out, pt, sl, SCALE, sel, ws, lse=lse, device_status=status)
        torch.cuda.synchronize()
        assert status.item() == 0
        got.append((d[cache.num_pages - used:], scores, out, lse))
    for name, a, b in zip(("digests", "scores", "out", "lse"), *got):
        assert torch.equal(a, b), name


def test_two_streams_at_once(cuda_lib):
    # the calls keep no state: two batches in flight on two streams give what each gives alone
    made = []
    for k in range(2):
        lens = [1500 + 700 * k, 333]
        table, used = page_tables(lens, 64 + k)
        cache, _ = random_cache(used, 2, 66 + k)
        sl, pt = dev(np.asarray(lens, np.int32)), dev(table)
        q, _ = random_q((2, 8, 128), 68 + k)
        d = torch.zeros((used, 2, kv.NVFP4KV_DIGEST_BYTES), dtype=U8, device="cuda")
        ws = torch.empty(kv.nvfp4kv_decode_workspace_size(cache, 2, 8), dtype=U8, device="cuda")
        made.append((cache, pt, sl, q, d, ws, table.shape[1]))

    def run(m, stream=None):
        cache, pt, sl, q, d, ws, pages = m
        scores, sel = torch.zeros((2, 2, pages), device="cuda"), torch.empty((2, 2, 20), dtype=torch.int32, device="cuda")
        out = torch.empty_like(q)
        if stream:
            stream.wait_stream(torch.cuda.current_stream())
        for _ in range(20):
            kv.nvfp4kv_page_digest(cache, pt, sl, d, stream=stream)
            kv.nvfp4kv_page_scores(cache, d, q, pt, sl, SCALE, scores, stream=stream)
            kv.nvfp4kv_select_pages(scores, sl, 20, 1, 2, sel, stream=stream)
            kv.nvfp4kv_decode_attention_selected(cache, q, out, pt, sl, SCALE, sel, ws, stream=stream)
        return scores, sel, out

    alone = [run(m) for m in made]
    torch.cuda.synchronize()
    together = [run(m, torch.cuda.Stream()) for m in made]
    torch.cuda.synchronize()
    for a, b in zip(alone, together):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("ahead", ["kernel", "copy", "clear", "other stream", "own kernel on another stream"])
def test_calls_wait_for_what_is_ahead(cuda_lib, ahead, captured):
    # a call's blocks may be placed before the work ahead of it ends; what that writes is seen all the same
    rng = np.random.default_rng(77)
    n, lens = 500, dev(np.asarray([8000, 7777], np.int32))
    news = [rng.standard_normal((2, 4, n)).astype(np.float32) for _ in range(3)]
    scores, src = torch.zeros((2, 4, n), device="cuda"), torch.empty((2, 4, n), device="cuda")
    sel, again = (torch.empty((2, 4, 60), dtype=torch.int32, device="cuda") for _ in range(2))
    busy = torch.rand((3000, 3000), device="cuda")
    side = torch.cuda.Stream()

    def step():
        for _ in range(4):
            busy.mul_(1.0).add_(0.0)                                           # some time for the work ahead
        if ahead == "kernel":
            torch.mul(src, 1.0, out=scores)
        elif ahead == "copy":
            scores.copy_(src)
        elif ahead == "clear":
            torch.mul(src, 1.0, out=scores)
            scores.zero_()
        else:
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                busy.mul_(1.0)
                torch.mul(src, 1.0, out=scores)
                if ahead.startswith("own"):
                    kv.nvfp4kv_select_pages(scores, lens, 60, 1, 2, again)
            kv.nvfp4kv_select_pages(src, lens, 60, 1, 2, sel)                  # something on this stream, too
            torch.cuda.current_stream().wait_stream(side)
        kv.nvfp4kv_select_pages(scores, lens, 60, 1, 2, sel)
        scores.fill_(-1.0)                                                     # not before the selection has read them
        kv.nvfp4kv_select_pages(scores, lens, 60, 1, 2, again)

    if captured:
        graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        src.copy_(dev(news[0]))
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            step()
    flat = np.concatenate([[0], np.arange(1, 58), [0, 0]])
    for new in news:
        src.copy_(dev(new))
        graph.replay() if captured else step()
        torch.cuda.synchronize()
        for b, pages in enumerate((500, 487)):
            for h in range(4):
                w = np.zeros(pages) if ahead == "clear" else new[b, h, :pages]
                same(sel[b, h].cpu().numpy().astype(int), evict_ref(w, pages, 60, 1, 2), f"{b} {h}")
                flat[-2:] = pages - 2, pages - 1
                same(again[b, h].cpu().numpy().astype(int), flat, f"again {b} {h}")


# --- a whole step ----------------------------------------------------------

def test_captured_decode_steps_over_selected_pages(cuda_lib):
    """As a server would use them: a step's plan, the normed and rotated append of its tokens, the digests of the pages
    they went into, the page scores, the selection and the decode over it; captured once, replayed for several steps
    that cross page borders, and checked against the references after each."""
    rng = np.random.default_rng(41)
    lens, hq, hkv, budget, first, recent = [395, 30, 158, 0, 16], 8, 2, 6, 1, 2
    B, steps, group, cols = len(lens), 5, hq // hkv, 30
    num_pages = sum(pages_of(lens)) + 12
    ids = rng.permutation(num_pages).astype(np.int32)
    table = np.full((B, cols), -1, np.int32)
    at = 0
    for b, n in enumerate(pages_of(lens)):
        table[b, :n] = ids[at:at + n]
        at += n
    cache, o = random_cache(num_pages, hkv, 42, gk=0.02, gv=0.03)
    pt, sl, new = dev(table), dev(np.asarray(lens, np.int32)), dev(np.ones(B, np.int32))
    stack, count = dev(ids[at:]), dev(np.array([num_pages - at], np.int32))
    digest = torch.zeros((num_pages, hkv, kv.NVFP4KV_DIGEST_BYTES), dtype=U8, device="cuda")
    kv.nvfp4kv_page_digest(cache, pt, sl, digest)
    cs = table_of(600, 128)
    weights = [bf16_round(1 + 0.3 * rng.standard_normal(128)) for _ in range(2)]
    dcs, dw = dev(cs), [torch.from_numpy(w).to(torch.bfloat16).cuda() for w in weights]
    qkv = torch.empty((B, hq + 2 * hkv, 128), dtype=torch.bfloat16, device="cuda")
    q, k, v = qkv.split((hq, hkv, hkv), 1)
    slots, pos = torch.empty(B, dtype=torch.int64, device="cuda"), torch.empty(B, dtype=torch.int32, device="cuda")
    before = torch.empty_like(sl)
    qr, out = (torch.empty((B, hq, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    lse, scores = torch.empty((B, hq), device="cuda"), torch.zeros((B, hkv, cols), device="cuda")
    sel = torch.empty((B, hkv, budget), dtype=torch.int32, device="cuda")
    ws = torch.empty(kv.nvfp4kv_decode_workspace_size(cache, B, hq), dtype=U8, device="cuda")
    status = status_word()

    def step():
        before.copy_(sl)
        kv.nvfp4kv_plan_append(pt, sl, new, stack, count, num_pages, sl, slots, count, positions=pos, device_status=status)
        kv.nvfp4kv_norm_rope_append(cache, q, k, v, slots, pos, dcs, qr, q_weight=dw[0], k_weight=dw[1], eps=EPS,
                                    device_status=status)
        kv.nvfp4kv_page_digest(cache, pt, sl, digest, first_tokens=before, device_status=status)
        kv.nvfp4kv_page_scores(cache, digest, qr, pt, sl, SCALE, scores, device_status=status)
        kv.nvfp4kv_select_pages(scores, sl, budget, first, recent, sel, device_status=status)
        kv.nvfp4kv_decode_attention_selected(cache, qr, out, pt, sl, SCALE, sel, ws, lse=lse, device_status=status)

    graph = torch.cuda.CUDAGraph()
    qkv.zero_()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    left = num_pages - at
    for i in range(steps):
        x = bf16_round(rng.standard_normal((B, hq + 2 * hkv, 128)) * 2.0)
        qkv.copy_(torch.from_numpy(x).to(torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        assert status.item() == 0
        for b in range(B):                                                     # the new pages, off the top of the stack
            if lens[b] % 16 == 0:
                left -= 1
                table[b, lens[b] // 16] = ids[at + left]
        same(pt.cpu().numpy(), table, "page table")
        assert count.item() == left
        p = np.asarray(lens, np.int32)
        made = [bf16_round(norm_rope_steps(a, w, EPS, cs, p, False)) for a, w in zip((x[:, :hq], x[:, hq:hq + hkv]), weights)]
        at_slot = np.array([int(table[b, n // 16]) * 16 + n % 16 for b, n in enumerate(lens)], np.int64)
        oracle.quantize_append(o, bits(made[1]), bits(x[:, hq + hkv:]), at_slot)
        for name, got, want in zip(PARTS, pool_host(cache), (o.k_data, o.v_data, o.k_scale, o.v_scale)):
            same(got, want, name)
        same(bits(qr.float().cpu().numpy()), bits(made[0]), "queries")
        lens = [n + 1 for n in lens]
        assert sl.tolist() == lens
        raw, sc, se = digest.cpu().numpy(), scores.cpu().numpy(), sel.cpu().numpy()
        got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
        for b, n in enumerate(lens):
            pages = -(-n // 16)
            for h in range(hkv):
                K, _ = sequence_rows(o, table[b], h, n)
                heads = made[0][b, h * group:(h + 1) * group].astype(np.float64)
                for page in range(pages):
                    hi, lo, scale = digest_ref(K[16 * page:16 * page + 16] / o.k_global_scale)
                    r = raw[table[b, page], h]
                    assert np.array_equal(e4m3_values(r[:128]), hi) and np.array_equal(e4m3_values(r[128:256]), lo)
                    want, tol = score_ref(heads, hi, lo, scale, SCALE * o.k_global_scale)
                    assert abs(sc[b, h, page] - want) <= tol
                chosen = evict_ref(sc[b, h, :pages], pages, budget, first, recent)
                assert np.array_equal(se[b, h, :len(chosen)], chosen) and (se[b, h, len(chosen):] == -1).all()
                for g in range(group):
                    r = attend_ref(o, table[b], h, n, chosen, heads[g])
                    check(got[b, h * group + g], r["out"], r["tol_out"], f"{i} {b} {h} {g}")
                    check(gl[b, h * group + g], r["lse"], r["tol_lse"], f"lse {i} {b} {h} {g}")
