"""The decode over selected pages with long lists to a warp: stages filled again
and again, the next entries taken over half way through a chunk of 32, the table of
64 entries going round, against the 64-bit reference."""
import numpy as np
import pytest
import torch

import nvfp4_quantized_paged_quantize_gb300 as kv
from scored_util import random_cache
from test_gpu_page_selection import pages_of, run_attend

pytestmark = pytest.mark.gpu


def most_entries(pairs, listed):
    """Entries of the longest warp's part, by the launch's rule: as many CTAs to a pair, up to eight, as two to an SM give
    room for, eight warps each; None where the device-wide cut is taken instead."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    splits = 1
    while splits < 8 and pairs * (splits + 1) <= 2 * sms:
        splits += 1
    ctas = pairs * splits
    if ctas > 2 * sms or listed * sms > 512 * splits * min(ctas, sms):
        return None
    return max((c1 - c0) * (w + 1) // 8 - (c1 - c0) * w // 8
               for c0, c1 in ((listed * r // splits, listed * (r + 1) // splits) for r in range(splits)) for w in range(8))


def long_lists(lens, budget, seed):
    """Lists in mixed order: distinct pages, the partial last one among them, entries that name none, and (of the last
    long sequence) some past its end."""
    rng = np.random.default_rng(seed)
    sel = np.full((len(lens), 1, budget), -1, np.int32)
    for b, n in enumerate(pages_of(lens)):
        m = min(n, budget)
        pick = rng.permutation(n)[:m]
        if m and n - 1 not in pick:
            pick[rng.integers(m)] = n - 1
        pick[rng.random(m) < 0.1] = -1
        if m and n - 1 not in pick:
            pick[m - 1 - rng.integers(min(m, 3))] = n - 1
        sel[b, 0, :m] = pick
    return sel


@pytest.mark.parametrize("pairs,budget,entries", [(160, 40, 5), (160, 64, 8), (160, 248, 31), (160, 256, 32), (160, 264, 33),
                                                  (160, 272, 34), (160, 384, 48), (160, 504, 63), (160, 512, 64), (160, 509, 64),
                                                  (304, 130, 17), (120, 528, 33), (120, 1024, 64), (70, 2048, 64), (38, 4096, 64)])
def test_long_lists(cuda_lib, pairs, budget, entries):
    assert most_entries(pairs, budget) == entries
    rng = np.random.default_rng(budget)
    # a few long sequences: all of the list used, a little more and a little less than that, half of it
    long = [16 * (budget + 7) - 5, 16 * budget, 16 * budget - 15, 8 * budget + 3]
    lens = rng.integers(0, 40, pairs)
    lens[rng.permutation(pairs)[:len(long)]] = long
    used = 97                                        # physical pages, which the sequences share
    table = rng.integers(0, used, (pairs, budget + 7)).astype(np.int32)
    cache, o = random_cache(used, 1, budget + 1, gk=0.3, gv=0.5)
    sel = long_lists(lens, budget, budget + 2)
    run_attend(cache, o, table, lens.tolist(), 2, sel, budget + 3)
    # entries past the sequences' ends, and pages outside the pool, all along the lists
    b = int(np.argmax(lens))
    at = np.arange(3, budget, 11)
    sel[b, 0, at] = pages_of(lens)[b] + at
    bad = {int(p) for p in sel[b, 0, 5::17] if 0 <= p < pages_of(lens)[b]}
    table[b, sorted(bad)] = used
    run_attend(cache, o, table, lens.tolist(), 2, sel, budget + 4, flags=kv.NVFP4KV_DEVERR_PAGE, skip={(b, p) for p in bad})
