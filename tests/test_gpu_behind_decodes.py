"""Calls right behind the library's own decodes: what they write comes after
everything that the decode, and an append ahead of it, read and wrote."""
import numpy as np
import pytest
import torch

import nvfp4_quantized_paged_quantize_gb300 as kv
from gpu_util import dev, status_word
from scored_util import SCALE, page_tables, random_cache, random_q

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def bf16(rng, *shape):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(BF16).cuda()


class Batch:
    """Sequences of no more than a page each (no pair of which the decode cuts), and the tokens of the step after them."""

    def __init__(self, lens, hkv=8, hq=16, seed=1):
        rng = np.random.default_rng(seed)
        self.B, self.hq, self.hkv = len(lens), hq, hkv
        table, used = page_tables(lens, seed, extra_cols=2)
        self.num_pages = used + self.B
        cache, _ = random_cache(self.num_pages, hkv, seed)
        self.pages = cache.pages.clone()
        self.cache = cache
        self.table, self.lens = dev(table), dev(np.asarray(lens, np.int32))
        self.free = dev(np.arange(used, self.num_pages, dtype=np.int32))
        self.q, _ = random_q((self.B, hq, 128), seed + 1)
        self.k, self.v, self.q2, self.k2, self.v2 = (bf16(rng, self.B, h, 128) for h in (hkv, hkv, hq, hkv, hkv))
        self.ones = torch.ones(self.B, dtype=torch.int32, device="cuda")
        # where an append ahead of the decode puts its tokens: the last ones that the decode reads (in pages of the free
        # stack's far end for sequences of none)
        slots = [int(table[b, 0]) * 16 + n - 1 if n else (used + b) * 16 for b, n in enumerate(lens)]
        self.slots = dev(np.asarray(slots, np.int64))
        self.out = torch.empty((self.B, hq, 128), device="cuda")
        self.ws = torch.zeros(kv.nvfp4kv_decode_workspace_size(cache, self.B, hq), dtype=torch.uint8, device="cuda")
        self.busy = torch.rand((2000, 2000), device="cuda")
        # what the step works on
        self.t, self.l, self.qs = self.table.clone(), self.lens.clone(), self.q.clone()
        self.count, self.plan_slots = dev(np.array([self.B], np.int32)), torch.empty(self.B, dtype=torch.int64, device="cuda")
        self.status = status_word()

    def reset(self):
        self.cache.pages.copy_(self.pages)
        self.t.copy_(self.table)
        self.l.copy_(self.lens)
        self.qs.copy_(self.q)
        self.count.fill_(self.B)
        self.out.fill_(float("nan"))
        self.busy.mul_(1.0)                                    # so that the calls queue up behind one another

    def decode(self, fused):
        if fused:
            kv.nvfp4kv_append_decode_attention(self.cache, self.k, self.v, self.slots, self.qs, self.out, self.t, self.l, SCALE, self.ws)
        else:
            kv.nvfp4kv_decode_attention(self.cache, self.qs, self.out, self.t, self.l, SCALE, self.ws)

    def plan(self):
        kv.nvfp4kv_plan_append(self.t, self.l, self.ones, self.free, self.count, self.num_pages, self.l, self.plan_slots, self.count,
                               device_status=self.status)

    def append(self):
        # into the decode's queries, and over the tokens that the append ahead wrote and the decode read
        kv.nvfp4kv_norm_rope_append(self.cache, self.q2, self.k2, self.v2, self.slots, None, None, self.qs)

    def state(self):
        return [x.clone() for x in (self.out, self.cache.pages, self.t, self.l, self.qs, self.plan_slots, self.count)]


LENS = {"a page each": [1 + b % 16 for b in range(1000)], "pages and nothing": [(b * 7) % 17 for b in range(300)],
        "nothing": [0] * 64, "more than 1024": [b % 17 for b in range(1500)]}


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("behind", ["plan", "append", "plan and append"])
def test_calls_behind_a_decode(cuda_lib, behind, lens, fused, captured):
    b = Batch(LENS[lens])
    calls = [b.plan] * ("plan" in behind) + [b.append] * ("append" in behind)
    # one call at a time
    b.reset()
    for call in [lambda: b.decode(fused)] + calls:
        torch.cuda.synchronize()
        call()
    torch.cuda.synchronize()
    want = b.state()

    def step():
        b.reset()
        b.decode(fused)
        for call in calls:
            call()

    if captured:
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
            step()
    for _ in range(5):
        graph.replay() if captured else step()
        torch.cuda.synchronize()
        for name, x, y in zip(("out", "pages", "table", "lens", "queries", "slots", "count"), b.state(), want):
            assert torch.equal(x, y), name
    assert b.status.item() == 0
