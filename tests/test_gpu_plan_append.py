"""The step plan: page tables, slots, positions and workspace rows against the
reference, request by request."""
import numpy as np
import pytest
import torch

import nvfp4_quantized_paged_quantize_gb300 as kv
from gpu_util import dev, status_word
from step_util import plan_ref
from test_gpu_canary import Guarded

pytestmark = pytest.mark.gpu

I32, I64 = torch.int32, torch.int64


class Plan:
    def __init__(self, cached, new, spare=5, tokens=None, extra_cols=2, seed=1, free=None, count=None, cols=None):
        rng = np.random.default_rng(seed)
        self.cached, self.new = np.asarray(cached, np.int32), np.asarray(new, np.int32)
        B, room = len(self.cached), cols * 16 if cols else 1 << 20
        fit = np.clip(self.cached.astype(np.int64), 0, room)                   # what the table has room for
        add = np.clip(self.new.astype(np.int64), 0, room - fit)
        have = -(-fit // 16)
        need = -(-(fit + add) // 16) - have
        cols = cols or int((have + need).max(initial=0)) + extra_cols
        self.num_pages = int(have.sum() + need.sum()) + spare
        ids = rng.permutation(self.num_pages).astype(np.int32)
        self.table = np.full((B, cols), -7, np.int32)
        at = 0
        for b, n in enumerate(np.minimum(have, cols)):
            self.table[b, :n] = ids[at:at + n]
            at += n
        self.free = ids[at:] if free is None else free
        self.count = len(self.free) if count is None else count
        self.tokens = int(add.sum()) + 3 if tokens is None else tokens
        self.pt, self.cl, self.nl, self.fp = dev(self.table), dev(self.cached), dev(self.new), dev(self.free)
        self.fc = dev(np.array([self.count], np.int32))
        self.outs = {"lens": Guarded((B,), I32), "slots": Guarded((self.tokens,), I64), "positions": Guarded((self.tokens,), I32),
                     "rows": Guarded((self.tokens,), I64), "cu_q": Guarded((B + 1,), I64), "cu_rows": Guarded((B + 1,), I64),
                     "free_left": Guarded((1,), I32)}
        self.status = status_word()

    def run(self):
        o = {k: g.t for k, g in self.outs.items()}
        kv.nvfp4kv_plan_append(self.pt, self.cl, self.nl, self.fp, self.fc, self.num_pages, o["lens"], o["slots"],
                               o["free_left"], positions=o["positions"], cu_q=o["cu_q"], ws_rows=o["rows"],
                               cu_prefix=o["cu_rows"], device_status=self.status)

    def check(self):
        torch.cuda.synchronize()
        want = plan_ref(self.table, self.cached, self.new, self.free, self.count, self.num_pages, self.tokens)
        assert self.status.item() == want["flags"]
        assert np.array_equal(self.pt.cpu().numpy(), want["table"])
        for k, g in self.outs.items():
            assert g.intact(), k
            assert g.t.tolist() == want[k], k
        return want


@pytest.mark.parametrize("batch,high,new", [(1, 0, 1), (1, 17, 0), (5, 40, 1), (7, 100, 33), (16, 3000, 700), (300, 500, 1),
                                            (1024, 64, 3), (1025, 64, 20), (2500, 30, 1), (3, 10, 9000)])
def test_plan(cuda_lib, batch, high, new):
    rng = np.random.default_rng(batch + new)
    p = Plan(rng.integers(0, high + 1, batch), rng.integers(0, new + 1, batch), seed=batch)
    p.run()
    want = p.check()
    assert want["flags"] == 0 and want["cu_q"][-1] == p.new.sum()


def test_page_borders_and_idle_requests(cuda_lib):
    # lengths around a page's end, with and without new tokens, no request at the front or the end taking any
    p = Plan([0, 0, 15, 16, 17, 31, 32, 1, 0, 16], [0, 1, 1, 1, 15, 1, 16, 0, 17, 0])
    p.run()
    assert p.check()["flags"] == 0


def test_no_requests_and_no_room(cuda_lib):
    p = Plan(np.zeros(0), np.zeros(0), tokens=5, cols=1)
    p.run()
    assert p.check()["flags"] == 0
    p = Plan([20, 3], [0, 0], tokens=0)
    p.run()
    assert p.check()["flags"] == 0


@pytest.mark.parametrize("count,tokens", [(0, 100), (1, 100), (3, 100), (4, 100), (100, 0), (100, 16), (100, 17), (100, 57)])
def test_too_few_pages_or_places(cuda_lib, count, tokens):
    # requests of 1, 16, 40, 0, 3 and 2 new tokens: the first that does not fit ends the plan, also for a smaller one behind
    p = Plan([15, 16, 100, 5, 16, 4], [1, 16, 40, 0, 3, 2], spare=100, tokens=tokens, count=count)
    p.run()
    want = p.check()
    # 0, 1, 2, 0, 1 and 0 pages: four; 62 tokens
    assert want["flags"] == (0 if count >= 4 and tokens >= 62 else kv.NVFP4KV_DEVERR_POOL)


def test_too_few_over_many_requests(cuda_lib):
    rng = np.random.default_rng(9)
    for at in (5, 1023, 1024, 1025, 2047, 2400):
        cached, new = rng.integers(0, 50, 2500), rng.integers(0, 4, 2500)
        new[at] = 3
        p = Plan(cached, new, tokens=int(new[:at + 1].sum()) - 1)
        p.run()
        want = p.check()
        assert want["flags"] == kv.NVFP4KV_DEVERR_POOL and want["cu_q"][-1] == new[:at].sum()


def test_bad_inputs_are_flagged(cuda_lib):
    # lengths below 0 and past the table (4 columns); page ids outside the pool, in the table and on the stack
    p = Plan([-5, 60, 70, 10, 2 ** 31 - 1, 3], [20, 5, 1, -3, 7, 2 ** 31 - 1], cols=4, spare=20)
    p.run()
    assert p.check()["flags"] & kv.NVFP4KV_DEVERR_LENGTH
    free = np.array([3, 1 << 30, -1, 2], np.int32)
    p = Plan([5, 0], [3, 40], free=free, cols=4, spare=1)
    p.table[0, 0] = p.num_pages
    p.pt = dev(p.table)
    p.run()
    assert p.check()["flags"] == kv.NVFP4KV_DEVERR_PAGE
    assert p.outs["slots"].t[:3].tolist() == [-1, -1, -1]
    for count in (-1, 5):
        p = Plan([0, 0], [16, 20], free=np.array([0, 1, 2, 3], np.int32), count=count, cols=4)
        p.run()
        assert p.check()["flags"] & kv.NVFP4KV_DEVERR_LENGTH


def test_sums_past_32_bits(cuda_lib):
    # requests that want 2^20 tokens each (3000 of them: more than 2^31 together), in small and in large blocks; the
    # first one fits
    for batch in (200, 3000):
        p = Plan(np.zeros(batch), np.zeros(batch), cols=1 << 16, tokens=50, spare=4)
        p.new[0], p.new[1:] = 20, 1 << 20
        p.nl = dev(p.new)
        p.run()
        want = p.check()
        assert want["flags"] == kv.NVFP4KV_DEVERR_POOL and want["lens"][:2] == [20, 0]


def test_in_place_and_without_the_optional_outputs(cuda_lib):
    rng = np.random.default_rng(3)
    for batch in (4, 1500):
        cached, new = rng.integers(0, 90, batch), rng.integers(0, 12, batch)
        p = Plan(cached, new)
        want = plan_ref(p.table, cached, new, p.free, p.count, p.num_pages, p.tokens)
        kv.nvfp4kv_plan_append(p.pt, p.cl, p.nl, p.fp, p.fc, p.num_pages, p.cl, p.outs["slots"].t, p.fc, device_status=p.status)
        torch.cuda.synchronize()
        assert p.cl.tolist() == want["lens"] and p.fc.tolist() == want["free_left"]
        assert p.outs["slots"].t.tolist() == want["slots"] and p.outs["slots"].intact()
        assert np.array_equal(p.pt.cpu().numpy(), want["table"]) and p.status.item() == 0


def test_captured_steps(cuda_lib):
    # a captured decode step: every replay appends one token to each request, in place
    batch, steps = 9, 40
    p = Plan(np.arange(batch) * 7, np.ones(batch), spare=batch * 4, tokens=batch, extra_cols=4)
    graph = torch.cuda.CUDAGraph()
    args = (p.pt, p.cl, p.nl, p.fp, p.fc, p.num_pages, p.cl, p.outs["slots"].t, p.fc)
    kv.load()
    with torch.cuda.graph(graph):
        kv.nvfp4kv_plan_append(*args, positions=p.outs["positions"].t, device_status=p.status)
    table, lens, count = p.table, p.cached, p.count
    for _ in range(steps):
        graph.replay()
        want = plan_ref(table, lens, p.new, p.free, count, p.num_pages, batch)
        table, lens, count = want["table"], want["lens"], want["free_left"][0]
        assert p.outs["slots"].t.tolist() == want["slots"] and p.outs["positions"].t.tolist() == want["positions"]
    assert p.cl.tolist() == list(lens) and p.fc.item() == count and p.status.item() == 0
    assert np.array_equal(p.pt.cpu().numpy(), table)
