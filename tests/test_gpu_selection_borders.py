"""The page selection where its threshold lies at the end of one of the parts
that it searches, scores on both sides, in every shape of its kernel."""
import numpy as np
import pytest
import torch

import nvfp4_quantized_paged_quantize_gb300 as kv
from gpu_util import dev, status_word
from select_model import border_wants, scores_across_an_end, scores_below_one_far_above, sorted_kept
from step_util import same
from test_gpu_canary import Guarded

pytestmark = pytest.mark.gpu

# pages that the scores have room for, pairs, parts: 256 threads; 1024 with 9 scores each; 1024 with 16 and more;
# clusters with 9; clusters with 16 and more; and, of many pairs, 1024 threads with more than 16
SHAPES = [(2000, 6, 1024), (2048, 5, 1024), (9000, 6, 2048), (15000, 6, 2048), (17000, 6, 2048), (80000, 6, 2048),
          (17000, 80, 2048)]


def check(x, budget, first=0, recent=0):
    """Rows of x float32 [pairs, pages], each a sequence's with one KV head."""
    pairs, n = x.shape
    out, status = Guarded((pairs, 1, budget), torch.int32), status_word()
    out.t.fill_(-7)
    kv.nvfp4kv_select_pages(dev(x[:, None]), dev(np.full(pairs, 16 * n - 5, np.int32)), budget, first, recent, out.t,
                            device_status=status)
    torch.cuda.synchronize()
    assert out.intact() and status.item() == 0
    got = out.t[:, 0].cpu().numpy().astype(int)
    for i in range(pairs):
        middle = sorted_kept(x[i, first:n - recent], budget - first - recent) if budget > first + recent else np.zeros(0, int)
        same(got[i], np.concatenate([np.arange(first), first + middle, np.arange(n - recent, n)]), f"row {i}")


@pytest.mark.parametrize("pages,pairs,bins", SHAPES)
@pytest.mark.parametrize("close,equal", [(3, 5), (3, 800), (200, 200), (400, 30), (400, 900)])
def test_scores_across_a_parts_end(cuda_lib, pages, pairs, bins, close, equal):
    x = np.stack([scores_across_an_end(pages, bins, close, equal, seed) for seed in range(pairs)])
    wants = border_wants(x[0], bins)
    assert len(wants) == close and all(border_wants(row, bins) == wants for row in x[1:3])
    for want in sorted({wants[0] - 1, wants[0], wants[1], wants[len(wants) // 2], wants[-1], wants[-1] + 1}):
        check(x, want)
    # the same with pages that stay in any case around them
    y = np.concatenate([np.full((pairs, 2), -9.0), x[:, :pages - 5], np.full((pairs, 3), 9.0)], 1).astype(np.float32)
    for want in border_wants(y[0, 2:-3], bins)[:2]:
        check(y, want + 5, 2, 3)


@pytest.mark.parametrize("pages,pairs,bins", SHAPES)
def test_scores_below_one_far_above(cuda_lib, pages, pairs, bins):
    x = np.stack([scores_below_one_far_above(pages, seed) for seed in range(pairs)])
    wants = sorted({w for row in x for w in border_wants(row, bins)})
    assert wants
    for want in wants[::max(1, len(wants) // 10)]:
        check(x, want)
