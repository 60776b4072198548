"""Where the calls that do not read the whole cache meet the borders of what they promise: rows of zeros beside pages
outside the cache."""
import math

import pytest
import torch

from tests import attention_cases as C
from tests import sparse_cases as S
from tests.test_gpu_pages import random_bounds, run_select

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def select_without(b, bnd, gone, n_select, sink, recent):
    """S.select where the pages `gone` of every sequence are outside the cache: they have the lowest score."""
    rows, Hkv, ps = b.q.shape[0], b.k.shape[1], b.k.shape[2]
    out = torch.full((rows, Hkv, n_select), -7, dtype=torch.int32)
    at = 0
    for i, (n, c) in enumerate(zip(b.lens, b.ctxs)):
        for r in range(at, at + n):
            pages = (c + r - at) // ps + 1
            for h in range(Hkv):
                s = S.scores(b, bnd, i, r, h, pages).tolist()
                s = [-math.inf if j in gone else x for j, x in enumerate(s)]
                free = sorted(range(sink, pages - recent), key=lambda j: (-s[j], j))
                chosen = list(range(sink)) + list(range(pages - recent, pages)) + free[:n_select - sink - recent]
                assert len(chosen) == n_select < pages
                out[r, h] = torch.tensor(sorted(chosen))
        at += n
    return out


# tokens by themselves (clusters of 16, of 2 and blocks alone), and chunks
@pytest.mark.parametrize("lens", [[1], [1] * 40, [1] * 200, [7], [16, 1, 13]])
@pytest.mark.parametrize("pages,gone,n_select", [
    (10, [1], 4), (10, [3, 4, 5], 8), (18, list(range(9, 17)), 12), (18, list(range(1, 9)), 12),
    (10, list(range(1, 9)), 5), (40, list(range(1, 30)), 20), (300, list(range(2, 290)), 100),
    (300, [5, 6, 290], 298)])
def test_rows_of_zeros_beside_pages_outside_the_cache(lens, pages, gone, n_select):
    """All scores are 0 but those of the pages outside, which come last.  (Every row sees all pages.)"""
    b = C.batch(1, lens, [16 * (pages - 1)] * len(lens), 4, 2, 64, 16, BF16)
    bnd = random_bounds(b, 1)
    b.q[::2] = 0.0
    want = select_without(b, bnd, gone, n_select, 1, 1)
    b.table[:, gone] = b.k.shape[0] + 3
    got, err = run_select(b, bnd, n_select)
    assert err == 1 and torch.equal(got, want)
