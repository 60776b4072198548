"""Where the calls that do not read the whole cache meet the borders of what they promise: rows of zeros beside pages
outside the cache or bounds that are infinite, prefixes that end behind a sequence's context, keys and bounds that are no
numbers, batches beyond 64 bits."""
import ctypes
import math

import pytest
import torch

from quantized_moe_expert_dequant_gb300 import binding as Bn
from tests import attention_cases as C
from tests import sparse_cases as S
from tests.test_attention_host import attention, cache
from tests.test_gpu_pages import random_bounds, run_bounds, run_select, shape

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16
i32 = dict(dtype=torch.int32, device="cuda")


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


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("lens", [[1], [1] * 40, [1] * 200, [7], [16, 1, 13]])
@pytest.mark.parametrize("pages", [100, 5000])
def test_rows_of_zeros_beside_infinite_bounds(lens, pages, dtype):
    """Zero times infinity is no number: such a page comes last, with those outside the cache, and changes nothing about
    the others."""
    lens = lens[:60] if pages > 1000 else lens
    ctx = [16 * 99] * len(lens)
    b = C.batch(1, lens, ctx, 4, 2, 64, 16, dtype)
    b.table = b.table[:, torch.arange(pages) % 100].contiguous()  # (pages may be there more than once)
    b.ctxs = [16 * (pages - 1)] * len(lens)
    b.ctx[:] = 16 * (pages - 1)
    bnd = random_bounds(b, 1)
    b.q.zero_()
    gone = [2, 3, 50, 97]
    for i in range(len(lens)):
        bnd[int(b.table[i, 4]), :, 1, 9] = float("inf")
    worst = gone + list(range(4, pages, 100))
    b.table[:, gone] = b.k.shape[0] + 3
    free = [j for j in range(1, pages - 1) if j not in worst] + sorted(worst)
    for n_select in (10, 70, pages - 3):
        want = sorted([0, pages - 1] + free[:n_select - 2])
        got, err = run_select(b, bnd, n_select)
        assert err == 1 and bool((got == torch.tensor(want, dtype=torch.int32)).all())


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("n,max_q", [(5, 2), (60, 2), (60, 64)])  # clusters, all CTAs, tiles of 128 rows
def test_prefixes_that_end_behind_a_sequences_context(n, max_q, dtype):
    """A sequence with fewer positions before its queries than the prefix has is computed by itself, also when it has
    the prefix's whole pages: what its own pages hold there is its own."""
    prefix, page = 130, 16
    lens = [1 + i % 2 for i in range(n)]
    ctxs = [[130, 129, 128, 131, 127][i % 5] for i in range(n)]
    b = C.batch(n + max_q, lens, ctxs, 4, 2, 64, page, dtype)
    for i in range(1, n):
        if ctxs[i] >= prefix:
            b.table[i, :prefix // page] = b.table[0, :prefix // page]
    err = torch.zeros(1, **i32)
    got = Bn.prefix_attention(Bn.KvCache(b.k, b.v), b.q, b.cu, b.ctx, b.table, torch.tensor([0, n], **i32),
                              torch.tensor([prefix], **i32), max_q, scale=0.2, device_error=err)
    ref, tol = b.reference(0.2)
    C.assert_within(got, ref, tol)
    assert int(err) == 0


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("D,page", [(64, 16), (128, 64), (64, 1024)])
def test_bounds_of_keys_that_are_no_numbers(dtype, D, page):
    """They show in both bounds of their dimension, wherever on the page they are, and in no other's."""
    lens, ctxs = [1, 300, 2 * page], [0, 7, page - 1]
    b = C.batch(D, lens, ctxs, 4, 2, D, page, dtype)
    for i, at, h, d in ((0, 0, 0, 3), (1, 20, 1, D - 1), (2, 3 * page - 2, 0, 8), (2, page + 9, 1, 0)):
        b.k[int(b.table[i, at // page]), h, at % page, d] = float("nan")
    b.k[int(b.table[1, 16 // page]), 0, :, 17] = float("nan")  # all of a dimension's
    before = random_bounds(b, 1)
    got, err = run_bounds(b, before)
    want = S.bounds(b, before)
    assert err == 0 and int(want.isnan().sum()) == 10
    assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.nan_to_num(0.0), want.nan_to_num(0.0))
    # such a page has the lowest score
    i, page_i = 1, int(b.table[1, 20 // page])
    rows = b.q[1:2]
    if page == 16:
        ctx = torch.tensor([16 * 18], **i32)
        picked = Bn.select_pages(Bn.KvCache(b.k, b.v), got, rows, torch.tensor([0, 1], **i32), ctx, b.table[1:2], 18, 0)
        lost = [j for j in range(19) if j not in picked[0, 1].tolist()]
        assert lost == [20 // page] and int(b.table[1, lost[0]]) == page_i


def test_pages_that_are_no_numbers_hide_no_sizes():
    """What fp32 scores may be off goes by the largest bounds of all pages, whichever order a thread meets them in: pages
    that only exact sums tell apart, then some of NaN, then some of zeros."""
    pages = 16 * 128 + 3
    b = C.batch(8, [1], [16 * (pages - 1)], 2, 1, 64, 16, F16)
    b.q[:] = torch.tensor([1.0, -1.0], device="cuda")[None, :, None].to(F16) * 2.0 ** -6
    b.q[:, :, 0] = 1024.0
    gen = torch.Generator().manual_seed(9)
    bnd = torch.randint(-3, 4, shape(b), generator=gen).sort(2).values.to(F16).cuda() / 16
    bnd[..., 0] = 512.0
    place = torch.arange(pages - 2) % 128  # of the pages that are scored, from the second on
    of = b.table[0, 1:pages - 1].long().cpu()
    bnd[of[(place >= 32) & (place < 64)]] = float("nan")
    bnd[of[place >= 64]] = 0.0
    s = S.scores(b, bnd, 0, 0, 0, pages)[1:-1]
    key = s.masked_fill(s.isnan(), -math.inf).tolist()
    order = sorted(range(len(key)), key=lambda j: (-key[j], j))
    for n_select in (12, 200, 400):
        want = sorted([0, pages - 1] + [1 + j for j in order[:n_select - 2]])
        got, err = run_select(b, bnd, n_select)
        assert err == 0 and got[0, 0].tolist() == want


def test_batches_beyond_64_bits_are_refused():
    """The tiles' line counts eight units a position and item, and its length times the CTAs has to fit.  (The question
    for the workspace is all that is asked here: 2^30 positions in each of a million sequences.)"""
    L, n = Bn.lib(), ctypes.c_int64()
    c = cache(page_size=1024, head_dim=128, n_pages=2 ** 20, n_kv_heads=8, head_stride=1024 * 128, token_stride=128,
              page_stride=8 * 1024 * 128)
    many = dict(table_width=2 ** 20, table_stride=2 ** 20, n_q_heads=8)
    ask = lambda seqs: L.moe_prefix_attention_workspace(
        ctypes.byref(c), ctypes.byref(attention(n_seqs=seqs, n_rows=seqs, **many)), 1, 64, ctypes.byref(n))
    assert ask(10 ** 6) == Bn.MOE_ERR_UNSUPPORTED
    assert ask(10 ** 5) == Bn.MOE_OK and n.value > 0
