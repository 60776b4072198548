"""Bounds of a page's keys (moe_page_bounds) and the selection of pages by them (moe_select_pages): both
are exact."""
import pytest
import torch

from quantized_moe_expert_dequant_gb300 import binding as Bn
from tests import attention_cases as C
from tests import sparse_cases as S

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16


def shape(b):
    return (b.k.shape[0], b.k.shape[1], 2, b.k.shape[3])


def random_bounds(b, seed, spread=1.0):
    gen = torch.Generator().manual_seed(seed)
    mid = torch.randn(shape(b)[:2] + (1, b.k.shape[3]), generator=gen) * spread
    reach = torch.rand(shape(b), generator=gen) + 0.5
    reach[:, :, 0] *= -1
    return (mid + reach).to(b.k.dtype).cuda()


def run_bounds(b, before, rows=None, **kw):
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = Bn.page_bounds(Bn.KvCache(b.k, b.v), before.clone(), b.cu, b.ctx, b.table,
                         n_rows=sum(b.lens) if rows is None else rows, device_error=err, **kw)
    torch.cuda.synchronize()
    return got, int(err)


def run_select(b, bnd, n_select, sink=1, recent=1, **kw):
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((b.q.shape[0], b.k.shape[1], n_select), -7, dtype=torch.int32, device="cuda")
    got = Bn.select_pages(Bn.KvCache(b.k, b.v), bnd, b.q, b.cu, b.ctx, b.table, n_select, sink,
                          recent, out=out, device_error=err, **kw)
    torch.cuda.synchronize()
    assert got is out
    return got.cpu(), int(err)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("D,page", [(64, 16), (128, 64), (64, 128), (128, 16), (128, 1024)])
def test_bounds(dtype, D, page):
    lens = [1, 1, 0, 70, 1, 300, 2, 1]
    ctxs = [0, 15, 40, 0, 1000, 63, 2 * page - 1, page]
    # stale values are NaN: none of them may show
    b = C.batch(D + page, lens, ctxs, 4, 2, D, page, dtype, token_major=page == 64)
    before = random_bounds(b, 1)
    got, err = run_bounds(b, before)
    assert err == 0
    assert torch.equal(got, S.bounds(b, before))
    again, _ = run_bounds(b, before, rows=sum(lens) + 9)  # rows is a bound
    assert torch.equal(again, got)


def test_bounds_of_many_sequences():
    lens = [(7 * i) % 4 for i in range(700)]
    ctxs = [(13 * i) % 50 for i in range(700)]
    b = C.batch(3, lens, ctxs, 2, 1, 64, 16, BF16)
    before = random_bounds(b, 2)
    got, err = run_bounds(b, before)
    assert err == 0 and torch.equal(got, S.bounds(b, before))


def test_bounds_on_bad_pages_and_sequences():
    b = C.batch(4, [3, 2, 40], [5, 9, 100], 2, 1, 64, 16, F16)
    before = random_bounds(b, 2)
    want = S.bounds(b, before)
    lost = [int(b.table[2, 7])]
    b.table[2, 7] = b.k.shape[0] + 5  # a page outside the cache
    lost += [int(b.table[1, j]) for j in range(1)]
    b.ctx[1] = 10 ** 6  # a sequence outside its table
    want[lost] = before[lost]
    got, err = run_bounds(b, before)
    assert err == 1 and torch.equal(got, want)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("Hq,Hkv,D,page,n_select,sink,recent", [
    (8, 2, 128, 16, 7, 1, 1), (4, 4, 64, 16, 9, 0, 2), (64, 1, 64, 32, 4, 2, 2),
    (6, 1, 128, 64, 5, 1, 3), (12, 2, 64, 16, 40, 4, 1)])
def test_select(dtype, Hq, Hkv, D, page, n_select, sink, recent):
    lens = [1, 3, 0, 1, 37, 1, 6]
    ctxs = [0, 20 * page - 1, 7, page * n_select, 30 * page + 5, 3000, page * n_select - 3]
    b = C.batch(Hq + D + n_select, lens, ctxs, Hq, Hkv, D, page, dtype, pad_rows=3)
    bnd = random_bounds(b, 5)
    got, err = run_select(b, bnd, n_select, sink, recent)
    assert err == 0
    assert torch.equal(got, S.select(b, bnd, n_select, sink, recent))


def test_select_single_tokens_and_streams():
    ctxs = [0, 15, 16, 300, 2000, 4100, 4096]
    b = C.batch(6, [1] * len(ctxs), ctxs, 8, 2, 128, 16, BF16)
    bnd = random_bounds(b, 6)
    want = S.select(b, bnd, 16, 1, 2)
    got, err = run_select(b, bnd, 16, 1, 2)
    assert err == 0 and torch.equal(got, want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, err = run_select(b, bnd, 16, 1, 2, stream=side)
    assert err == 0 and torch.equal(got, want)


def test_select_in_long_contexts():
    # more pages than the scores that are kept in shared memory
    b = C.batch(7, [2, 1], [150000, 131072], 4, 2, 64, 16, F16)
    bnd = random_bounds(b, 7)
    got, err = run_select(b, bnd, 65, 1, 2)
    assert err == 0 and torch.equal(got, S.select(b, bnd, 65, 1, 2))


@pytest.mark.parametrize("n_select", [12, 500])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_select_scores_that_fp32_does_not_tell_apart(dtype, n_select):
    """One dimension adds 2^20 to every score, the others differ by far less than its fp32 step (2^-3):
    the order is in bits that only exact sums have.  Ties go to the lower page."""
    b = C.batch(8, [1, 2], [16 * 900 + 3, 16 * 700], 2, 1, 64, 16, dtype)
    b.q[:] = torch.tensor([1.0, -1.0], device="cuda")[None, :, None].to(dtype) * 2.0 ** -6
    b.q[:, :, 0] = 1024.0
    gen = torch.Generator().manual_seed(9)
    bnd = torch.randint(-3, 4, shape(b), generator=gen).sort(2).values.to(dtype).cuda() / 16
    bnd[..., 0] = 512.0
    want = S.select(b, bnd, n_select, 1, 1)
    s = S.scores(b, bnd, 0, 0, 0, 900)
    assert len(set(s.float().tolist())) < 20 < len(set(s.tolist())) < 900
    got, err = run_select(b, bnd, n_select)
    assert err == 0 and torch.equal(got, want)


def test_select_among_equal_scores():
    b = C.batch(10, [1, 1, 3], [16 * 300, 16 * 50 + 2, 16 * 2100], 4, 2, 128, 16, BF16)
    bnd = random_bounds(b, 10)
    bnd[:] = bnd[:1]  # all pages alike
    b.q[1] = 0.0      # a row of padding
    for n_select in (7, 64, 100, 1000):
        got, err = run_select(b, bnd, n_select, 2, 3)
        assert err == 0 and torch.equal(got, S.select(b, bnd, n_select, 2, 3))


def test_select_extremes():
    """Scores beyond fp32's range are compared too, in fp64; NaN has the lowest."""
    b = C.batch(11, [1, 1], [16 * 300, 16 * 200], 4, 2, 64, 16, BF16)
    bnd = random_bounds(b, 11)
    big = bnd.clone()
    big[:200] = (big[:200].float() * 2.0 ** 60).to(BF16)
    b.q *= 2.0 ** 90
    got, err = run_select(b, big, 12)
    assert err == 0 and torch.equal(got, S.select(b, big, 12, 1, 1))
    b.q[:] = float("nan")
    got, err = run_select(b, bnd, 12)
    assert err == 0
    assert got.min() >= 0 and bool((got.diff(dim=-1) > 0).all())


def test_select_with_bad_pages_and_sequences():
    b = C.batch(12, [2, 1, 4], [16 * 90, 16 * 60, 16 * 70], 4, 2, 64, 16, F16)
    bnd = random_bounds(b, 12)
    want = S.select(b, bnd, 10, 1, 1)
    lost = int(want[0, 0, 4])
    b.table[0, lost] = -3
    got, err = run_select(b, bnd, 10)
    assert err == 1
    assert lost not in got[0].flatten().tolist()
    assert torch.equal(got[2:], want[2:])
    b.ctx[1] = -1
    got, err = run_select(b, bnd, 10)
    assert err == 1 and bool((got[2] == -7).all()) and torch.equal(got[3:], want[3:])


def test_select_in_parts_of_a_large_batch():
    """More rows than one launch's scores hold (2^28 bytes): 2 heads, 16384 table entries, 1024 rows."""
    n = 1100
    b = C.batch(13, [n], [16 * 40], 2, 2, 64, 16, BF16)
    wide = torch.zeros((1, 16384), dtype=torch.int32, device="cuda")
    wide[:, :b.table.shape[1]] = b.table
    want_table, b.table = b.table, wide
    bnd = random_bounds(b, 13)
    got, err = run_select(b, bnd, 8)
    b.table = want_table
    want = S.select(C.Batch(b.k.cpu(), b.v.cpu(), b.q.cpu(), b.cu.cpu(), b.ctx.cpu(), b.table.cpu(), b.lens,
                            b.ctxs), bnd.cpu(), 8, 1, 1)
    assert err == 0 and torch.equal(got, want)


def test_captured():
    b = C.batch(14, [1, 1, 1], [700, 900, 3], 4, 2, 64, 16, BF16)
    before = random_bounds(b, 14)
    cache = Bn.KvCache(b.k, b.v)
    bnd = before.clone()
    def step():
        Bn.page_bounds(cache, bnd, b.cu, b.ctx, b.table, n_rows=3)
        return Bn.select_pages(cache, bnd, b.q, b.cu, b.ctx, b.table, 6)
    g = torch.cuda.CUDAGraph()
    step()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        out = step()
    bnd.copy_(before)
    # a token later, with other keys
    b.ctx += 1
    b.ctxs = [c + 1 for c in b.ctxs]
    for i, c in enumerate(b.ctxs):
        b.k[int(b.table[i, c // 16]), :, c % 16] = 3.0
    g.replay()
    torch.cuda.synchronize()
    want = S.bounds(b, before)
    assert torch.equal(bnd, want)
    assert torch.equal(out.cpu(), S.select(b, want, 6, 1, 1))


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("D", [64, 128])
def test_select_for_chunks_of_odd_kinds(dtype, D):
    """Rows in tiles of 16 that two sequences share: large, tiny, zero and tied ones side by side."""
    b = C.batch(15 + D, [21, 9, 40], [16 * 150, 16 * 90 + 3, 16 * 300], 12, 2, D, 16, dtype)
    bnd = random_bounds(b, 15)
    bnd[b.table[2, 40:200].long()] = bnd[b.table[2, 40:41].long()]  # pages alike
    b.q[3] *= 2.0 ** 12
    b.q[4] *= 2.0 ** -14
    b.q[5] = 0.0
    b.q[22:25] = b.q[22]
    for n_select in (5, 60):
        got, err = run_select(b, bnd, n_select, 1, 2)
        assert err == 0 and torch.equal(got, S.select(b, bnd, n_select, 1, 2))
    if dtype == BF16:
        b.q[6] *= 2.0 ** 120  # sums and scores beyond fp32
        got, err = run_select(b, bnd, 9, 1, 2)
        assert err == 0 and torch.equal(got, S.select(b, bnd, 9, 1, 2))


def test_select_beyond_fp32_for_chunks():
    b = C.batch(16, [8], [16 * 900], 2, 1, 64, 16, BF16)
    b.q[:] = torch.tensor([1.0, -1.0], device="cuda")[None, :, None].to(BF16) * 2.0 ** -6
    b.q[:, :, 0] = 1024.0
    gen = torch.Generator().manual_seed(9)
    bnd = torch.randint(-3, 4, shape(b), generator=gen).sort(2).values.to(BF16).cuda() / 16
    bnd[..., 0] = 512.0
    for n_select in (12, 500):
        got, err = run_select(b, bnd, n_select)
        assert err == 0 and torch.equal(got, S.select(b, bnd, n_select, 1, 1))
