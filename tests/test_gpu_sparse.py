"""Attention over listed pages (moe_sparse_attention) against the formula in fp64."""
import pytest
import torch

from quantized_moe_expert_dequant_gb300 import binding as Bn
from tests import attention_cases as C
from tests import sparse_cases as S

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16


def run(b, pages, scale=None, want_err=0, **kw):
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = Bn.sparse_attention(Bn.KvCache(b.k, b.v), b.q, b.cu, b.ctx, b.table, pages, scale,
                              device_error=err, **kw)
    torch.cuda.synchronize()
    assert int(err) == want_err
    return out


HEADS = [(8, 8, 64), (8, 2, 128), (6, 1, 64), (5, 1, 128), (24, 1, 128), (32, 1, 64), (14, 2, 64)]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("page", [16, 64, 256])
def test_tokens(dtype, Hq, Hkv, D, page):
    # with a few rows clusters take them, with many the shared line
    for n in (1, 3, 40):
        ctxs = [(i * i * 97 + 5 * i) % 2500 for i in range(n)]
        b = C.batch(Hq + D + page + n, [1] * n, ctxs, Hq, Hkv, D, page, dtype,
                    token_major=page == 64)
        pages = S.random_lists(b, 5, n)
        ref, tol = S.attention(b, pages, D ** -0.5)
        C.assert_within(run(b, pages), ref, tol, f"{n} rows")


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 128), (6, 1, 64)])
def test_chunks(dtype, Hq, Hkv, D):
    lens, ctxs = [1, 70, 0, 33, 2], [500, 0, 9, 1000, 31]
    b = C.batch(Hq + D, lens, ctxs, Hq, Hkv, D, 16, dtype, pad_rows=4)
    pages = S.random_lists(b, 9, 1)
    ref, tol = S.attention(b, pages, 0.2)
    out = torch.full_like(b.q, 7.0)
    got = run(b, pages, 0.2, out=out)
    C.assert_within(got[:-4], ref[:-4], tol[:-4])
    assert bool((got[-4:] == 7.0).all())


def test_long_lists():
    b = C.batch(1, [1, 1], [70000, 33000], 8, 2, 128, 64, BF16)
    pages = S.random_lists(b, 700, 2)
    ref, tol = S.attention(b, pages, 0.09)
    C.assert_within(run(b, pages, 0.09), ref, tol)


def test_all_pages_is_causal_attention():
    lens, ctxs = [3, 1, 20], [100, 777, 5]
    b = C.batch(2, lens, ctxs, 8, 2, 128, 16, F16)
    pages = S.random_lists(b, 60, 2)  # more than any row sees: all
    ref, tol = b.reference(0.1)
    C.assert_within(run(b, pages, 0.1), ref, tol)


def test_lists_of_any_kind():
    """Entries in no order, none at all, behind the row's last page, and one page twice."""
    b = C.batch(3, [1, 1, 1, 2], [200, 300, 500, 640], 4, 2, 64, 16, BF16)
    pages = torch.tensor([[[12, 3, -1, 7, 0, 13], [-1, -1, 5, -1, 2, 1]],
                          [[-1] * 6, [18, 17, 16, 2, 1, 0]],
                          [[4, 4, 9, 31, 4, 4], [32, 33, 99999999, 2147483647, -2147483648, 31]],
                          [[0, 40, 39, 1, 2, 3], [40, 40, 40, 40, 40, 40]],
                          [[40, 0, 5, 6, 7, -5], [1, 2, 3, 4, 5, 6]]], dtype=torch.int32,
                         device="cuda")
    ref, tol = S.attention(b, pages, 0.3)
    got = run(b, pages, 0.3)
    C.assert_within(got, ref, tol)
    assert bool((got[1, :2] == 0).all())  # a row that sees nothing


def test_rows_that_share_the_list_entries_of_few_pages():
    # fewer pages than entries: only as many entries as the row has pages are read
    b = C.batch(4, [1], [20], 4, 1, 64, 16, F16)
    pages = torch.tensor([[[1, 0, 1, 1]]], dtype=torch.int32, device="cuda")
    ref, tol = S.attention(b, pages, 0.3)
    C.assert_within(run(b, pages, 0.3), ref, tol)


def test_bad_pages_and_sequences():
    b = C.batch(5, [1, 1, 2], [100, 200, 300], 4, 2, 64, 16, BF16)
    pages = S.random_lists(b, 6, 3)
    ref, tol = S.attention(b, pages, 0.2)
    good = b.table.clone()
    hit = int(pages[0, 0, 2])
    b.table[0, hit] = b.k.shape[0]  # outside the cache: as if it were not listed
    less = pages.clone()
    less[0][less[0] == hit] = -1
    b2 = C.Batch(b.k, b.v, b.q, b.cu, b.ctx, good, b.lens, b.ctxs)
    ref0, tol0 = S.attention(b2, less, 0.2)
    C.assert_within(run(b, pages, 0.2, want_err=1), ref0, tol0)
    b.table = good
    b.ctx[1] = 10 ** 7
    out = torch.full_like(b.q, 7.0)
    got = run(b, pages, 0.2, want_err=1, out=out)
    keep = [0, 2, 3]
    C.assert_within(got[keep], ref[keep], tol[keep])
    assert bool((got[1] == 7.0).all())


@pytest.mark.parametrize("n", [2, 60])
def test_streams_graphs_and_workspaces(n):
    b = C.batch(6, [1] * n, [(37 * i) % 900 for i in range(n)], 8, 2, 128, 16, BF16)
    pages = S.random_lists(b, 7, 4)
    want = run(b, pages)
    assert torch.equal(run(b, pages), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert torch.equal(run(b, pages, stream=side), want)
    cache = Bn.KvCache(b.k, b.v)
    g, out = torch.cuda.CUDAGraph(), torch.zeros_like(b.q)
    ws = torch.full((1 << 24,), 255, dtype=torch.uint8, device="cuda")  # anything may be in it
    with torch.cuda.graph(g):
        Bn.sparse_attention(cache, b.q, b.cu, b.ctx, b.table, pages, out=out, workspace=ws)
    for _ in range(2):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_strided_queries():
    b = C.batch(7, [1, 3], [100, 50], 6, 2, 64, 16, F16)
    pages = S.random_lists(b, 4, 5)
    ref, tol = S.attention(b, pages, 0.2)
    wide = torch.full((4, 10, 72), float("nan"), dtype=F16, device="cuda")
    wide[:, 2:8, :64] = b.q
    b.q = wide[:, 2:8, :64]
    out = torch.full((4, 8, 64), 3.0, dtype=F16, device="cuda")
    got = run(b, pages, 0.2, out=out[:, 1:7])
    C.assert_within(got, ref, tol)
    assert bool((out[:, 0] == 3).all()) and bool((out[:, 7] == 3).all())


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_a_decode_step(dtype):
    """A step of a layer: keys and values written, bounds kept up, pages selected, attention over them;
    while the selection takes all pages, the result is that of dense attention."""
    Hq, Hkv, D, page, n = 8, 2, 64, 16, 4
    ctxs = [5, 100, 333, 1000]
    b = C.batch(8, [1] * n, ctxs, Hq, Hkv, D, page, dtype, stale=0.0)
    cache = Bn.KvCache(b.k, b.v)
    bnd = torch.zeros((b.k.shape[0], Hkv, 2, D), dtype=dtype, device="cuda")
    zero = torch.zeros_like(b.ctx)
    # the contexts, as prompts: everything before the tokens' pages
    prompt = C.Batch(b.k, b.v, b.q, torch.tensor([0] + torch.tensor(ctxs).cumsum(0).tolist(),
                                                 dtype=torch.int32, device="cuda"), zero, b.table, ctxs,
                     [0] * n)
    Bn.page_bounds(cache, bnd, prompt.cu, zero, b.table, n_rows=sum(ctxs))
    gen = torch.Generator().manual_seed(3)
    qkv = [(torch.randn((n, h, D), generator=gen)).to(dtype).cuda() for h in (Hq, Hkv, Hkv)]
    pos = b.ctx.clone()
    slots = torch.stack([b.table[i, c // page] * page + c % page for i, c in enumerate(ctxs)])
    inv = 1e4 ** (-torch.arange(0, D, 2, device="cuda", dtype=torch.float64) / D)
    q = Bn.qk_norm_rope(cache, *qkv, pos, slots.to(torch.int32), inv)
    Bn.page_bounds(cache, bnd, b.cu, b.ctx, b.table, n_rows=n)
    b.q = q
    used = S.bounds(prompt, torch.zeros_like(bnd))
    used = S.bounds(b, used)
    assert torch.equal(bnd, used)
    for k in (8, 64):
        pages = Bn.select_pages(cache, bnd, q, b.cu, b.ctx, b.table, k, sink=1, recent=2)
        assert torch.equal(pages.cpu(), S.select(b, used, k, 1, 2))
        got = Bn.sparse_attention(cache, q, b.cu, b.ctx, b.table, pages)
        ref, tol = S.attention(b, pages, D ** -0.5)
        C.assert_within(got, ref, tol)
        if k == 64:
            ref, tol = b.reference(D ** -0.5)
            C.assert_within(got, ref, tol)
