"""Rows before the first sequence, strided tables, caches beyond 32 bits and offsets that do not fit together, for the
calls that do not read the whole cache."""
import pytest
import torch

from quantized_moe_expert_dequant_gb300 import binding as Bn
from tests import attention_cases as C
from tests import sparse_cases as S
from tests.test_gpu_pages import random_bounds
from tests.test_gpu_prefix import Groups

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16
i32 = dict(dtype=torch.int32, device="cuda")


def padded(b, before):
    """q with rows before the first sequence's, offsets and a table with a stride of its own."""
    q = torch.cat([torch.full((before, *b.q.shape[1:]), float("nan"), dtype=b.q.dtype, device="cuda"), b.q])
    wide = torch.full((b.table.shape[0], b.table.shape[1] + 5), 99999, **i32)
    wide[:, :b.table.shape[1]] = b.table
    return q, b.cu + before, wide[:, :b.table.shape[1]]


@pytest.mark.parametrize("lens", [[1] * 9, [1, 3, 0, 20, 1, 1, 2, 0, 40]])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_rows_before_the_first_sequence(lens, dtype):
    ctxs = [(i * 211) % 900 for i in range(9)]
    b = C.batch(1 + len(set(lens)), lens, ctxs, 8, 2, 64, 16, dtype)
    q, cu, table = padded(b, 3)
    cache, err, rows = Bn.KvCache(b.k, b.v), torch.zeros(1, **i32), sum(lens)
    before = random_bounds(b, 2)
    bnd = Bn.page_bounds(cache, before.clone(), cu, b.ctx, table, n_rows=rows + 3, device_error=err)
    assert torch.equal(bnd, S.bounds(b, before))
    out = torch.full((rows + 3, 2, 9), -7, **i32)
    Bn.select_pages(cache, bnd, q, cu, b.ctx, table, 9, 1, 2, out=out, device_error=err)
    assert torch.equal(out[3:].cpu(), S.select(b, bnd, 9, 1, 2)) and bool((out[:3] == -7).all())
    pages = out[3:].contiguous()
    got = torch.full_like(q, 7.0)
    Bn.sparse_attention(cache, q, cu, b.ctx, table, out, 0.2, out=got, device_error=err)
    ref, tol = S.attention(b, pages, 0.2)
    C.assert_within(got[3:], ref, tol)
    assert bool((got[:3] == 7).all())
    got.fill_(7.0)
    for max_q in (64, max(lens)):
        Bn.prefix_attention(cache, q, cu, b.ctx, table, torch.tensor([0, 9], **i32),
                            torch.tensor([0], **i32), max_q, scale=0.2, out=got, device_error=err)
        ref, tol = b.reference(0.2)
        C.assert_within(got[3:], ref, tol)
        assert bool((got[:3] == 7).all())
    assert int(err) == 0


@pytest.mark.parametrize("token_major", [False, True])
def test_a_cache_beyond_32_bits(token_major):
    Hq, Hkv, D, page = 8, 4, 128, 64
    n_pages = 2 ** 32 // (Hkv * D * page) + 40
    shape = (n_pages, page, Hkv, D) if token_major else (n_pages, Hkv, page, D)
    k, v = (torch.empty(shape, dtype=BF16, device="cuda") for _ in range(2))
    k[:40], v[:40] = 7.0, 7.0                # where an offset of 32 bits would end up
    if token_major:
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    gen = torch.Generator().manual_seed(1)
    table = (torch.randperm(40, generator=gen)[:20] + n_pages - 40).to(torch.int32).view(2, 10)
    for t in table.flatten().tolist():
        k[t] = torch.randn((Hkv, page, D), generator=gen).to(BF16).cuda()
        v[t] = torch.randn((Hkv, page, D), generator=gen).to(BF16).cuda()
    q = torch.randn((2, Hq, D), generator=gen).to(BF16).cuda()
    b = C.Batch(k, v, q, torch.tensor([0, 1, 2], **i32), torch.tensor([600, 500], **i32), table.cuda(),
                [1, 1], [600, 500])
    cache = Bn.KvCache(k, v)
    bnd = torch.zeros((n_pages, Hkv, 2, D), dtype=BF16, device="cuda")
    zero = torch.zeros(2, **i32)
    Bn.page_bounds(cache, bnd, torch.tensor([0, 601, 1102], **i32), zero, b.table, n_rows=1102)
    whole = C.Batch(k, v, q, b.cu, zero, b.table, [601, 501], [0, 0])
    want = S.bounds(whole, torch.zeros_like(bnd))
    assert torch.equal(bnd, want)
    pages = Bn.select_pages(cache, bnd, q, b.cu, b.ctx, b.table, 5)
    assert torch.equal(pages.cpu(), S.select(b, bnd, 5, 1, 1))
    ref, tol = S.attention(b, pages, 0.1)
    C.assert_within(Bn.sparse_attention(cache, q, b.cu, b.ctx, b.table, pages, 0.1), ref, tol)
    b.table[1, :6] = b.table[0, :6]
    ref, tol = b.reference(0.1)
    for max_q in (1, 64):                    # clusters and tiles
        got = Bn.prefix_attention(cache, q, b.cu, b.ctx, b.table, torch.tensor([0, 2], **i32),
                                  torch.tensor([384], **i32), max_q, scale=0.1)
        C.assert_within(got, ref, tol)


@pytest.mark.parametrize("max_q", [2, 64])
def test_offsets_out_of_range_at_a_groups_end(max_q):
    """The group's sequences may be refused with it; other groups, and rows of no valid sequence, do not notice."""
    G = Groups(3, [0, 3, 5, 7], [64, 96, 48], [1, 2, 1, 1, 1, 2, 1], [10, 20, 30, 40, 50, 5, 60], 4, 2, 64, 16,
               BF16)
    b, table = G.b, G.b.table.clone()
    ref, tol = b.reference(0.2)
    good = b.cu.clone()
    for bad in (10 ** 6, -5):
        b.cu[7] = bad                        # the end of the last group
        out = torch.full_like(b.q, 7.0)
        got = G.run(max_q, None, 0.2, want_err=1, table=table, out=out)
        C.assert_within(got[:6], ref[:6], tol[:6])
        written = got[6:8]                   # the group's first sequence: right or left alone
        if not bool((written == 7).all()):
            C.assert_within(written, ref[6:8], tol[6:8])
        assert bool((got[8:] == 7).all())
        b.cu.copy_(good)


def test_groups_whose_pages_are_read_by_two_calls_at_once():
    """Two batches over one cache, on two streams, with workspaces of their own."""
    A = Groups(5, [0, 30], [2000], [1] * 30, [i * 7 for i in range(30)], 8, 2, 128, 64, BF16)
    b = A.b
    cache = Bn.KvCache(b.k, b.v)
    want = A.run(64)
    args = (cache, b.q, b.cu, b.ctx, A.hidden, torch.tensor([0, 30], **i32), torch.tensor([2000], **i32), 64)
    streams, outs = [torch.cuda.Stream(), torch.cuda.Stream()], []
    torch.cuda.synchronize()
    for _ in range(10):
        for s in streams:
            with torch.cuda.stream(s):
                outs.append(Bn.prefix_attention(*args))
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, want)
