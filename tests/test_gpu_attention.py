"""Attention over the pages of a cache against the formula in fp64: trees of drafted tokens and
single tokens (moe_tree_attention), prompts (moe_prompt_attention)."""
import pytest
import torch

from quantized_moe_expert_dequant_gb300 import binding as Bn
from tests import attention_cases as C

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16


def tree_masks(seed, lens, ancestors=True):
    """One int per row: bit j set when the row sees drafted token j."""
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda lo, hi: int(torch.randint(lo, hi + 1, (1,), generator=gen))
    masks = []
    for n in lens:
        rows = []
        for j in range(n):
            if ancestors:
                up = rnd(max(-1, j - 5), j - 1) if j else -1
                rows.append((rows[up] if up >= 0 else 0) | 1 << j)
            else:
                rows.append(rnd(0, 2 ** 62) & ((1 << n) - 1))
        masks += rows
    return masks


def mask_tensor(masks):
    return torch.tensor([m - (1 << 64) if m >> 63 else m for m in masks], dtype=torch.int64,
                        device="cuda")


def run_tree(b, max_q, masks=None, scale=None, **kw):
    cache = Bn.KvCache(b.k, b.v)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = Bn.tree_attention(cache, b.q, b.cu, b.ctx, b.table, max_q,
                            None if masks is None else mask_tensor(masks), scale,
                            device_error=err, **kw)
    torch.cuda.synchronize()
    assert int(err) == 0
    return out


def run_prompt(b, scale=None, **kw):
    cache = Bn.KvCache(b.k, b.v)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = Bn.prompt_attention(cache, b.q, b.cu, b.ctx, b.table, scale, device_error=err, **kw)
    torch.cuda.synchronize()
    assert int(err) == 0
    return out


HEADS = [(8, 8, 64), (8, 2, 128), (6, 1, 64), (5, 1, 128), (24, 3, 128), (14, 2, 64)]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("page", [16, 64, 256])
def test_single_tokens(dtype, Hq, Hkv, D, page):
    ctxs = [0, 1, 15, 16, 62, 63, 64, 65, 127, 300, 1000, 2049]
    b = C.batch(Hq + D + page, [1] * len(ctxs), ctxs, Hq, Hkv, D, page, dtype)
    ref, tol = b.reference(D ** -0.5)
    C.assert_within(run_tree(b, 1), ref, tol)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("ancestors", [True, False])
def test_trees(dtype, Hq, Hkv, D, ancestors):
    lens = [1, 64, 0, 3, 17, 33, 48, 2]
    ctxs = [100, 0, 50, 63, 64, 1000, 13, 0]
    b = C.batch(Hq * D, lens, ctxs, Hq, Hkv, D, 32, dtype)
    masks = tree_masks(D + Hq, lens, ancestors)
    ref, tol = b.reference(0.11, masks)
    C.assert_within(run_tree(b, 64, masks, 0.11), ref, tol)


@pytest.mark.parametrize("max_q", [1, 2, 3, 4, 5, 8, 9, 16, 31])
@pytest.mark.parametrize("Hq,Hkv", [(4, 4), (8, 2), (7, 1)])
def test_tree_of_every_height(max_q, Hq, Hkv):
    lens = [max_q, 1, max_q, max(1, max_q - 1)]
    b = C.batch(max_q, lens, [513, 70, 0, 190], Hq, Hkv, 128, 16, BF16)
    masks = tree_masks(max_q, lens)
    ref, tol = b.reference(128 ** -0.5, masks)
    C.assert_within(run_tree(b, max_q, masks), ref, tol)
    ref, tol = b.reference(128 ** -0.5)
    C.assert_within(run_tree(b, max_q), ref, tol)


@pytest.mark.parametrize("Hq,Hkv", [(32, 8), (12, 2)])
def test_long_contexts(Hq, Hkv):
    lens, ctxs = [5, 1, 1], [70001, 4096, 33]
    b = C.batch(3, lens, ctxs, Hq, Hkv, 128, 64, BF16)
    masks = tree_masks(4, lens)
    ref, tol = b.reference(128 ** -0.5, masks)
    C.assert_within(run_tree(b, 5, masks), ref, tol)


def test_many_short_sequences():
    gen = torch.Generator().manual_seed(8)
    n = 700
    lens = torch.randint(0, 4, (n,), generator=gen).tolist()
    ctxs = torch.randint(0, 90, (n,), generator=gen).tolist()
    b = C.batch(5, lens, ctxs, 4, 2, 64, 16, F16)
    masks = tree_masks(4, lens)
    ref, tol = b.reference(0.125, masks)
    C.assert_within(run_tree(b, 3, masks), ref, tol)


@pytest.mark.parametrize("Hq,Hkv,D", [(8, 1, 128), (16, 2, 64), (9, 3, 128)])
def test_large_trees_behind_long_contexts(Hq, Hkv, D):
    """Items whose positions several CTAs share, drafts across a step's border, empty rows."""
    lens, ctxs = [64, 33, 5, 64, 64], [20010, 5120, 127, 0, 5100]
    b = C.batch(Hq + D, lens, ctxs, Hq, Hkv, D, 64, F16)
    masks = tree_masks(D, lens, False)
    masks[3] = masks[70] = masks[110] = 0   # the last one has no context either
    ref, tol = b.reference(D ** -0.5, masks)
    out = run_tree(b, 64, masks)
    C.assert_within(out, ref, tol)
    assert not bool(out[110].any()) and bool(out[70].any())


@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 128), (4, 4, 64), (6, 1, 128)])
def test_prompts_that_many_ctas_share(Hq, Hkv, D):
    lens, ctxs = [700, 1, 3, 130, 0, 2100], [9000, 12345, 0, 1023, 8000, 0]
    b = C.batch(Hq * D, lens, ctxs, Hq, Hkv, D, 128, BF16)
    ref, tol = b.reference(D ** -0.5)
    C.assert_within(run_prompt(b), ref, tol)


@pytest.mark.parametrize("group", [33, 40, 64])
@pytest.mark.parametrize("D", [64, 128])
def test_many_query_heads_on_one(group, D):
    lens, ctxs = [1, 30, 5], [77, 0, 1300]
    b = C.batch(group + D, lens, ctxs, group, 1, D, 16, BF16)
    ref, tol = b.reference(D ** -0.5)
    C.assert_within(run_prompt(b), ref, tol)
    C.assert_within(run_tree(b, 30), ref, tol)
    masks = tree_masks(group, lens, False)
    ref, tol = b.reference(D ** -0.5, masks)
    C.assert_within(run_tree(b, 30, masks), ref, tol)


@pytest.mark.parametrize("kind,max_q", [("tree", 2), ("tree", 30), ("prompt", 0)])
def test_rows_before_the_first_sequence_stay(kind, max_q):
    b = C.batch(81, [2, 30 if max_q != 2 else 1], [40, 3], 4, 2, 64, 16, BF16, pad_rows=5)
    rows = b.q.shape[0] - 5
    ref, tol = b.reference(0.125)
    shifted = torch.cat([torch.full_like(b.q[:5], float("nan")), b.q[:rows]])
    out = torch.full_like(shifted, 5.0)
    moved = C.Batch(b.k, b.v, shifted, b.cu + 5, b.ctx, b.table, b.lens, b.ctxs)
    run_tree(moved, max_q, out=out) if kind == "tree" else run_prompt(moved, out=out)
    C.assert_within(out[5:], ref[:rows], tol[:rows])
    assert bool((out[:5] == 5).all())


def test_many_prompts():
    gen = torch.Generator().manual_seed(9)
    n = 900
    lens = torch.randint(0, 40, (n,), generator=gen).tolist()
    ctxs = [0 if i % 3 else 200 for i in range(n)]
    b = C.batch(6, lens, ctxs, 4, 2, 64, 16, BF16)
    ref, tol = b.reference(0.125)
    C.assert_within(run_prompt(b), ref, tol)


def test_rows_that_see_nothing_are_zeros():
    lens = [4, 1, 2]
    b = C.batch(11, lens, [0, 0, 40], 6, 2, 64, 16, BF16)
    masks = [0, 1, 0, 0b1010, 0, 0, 0b11]
    out = run_tree(b, 4, masks)
    ref, tol = b.reference(0.125, masks)
    C.assert_within(out, ref, tol)
    for r in (0, 2, 4):
        assert not bool(out[r].any())


def test_large_scores_and_equal_scores():
    """Scores hundreds apart, and all the same: the running maximum is what keeps them finite."""
    for scale in (8.0, 1e-6):
        b = C.batch(21, [3, 1], [700, 64], 8, 2, 128, 64, BF16, q_scale=4.0)
        ref, tol = b.reference(scale)
        C.assert_within(run_tree(b, 3, None, scale), ref, tol)
        C.assert_within(run_prompt(b, scale), ref, tol)


def test_rising_scores():
    """Each position outweighs all before it, so the maximum moves in every step."""
    b = C.batch(22, [2, 130], [1500, 0], 4, 1, 64, 64, BF16)
    b.q.fill_(1.0)
    for i in range(2):
        n = b.lens[i] + b.ctxs[i]
        for j in range(-(-n // 64)):
            ramp = torch.arange(64, device="cuda", dtype=torch.float32) + 64 * j
            b.k[b.table[i, j].long(), 0, :, :] = (ramp[:, None] / 64).to(BF16)
    for scale in (0.125, 1.0):
        ref, tol = b.reference(scale)
        C.assert_within(run_prompt(b, scale), ref, tol)
    masks = [3, 3]
    one = C.Batch(b.k, b.v, b.q[:2], b.cu[:2].contiguous(), b.ctx[:1].contiguous(), b.table[:1],
                  [2], [1500])
    ref, tol = one.reference(0.5, masks)
    C.assert_within(run_tree(one, 2, masks, 0.5), ref, tol)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("page", [16, 128])
def test_prompts(dtype, Hq, Hkv, D, page):
    lens = [1, 2, 31, 0, 64, 65, 127, 128, 129, 257, 400]
    b = C.batch(Hq + D, lens, [0] * len(lens), Hq, Hkv, D, page, dtype)
    ref, tol = b.reference(D ** -0.5)
    C.assert_within(run_prompt(b), ref, tol)


@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
def test_chunks_behind_a_prefix(Hq, Hkv, D):
    lens = [1, 63, 0, 128, 200]
    ctxs = [500, 64, 7, 129, 1]
    b = C.batch(Hq + D, lens, ctxs, Hq, Hkv, D, 32, BF16)
    ref, tol = b.reference(D ** -0.5)
    C.assert_within(run_prompt(b), ref, tol)


def test_a_long_prompt():
    b = C.batch(9, [3001, 17], [0, 5000], 8, 2, 128, 64, BF16)
    ref, tol = b.reference(128 ** -0.5)
    C.assert_within(run_prompt(b), ref, tol)


@pytest.mark.parametrize("kind", ["tree", "prompt"])
def test_strides(kind):
    """Pages of [page, head] order, queries and outputs inside wider rows, a table inside a wider
    one, and the largest page."""
    for page, token_major in ((64, True), (1024, False), (16, True)):
        lens, ctxs = [5, 20, 1], [90, 3, 2000]
        b = C.batch(31, lens, ctxs, 10, 2, 64, page, BF16, token_major=token_major)
        wide = torch.zeros((b.q.shape[0], 16, 96), dtype=BF16, device="cuda")
        wide[:, 3:13, 16:80] = b.q
        b.q = wide[:, 3:13, 16:80]
        big = torch.full((3, b.table.shape[1] + 5), 1 << 30, dtype=torch.int32, device="cuda")
        big[:, :b.table.shape[1]] = b.table
        b.table = big[:, :b.table.shape[1]]
        hold = torch.full((b.q.shape[0], 12, 72), 7.0, dtype=BF16, device="cuda")
        out = hold[:, 1:11, 8:]
        ref, tol = b.reference(0.125)
        run = (lambda: run_tree(b, 20, out=out)) if kind == "tree" else (lambda: run_prompt(b, out=out))
        C.assert_within(run(), ref, tol)
        assert bool((hold[:, 0] == 7).all() and (hold[:, 11] == 7).all() and (hold[..., :8] == 7).all())


@pytest.mark.parametrize("kind", ["tree", "prompt"])
def test_rows_behind_the_last_sequence_stay(kind):
    b = C.batch(41, [3, 2], [30, 0], 4, 2, 128, 16, BF16, pad_rows=6)
    b.q[5:] = float("nan")
    out = torch.full_like(b.q, 5.0)
    run_tree(b, 3, out=out) if kind == "tree" else run_prompt(b, out=out)
    ref, tol = b.reference(128 ** -0.5)
    C.assert_within(out[:5], ref[:5], tol[:5])
    assert bool((out[5:] == 5).all())


@pytest.mark.parametrize("kind", ["tree", "prompt"])
def test_no_rows_or_no_sequences(kind):
    b = C.batch(42, [0, 0], [30, 0], 4, 2, 128, 16, BF16)
    run = (lambda x: run_tree(x, 1)) if kind == "tree" else run_prompt
    assert run(b).shape == (0, 4, 128)
    b = C.batch(42, [2], [30], 4, 2, 128, 16, BF16)
    b.cu, b.ctx, b.table = b.cu[:1].contiguous(), b.ctx[:0], b.table[:0]
    out = torch.full_like(b.q, 5.0)
    (run_tree(b, 1, out=out) if kind == "tree" else run_prompt(b, out=out))
    assert bool((out == 5).all())


@pytest.mark.parametrize("kind", ["tree", "prompt"])
def test_bad_device_data_is_reported(kind):
    """A page outside the cache, and sequences outside their bounds: the error bit, nothing read or
    written there, the other sequences right."""
    lens, ctxs = [2, 3, 2], [100, 40, 7]
    for case in ("page", "negative page", "ctx", "negative ctx", "cu", "too many"):
        b = C.batch(43, lens, ctxs, 4, 2, 64, 16, BF16)
        ref, tol = b.reference(0.125)
        cu, ctx, table = b.cu.clone(), b.ctx.clone(), b.table.clone()
        max_q = 3
        if case == "page":
            table[1, 1] = b.k.shape[0]
        elif case == "negative page":
            table[1, 0] = -5
        elif case == "ctx":
            ctx[1] = 1 << 30
        elif case == "negative ctx":
            ctx[1] = -1
        elif case == "cu":
            cu = torch.tensor([0, 2, 9, 7], dtype=torch.int32, device="cuda")
        else:
            max_q = 2
            if kind == "prompt":
                continue
        out = torch.full_like(b.q, 5.0)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        cache = Bn.KvCache(b.k, b.v)
        if kind == "tree":
            Bn.tree_attention(cache, b.q, cu, ctx, table, max_q, scale=0.125, out=out,
                              device_error=err)
        else:
            Bn.prompt_attention(cache, b.q, cu, ctx, table, 0.125, out=out, device_error=err)
        torch.cuda.synchronize()
        assert int(err) == 1, case
        good = [0, 1] if case == "cu" else [0, 1, 5, 6]
        C.assert_within(out[good], ref[good], tol[good], case)
        if "page" not in case and case != "cu":
            assert bool((out[2:5] == 5).all()), case


@pytest.mark.parametrize("kind", ["tree", "prompt"])
def test_captured_and_replayed(kind):
    """A captured call reads lengths, pages and masks when it is replayed, not when it was taken."""
    first = C.batch(51, [3, 1, 2], [200, 0, 64], 8, 2, 128, 16, BF16, extra_pages=40)
    then = C.batch(52, [1, 3, 2], [17, 300, 65], 8, 2, 128, 16, BF16, extra_pages=40)
    n_pages = max(first.k.shape[0], then.k.shape[0])
    k = torch.zeros((n_pages,) + tuple(first.k.shape[1:]), dtype=BF16, device="cuda")
    v = torch.zeros_like(k)
    table = torch.zeros((3, 30), dtype=torch.int32, device="cuda")
    q, cu, ctx = first.q.clone(), first.cu.clone(), first.ctx.clone()
    mask = torch.zeros(6, dtype=torch.int64, device="cuda")
    out = torch.zeros_like(q)
    cache = Bn.KvCache(k, v)

    def fill(b):
        k[:b.k.shape[0]], v[:b.v.shape[0]] = b.k, b.v
        table.zero_()
        table[:, :b.table.shape[1]] = b.table
        q.copy_(b.q), cu.copy_(b.cu), ctx.copy_(b.ctx)
        masks = tree_masks(7, b.lens)
        mask.copy_(mask_tensor(masks))
        return masks

    def call():
        if kind == "tree":
            Bn.tree_attention(cache, q, cu, ctx, table, 3, mask, out=out)
        else:
            Bn.prompt_attention(cache, q, cu, ctx, table, out=out)

    fill(first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for b in (then, first, then):
        masks = fill(b)
        out.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        ref, tol = b.reference(128 ** -0.5, masks if kind == "tree" else None)
        C.assert_within(out, ref, tol)


@pytest.mark.parametrize("kind", ["tree", "prompt"])
def test_two_streams_and_repeats(kind):
    """Calls at once on two streams, and the same call again, give the same bytes."""
    b = C.batch(61, [4, 1, 60], [3000, 900, 5], 8, 2, 128, 16, BF16)
    cache = Bn.KvCache(b.k, b.v)

    def call(stream=None):
        if kind == "tree":
            return Bn.tree_attention(cache, b.q, b.cu, b.ctx, b.table, 60, stream=stream)
        return Bn.prompt_attention(cache, b.q, b.cu, b.ctx, b.table, stream=stream)

    want = call()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [call(streams[i % 2]) for i in range(20)]
    outs.append(call(streams[0].cuda_stream))
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("kind,max_q", [("tree", 2), ("tree", 40), ("prompt", 0)])
def test_workspaces(kind, max_q):
    """A caller's workspace, filled with anything, does; one that is too small is refused and nothing is
    written."""
    b = C.batch(71, [2, 40 if max_q != 2 else 1], [3000, 900], 8, 2, 128, 16, BF16)
    wide = torch.zeros((2, 4000), dtype=torch.int32, device="cuda")  # too long for clusters
    wide[:, :b.table.shape[1]] = b.table
    b.table = wide
    cache = Bn.KvCache(b.k, b.v)
    out = torch.full_like(b.q, 5.0)

    def call(ws):
        if kind == "tree":
            return Bn.tree_attention(cache, b.q, b.cu, b.ctx, b.table, max_q, workspace=ws, out=out)
        return Bn.prompt_attention(cache, b.q, b.cu, b.ctx, b.table, workspace=ws, out=out)

    for n in (0, 4096):
        with pytest.raises(Bn.MoeError) as e:
            call(torch.zeros(n, dtype=torch.uint8, device="cuda"))
        assert e.value.rc == Bn.MOE_ERR_INVALID_ARG
    torch.cuda.synchronize()
    assert bool((out == 5).all())
    ref, tol = b.reference(128 ** -0.5)
    for fill in (0, 255, 127):
        ws = torch.full((1 << 27,), fill, dtype=torch.uint8, device="cuda")
        C.assert_within(call(ws), ref, tol)
        C.assert_within(call(ws), ref, tol)


@pytest.mark.parametrize("n,Hkv", [(1, 1), (1, 19), (2, 10), (3, 6), (19, 2), (20, 2), (38, 1), (39, 1)])
@pytest.mark.parametrize("D", [64, 128])
def test_few_items(n, Hkv, D):
    """Around the counts of items from which clusters of 16 and of 8 CTAs give way to the shared line;
    sequences shorter than a cluster has tiles, without rows, without context."""
    lens = [1 + i % 3 for i in range(n)]
    ctxs = [(0, 3, 700, 64, 2500)[i % 5] for i in range(n)]
    if n > 2:
        lens[1] = 0
    b = C.batch(n + D, lens, ctxs, 5 * Hkv, Hkv, D, 32, F16 if n % 2 else BF16)
    masks = tree_masks(n, lens)
    ref, tol = b.reference(D ** -0.5, masks)
    C.assert_within(run_tree(b, 3, masks), ref, tol)
    one = run_tree(b, 3, masks)
    assert torch.equal(one.view(torch.int16), run_tree(b, 3, masks).view(torch.int16))


def test_a_table_longer_than_the_sequences():
    """The table's width bounds the lengths; entries that no sequence uses are not read."""
    lens, ctxs = [3, 40], [100, 20]
    b = C.batch(72, lens, ctxs, 4, 2, 64, 16, BF16)
    wide = torch.full((2, 4000), 1 << 30, dtype=torch.int32, device="cuda")
    wide[:, :b.table.shape[1]] = b.table
    b.table = wide
    ref, tol = b.reference(0.125)
    C.assert_within(run_tree(b, 40), ref, tol)
    C.assert_within(run_prompt(b), ref, tol)
