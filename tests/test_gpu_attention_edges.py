"""Attention where its kernels can go wrong: references that the scores outgrow, rows that share a warp
with others, queries that are not finite, weights far below the largest."""
import pytest
import torch

from quantized_moe_expert_dequant_gb300 import binding as Bn
from tests import attention_cases as C
from tests.test_gpu_attention import mask_tensor, run_prompt, run_tree, tree_masks

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16


def differing(a, b):
    """The number of elements whose bytes differ."""
    return int((a.view(torch.int16) != b.view(torch.int16)).sum())


def positions(b, i):
    """(page, place in it) of the positions of sequence i."""
    at = torch.arange(b.lens[i] + b.ctxs[i], device=b.k.device)
    page = b.k.shape[2]
    return b.table[i, at // page].long(), at % page


@pytest.mark.parametrize("kind", ["tree", "prompt"])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("D", [64, 128])
def test_scores_that_outgrow_their_reference_in_every_step(kind, dtype, D):
    """Scores rise by about 16 every 128 positions, so each step's weights are formed twice, first
    relative to a reference that they exceed by a factor of e^16 (infinite in fp16)."""
    lens, ctxs = [60, 33], [900, 400]
    b = C.batch(D, lens, ctxs, 8, 2, D, 32, dtype, q_scale=0.2)
    b.q[..., 0] = 4.0
    for i in range(2):
        pages, place = positions(b, i)
        ramp = torch.arange(len(pages), device="cuda") / 32.0
        b.k[pages, :, place, 0] = ramp[:, None].to(dtype)
    masks = tree_masks(D, lens)
    ref, tol = b.reference(1.0, masks if kind == "tree" else None)
    run = (lambda: run_tree(b, 60, masks, 1.0)) if kind == "tree" else (lambda: run_prompt(b, 1.0))
    out = run()
    C.assert_within(out, ref, tol)
    for _ in range(5):
        assert differing(run(), out) == 0


@pytest.mark.parametrize("group,max_q", [(1, 1), (3, 5), (7, 1), (16, 1), (5, 4), (11, 2), (16, 2)])
@pytest.mark.parametrize("D", [64, 128])
def test_clusters_whose_warps_split(group, max_q, D):
    """A cluster an item with rows that leave lanes of a warp without work in the join, and CTAs without
    tiles beside those that have some."""
    lens, ctxs = [max_q, 1, max_q], [5, 64 * 7, 129]
    b = C.batch(group * D, lens, ctxs, group, 1, D, 16, BF16)
    masks = tree_masks(group, lens)
    ref, tol = b.reference(D ** -0.5, masks)
    out = run_tree(b, max_q, masks)
    C.assert_within(out, ref, tol)
    for _ in range(5):
        assert differing(run_tree(b, max_q, masks), out) == 0


@pytest.mark.parametrize("Hq,Hkv,D", [(3, 1, 64), (10, 2, 128), (6, 1, 128), (14, 2, 64), (11, 1, 128)])
@pytest.mark.parametrize("ctx", [0, 3000])
def test_rows_that_do_not_fill_their_warps(Hq, Hkv, D, ctx):
    """Groups that do not divide a tile's 128 rows, last tiles of a few rows; items that one CTA has whole
    (short tables) and that several share (long ones)."""
    lens, ctxs = [45, 64, 1, 23], [ctx, 17, 5, 300]
    b = C.batch(Hq * D, lens, ctxs, Hq, Hkv, D, 64, BF16)
    ref, tol = b.reference(D ** -0.5)
    out = run_prompt(b)
    C.assert_within(out, ref, tol)
    assert differing(run_prompt(b), out) == 0
    masks = tree_masks(D, lens)
    ref, tol = b.reference(D ** -0.5, masks)
    out = run_tree(b, 64, masks)
    C.assert_within(out, ref, tol)
    assert differing(run_tree(b, 64, masks), out) == 0


@pytest.mark.parametrize("kind", ["tree", "prompt"])
@pytest.mark.parametrize("D", [64, 128])
def test_waits_that_give_up(kind, D):
    """A limit shorter than the kernel's ordinary waits: at some of them it gives up, with copies and products
    under way or without, reports that in the error word and ends; calls with the usual limit are
    right again.  Nothing is out of order on the device, only out of time."""
    lens, ctxs = [60, 33], [3000, 5000]
    b = C.batch(D, lens, ctxs, 8, 2, D, 32, BF16)
    cache = Bn.KvCache(b.k, b.v)
    ref, tol = b.reference(D ** -0.5)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def call():
        err.zero_()
        if kind == "tree":
            out = Bn.tree_attention(cache, b.q, b.cu, b.ctx, b.table, 60, device_error=err)
        else:
            out = Bn.prompt_attention(cache, b.q, b.cu, b.ctx, b.table, device_error=err)
        torch.cuda.synchronize()
        return out, int(err)

    C.assert_within(call()[0], ref, tol)
    seen = []
    try:
        for cycles in (1, 200, 500, 1000, 1500, 2000, 2500, 3000, 4000, 6000, 10000):
            Bn.debug_attention_wait_cycles(cycles)
            for _ in range(4):
                seen.append(call()[1])
    finally:
        Bn.debug_attention_wait_cycles(0)
    assert set(seen) <= {0, 2} and set(seen[:4]) == {2}, seen
    out, e = call()
    assert e == 0
    C.assert_within(out, ref, tol)


@pytest.mark.parametrize("group", [5, 6, 7, 4])
@pytest.mark.parametrize("kind", ["tree", "prompt"])
@pytest.mark.parametrize("D", [64, 128])
def test_what_other_rows_hold_does_not_show(group, kind, D):
    """The first sequence's bytes do not depend on the queries of the next one, on rows behind the last, on
    what pages hold behind its positions, or on what an earlier call left in shared memory: all of that
    is in the tiles beside its rows.  Its scores' maximum moves from step to step, so that a vote of
    other rows for a new reference would change how its weights are rounded."""
    lens, ctxs = [20, 3], [1100, 60]
    masks = tree_masks(3, lens) + [0] * 40
    want = None
    for junk in (0.0, 50.0, -50.0, 400.0):
        b = C.batch(group, lens, ctxs, 2 * group, 2, D, 64, BF16, pad_rows=40, stale=junk)
        b.q[20:23] *= max(1.0, junk)
        b.q[23:] = junk
        fill = C.batch(99, [64, 64], [1500, 10], 2 * group, 2, D, 64, BF16)
        fill.q.mul_(1 + abs(junk))
        run_prompt(fill)                     # leaves its queries in shared memory
        run_tree(fill, 64)
        if kind == "tree":
            out = run_tree(b, 20, masks)
        else:
            out = run_prompt(b)
        if want is None:
            want = out[:20].clone()
            ref, tol = b.reference(D ** -0.5, masks if kind == "tree" else None)
            C.assert_within(want, ref[:20], tol[:20])
        assert differing(out[:20], want) == 0, junk


@pytest.mark.parametrize("kind,lens", [("tree", [2, 1]), ("tree", [60, 33]), ("prompt", [60, 33])])
@pytest.mark.parametrize("ctxs", [[40, 7], [9000, 4000]])
@pytest.mark.parametrize("D", [64, 128])
def test_a_query_that_is_nan_gives_nan(kind, lens, ctxs, D):
    """... in its own row and head and nowhere else, whether one CTA has its item or several share it."""
    b = C.batch(D, lens, ctxs, 8, 2, D, 32, BF16)
    ref, tol = b.reference(D ** -0.5)
    rows = [(1, 3), (lens[0], 0), (lens[0], 7)]
    bad = torch.zeros(ref.shape, dtype=torch.bool, device="cuda")
    for r, h in rows:
        b.q[r, h, 5] = float("nan")
        bad[r, h] = True
    out = run_prompt(b) if kind == "prompt" else run_tree(b, max(lens))
    assert bool(out[bad].isnan().all())
    C.assert_within(out[~bad], ref[~bad], tol[~bad])


@pytest.mark.parametrize("kind,max_q,wide", [("tree", 2, False), ("tree", 2, True), ("tree", 60, False),
                                             ("tree", 60, True), ("prompt", 60, False),
                                             ("prompt", 60, True)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("gap", [12.0, 17.0, 18.0, 22.0])
@pytest.mark.parametrize("at", [0, 290])
def test_small_weights_of_fp16_caches_are_kept(kind, max_q, wide, D, gap, at):
    """One position of each sequence outweighs every other one by about e^gap and has the value zero, so
    the output is what the small weights bring: they are not lost in the range of fp16.  The kernels form
    weights times 2^15 (trees of up to 32 rows) or 2^8 (tiles, beside a position that stands out so),
    a weight of 1 being in the divisor, so that half of fp16's least step is 2^-40 or 2^-33 of it."""
    lens, ctxs = [max_q, 33 if max_q > 33 else 1], [1000, 300]
    b = C.batch(D, lens, ctxs, 8, 2, D, 32, F16, q_scale=0.1)
    b.q[..., 0] = 4.0
    b.v.copy_(256 + 50 * b.v)
    for i in range(2):
        pages, place = positions(b, i)
        b.k[pages, :, place, 0] = 0.0
        b.k[pages[at], :, place[at]] = 0.0
        b.k[pages[at], :, place[at], 0] = gap / 4.0
        b.v[pages[at], :, place[at]] = 0.0
    if wide:                                 # several CTAs share an item
        b.table = torch.cat([b.table, torch.full((2, 4000), -1, dtype=torch.int32, device="cuda")], 1)
    least = 2.0 ** -40 if max_q == 2 else 2.0 ** -33
    ref, tol = b.reference(1.0, least=least)
    out = run_prompt(b, 1.0) if kind == "prompt" else run_tree(b, max_q, None, 1.0)
    C.assert_within(out, ref, tol)


def test_equal_weights_of_fp16_caches():
    """All scores alike over many steps, so that all weights are the same power of two and none is rounded;
    and the same with values as large as fp16 holds."""
    for value in (1.0, 60000.0):
        b = C.batch(5, [60, 2], [2000, 700], 8, 2, 128, 32, F16)
        b.q.fill_(0.0)
        b.v.copy_(value * b.v.clamp(-1, 1))
        ref, tol = b.reference(1.0, least=0.0)
        C.assert_within(run_prompt(b, 1.0), ref, tol)
        C.assert_within(run_tree(b, 60, None, 1.0), ref, tol)
        two = C.Batch(b.k, b.v, b.q[60:], torch.tensor([0, 2], dtype=torch.int32, device="cuda"),
                      b.ctx[1:], b.table[1:], [2], [700])
        C.assert_within(run_tree(two, 2, None, 1.0), ref[60:], tol[60:])


@pytest.mark.parametrize("token_major", [False, True])
def test_a_cache_beyond_32_bits(token_major):
    """Pages whose elements lie beyond 2^32 of the cache's first: written, and read by both attentions."""
    Hq, Hkv, D, page = 8, 4, 128, 64
    n_pages = 2 ** 32 // (Hkv * D * page) + 40
    shape = (n_pages, page, Hkv, D) if token_major else (n_pages, Hkv, page, D)
    k, v = (torch.empty(shape, dtype=BF16, device="cuda") for _ in range(2))
    k[:40], v[:40] = 7.0, 7.0                # where an offset of 32 bits would end up
    if token_major:
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    cache = Bn.KvCache(k, v)
    n, gen = 300, torch.Generator().manual_seed(1)
    order = (torch.randperm(40, generator=gen)[:5] + n_pages - 40).to(torch.int32)
    at = torch.arange(n)
    slots = (order[at // page] * page + at % page).to(torch.int32).cuda()
    x = torch.randn((n, Hq + 2 * Hkv, D), generator=gen).to(BF16).cuda()
    q = Bn.qk_norm_rope(cache, x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], at.int().cuda(), slots,
                        None)
    assert torch.equal(k[order.long().cuda()[at.cuda() // page], :, at.cuda() % page],
                       x[:, Hq:Hq + Hkv])
    assert bool((k[:40] == 7).all() and (v[:40] == 7).all())
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")
    table = order.view(1, 5).cuda()
    b = C.Batch(k, v, q, i32(0, n), i32(0), table, [n], [0])
    ref, tol = b.reference(D ** -0.5)
    C.assert_within(run_prompt(b), ref, tol)
    for last in (2, 40):                     # rows of a tree: both kinds of tiles
        b = C.Batch(k, v, q[n - last:], i32(0, last), i32(n - last), table, [last], [n - last])
        C.assert_within(run_tree(b, last), ref[n - last:], tol[n - last:])
