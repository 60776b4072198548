"""Attention of sequences that share their first pages (moe_prefix_attention) against the formula in fp64."""
import pytest
import torch

from quantized_moe_expert_dequant_gb300 import binding as Bn
from tests import attention_cases as C
from tests.test_gpu_attention import mask_tensor, tree_masks

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16


class Groups:
    """A batch in which sequences cu[g] .. cu[g + 1] - 1 share the pages of prefix[g] positions.  What the
    others' rows of the table name there is no page at all: nothing may be read by them."""

    def __init__(self, seed, cu, prefix, lens, after, Hq, Hkv, D, page, dtype, **kw):
        self.cu, self.prefix = cu, prefix
        ctxs = list(after)
        for g, p in enumerate(prefix):
            for i in range(cu[g], cu[g + 1]):
                ctxs[i] += p
        self.b = b = C.batch(seed, lens, ctxs, Hq, Hkv, D, page, dtype, **kw)
        self.hidden = b.table.clone()  # the table that the call gets
        for g, p in enumerate(prefix):
            n = p // page
            for i in range(cu[g] + 1, cu[g + 1]):
                b.table[i, :n] = b.table[cu[g], :n]
                self.hidden[i, :n] = -9

    def run(self, max_q, masks=None, scale=None, want_err=0, table=None, **kw):
        b = self.b
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        i32 = dict(dtype=torch.int32, device="cuda")
        out = Bn.prefix_attention(
            Bn.KvCache(b.k, b.v), b.q, b.cu, b.ctx, self.hidden if table is None else table,
            torch.tensor(self.cu, **i32), torch.tensor(self.prefix, **i32), max_q,
            None if masks is None else mask_tensor(masks), scale, device_error=err, **kw)
        torch.cuda.synchronize()
        assert int(err) == want_err
        return out


HEADS = [(8, 8, 64), (8, 2, 128), (6, 1, 64), (5, 1, 128), (24, 3, 128), (64, 1, 64)]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("page", [16, 64, 256])
def test_single_tokens(dtype, Hq, Hkv, D, page):
    # two groups, one sequence before them, two behind; a prefix that ends inside a page
    n = 14
    after = [(i * 53) % 300 for i in range(n)]
    G = Groups(Hq + D + page, [1, 8, 12], [1500, 777], [1] * n, after, Hq, Hkv, D, page, dtype)
    ref, tol = G.b.reference(D ** -0.5)
    C.assert_within(G.run(1), ref, tol)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
def test_single_tokens_on_the_tiles(dtype, Hq, Hkv, D):
    """The same with room for more tokens a sequence, and more rows than the other forms take."""
    n = 14
    after = [(i * 53) % 300 for i in range(n)]
    G = Groups(Hq + D, [1, 8, 12], [1500, 777], [1] * n, after, Hq, Hkv, D, 64, dtype)
    ref, tol = G.b.reference(D ** -0.5)
    C.assert_within(G.run(64), ref, tol)
    short = Groups(Hq + D, [0, 5, 14], [130, 64], [1] * n, after, Hq, Hkv, D, 64, dtype)
    ref, tol = short.b.reference(D ** -0.5)
    C.assert_within(short.run(64), ref, tol)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("Hq,Hkv,D,n", [(8, 2, 128, 90), (6, 1, 64, 150), (16, 16, 64, 20)])
def test_many_short_sequences(dtype, Hq, Hkv, D, n):
    """All CTAs share the items of many sequences; groups of one and of none, sequences without rows."""
    lens = [(i * 7 + 3) % 4 for i in range(n)]
    cu = [0, 1, 1, n // 3, n // 2, n - 2]
    G = Groups(Hq + n, cu, [48, 100, 333, 64, 16], lens, [(i * 31) % 150 for i in range(n)], Hq, Hkv, D, 16,
               dtype)
    masks = tree_masks(n, lens)
    ref, tol = G.b.reference(0.2, masks)
    C.assert_within(G.run(3, masks, 0.2), ref, tol)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("ancestors", [True, False])
def test_trees(dtype, Hq, Hkv, D, ancestors):
    lens = [1, 64, 0, 3, 17, 33, 48, 2, 0]
    after = [100, 0, 50, 63, 64, 300, 13, 0, 0]
    G = Groups(Hq * D, [0, 3, 4, 9], [320, 1000, 64], lens, after, Hq, Hkv, D, 32, dtype)
    masks = tree_masks(D + Hq, lens, ancestors)
    ref, tol = G.b.reference(0.11, masks)
    C.assert_within(G.run(64, masks, 0.11), ref, tol)
    ref, tol = G.b.reference(0.11)
    C.assert_within(G.run(64, None, 0.11), ref, tol)  # causal without masks


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_long_prefixes_in_many_parts(dtype):
    G = Groups(5, [0, 6], [30000], [1, 2, 1, 4, 1, 8], [0, 5, 1000, 64, 3, 9], 8, 2, 128, 64, dtype)
    ref, tol = G.b.reference(0.09)
    C.assert_within(G.run(8, None, 0.09), ref, tol)


def test_many_sequences_and_rows():
    n = 600  # more rows than a tile pair has, more sequences than a block has threads
    G = Groups(6, [0, 400, 401, 600], [256, 0, 48], [1 + i % 2 for i in range(n)],
               [(i * 7) % 40 for i in range(n)], 4, 1, 64, 16, BF16)
    ref, tol = G.b.reference(0.2)
    C.assert_within(G.run(2, None, 0.2), ref, tol)


def test_prefixes_of_no_use():
    """Shorter than a page, none, longer than a sequence's context: those are computed by themselves."""
    G = Groups(7, [0, 2, 4, 6], [15, 0, 64], [1, 2, 1, 1, 1, 1], [20, 30, 40, 50, 60, 70], 4, 2, 64,
               16, F16)
    b = G.b
    ref, tol = b.reference(0.2)
    C.assert_within(G.run(2, None, 0.2), ref, tol)
    G.prefix = [15, 0, 130]  # of contexts of 124 and 134 positions; the last one shares 128
    b.table[4, :8] = b.table[5, :8]
    table = b.table.clone()
    ref, tol = b.reference(0.2)
    C.assert_within(G.run(2, None, 0.2, table=table), ref, tol)
    none = Groups(7, [0], [], [1, 2, 1, 1, 1, 1], [20, 30, 40, 50, 60, 70], 4, 2, 64, 16, F16)
    ref, tol = none.b.reference(0.2)
    C.assert_within(none.run(2, None, 0.2), ref, tol)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("D", [64, 128])
def test_scores_that_outgrow_the_first_steps(dtype, D):
    G = Groups(8, [0, 5], [2000], [1, 3, 1, 1, 2], [200, 300, 0, 17, 150], 8, 2, D, 16, dtype)
    b = G.b
    for i, at in ((0, 1990), (0, 700), (1, 2100), (4, 2149)):  # keys that one query each likes best
        page = int(b.table[i, at // 16])
        b.k[page, :, at % 16] = 4 * b.q[i, ::4]
    ref, tol = b.reference(0.3)
    C.assert_within(G.run(3, None, 0.3), ref, tol)


def test_rows_that_see_nothing():
    lens = [2, 3]
    G = Groups(9, [0, 2], [0], lens, [0, 0], 4, 2, 64, 16, BF16)
    masks = [0, 3, 1, 0, 5]
    ref, tol = G.b.reference(0.2, masks)
    got = G.run(3, masks, 0.2)
    C.assert_within(got, ref, tol)
    assert bool((got[0] == 0).all()) and bool((got[3] == 0).all())


def test_bad_groups_and_sequences():
    G = Groups(10, [0, 3, 5], [64, 96], [1, 2, 1, 1, 1], [10, 20, 30, 40, 50], 4, 2, 64, 16, BF16)
    b, table = G.b, G.b.table.clone()
    ref, tol = b.reference(0.2)
    good = G.cu, G.prefix
    # groups out of range: the error bit, and every sequence by itself
    for cu, prefix in (([0, 9, 9], [64, 96]), ([-1, 3, 5], [64, 96]), ([3, 0, 5], [64, 96]),
                       ([0, 3, 5], [64, 10 ** 6]), ([0, 3, 5], [-5, 96])):
        G.cu, G.prefix = cu, prefix
        C.assert_within(G.run(2, None, 0.2, want_err=1, table=table), ref, tol, f"{cu} {prefix}")
    G.cu, G.prefix = good
    # a page of the prefix outside the cache: zeros in its place, the other group as before
    bad = table.clone()
    bad[0, 1] = b.k.shape[0] + 1
    got = G.run(2, None, 0.2, want_err=1, table=bad)
    C.assert_within(got[4:], ref[4:], tol[4:])
    # a sequence outside its table: its rows are not written, the others of its group are right
    b.ctx[1] = 10 ** 6
    out = torch.full_like(b.q, 7.0)
    got = G.run(2, None, 0.2, want_err=1, table=table, out=out)
    keep = [0, 3, 4, 5]
    C.assert_within(got[keep], ref[keep], tol[keep])
    assert bool((got[1:3] == 7.0).all())


def test_streams_graphs_and_workspaces():
    G = Groups(11, [0, 20, 30], [3000, 400], [1 + i % 3 for i in range(30)],
               [(i * 31) % 200 for i in range(30)], 8, 2, 128, 16, BF16, pad_rows=3)
    b = G.b
    want = torch.full_like(b.q, 5.0)
    G.run(3, out=want)
    assert bool((want[-3:] == 5.0).all())
    ref, tol = b.reference(128 ** -0.5)
    C.assert_within(want[:-3], ref[:-3], tol[:-3])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert torch.equal(G.run(3, stream=side)[:-3], want[:-3])
    cache = Bn.KvCache(b.k, b.v)
    i32 = dict(dtype=torch.int32, device="cuda")
    cu, prefix = torch.tensor(G.cu, **i32), torch.tensor(G.prefix, **i32)
    out = torch.zeros_like(b.q)
    ws = torch.full((1 << 27,), 255, dtype=torch.uint8, device="cuda")  # anything may be in it
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        Bn.prefix_attention(cache, b.q, b.cu, b.ctx, G.hidden, cu, prefix, 3, out=out, workspace=ws)
    for _ in range(2):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[:-3], want[:-3])
    # replayed on other lengths: the second group shares nothing any more
    prefix[1] = 0
    g.replay()
    torch.cuda.synchronize()
    assert not torch.isnan(out[:sum(b.lens[:20])]).any()
    C.assert_within(out[:sum(b.lens[:20])], ref[:sum(b.lens[:20])], tol[:sum(b.lens[:20])])


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 128), (6, 1, 64), (4, 4, 64), (16, 1, 128)])
@pytest.mark.parametrize("page", [16, 128])
def test_few_sequences_in_both_forms(dtype, Hq, Hkv, D, page):
    """A narrow table goes to clusters, one that could hold long sequences to the tiles.  Sequences of one step
    and of many, an odd number of them, with a group in between that has none."""
    lens, after = [1, 2, 1, 1, 2, 1, 1], [0, 700, 1, 127, 128, 300, 40]
    G = Groups(13 + D, [0, 2, 2, 6], [400, 99, 260], lens, after, Hq, Hkv, D, page, dtype)
    masks = tree_masks(5, lens)
    ref, tol = G.b.reference(0.1, masks)
    C.assert_within(G.run(2, masks, 0.1), ref, tol)
    wide = torch.full((7, 20000 // page), -4, dtype=torch.int32, device="cuda")
    wide[:, :G.hidden.shape[1]] = G.hidden
    C.assert_within(G.run(2, masks, 0.1, table=wide), ref, tol)


def test_waits_that_give_up():
    """With a limit that its waits run into, the call ends with the time-out bit and the next is right."""
    G = Groups(12, [0, 8], [6000], [1] * 8, [100] * 8, 8, 2, 128, 64, BF16)
    b = G.b
    ref, tol = b.reference(128 ** -0.5)
    cache = Bn.KvCache(b.k, b.v)
    i32 = dict(dtype=torch.int32, device="cuda")
    cu, prefix = torch.tensor(G.cu, **i32), torch.tensor(G.prefix, **i32)

    def call():
        err = torch.zeros(1, **i32)
        out = Bn.prefix_attention(cache, b.q, b.cu, b.ctx, G.hidden, cu, prefix, 16,
                                  device_error=err)  # (room for 64 rows: on the tiles)
        torch.cuda.synchronize()
        return out, int(err)

    call()
    seen = []
    try:
        for cycles in (1, 500, 1500, 3000):
            Bn.debug_attention_wait_cycles(cycles)
            seen += [call()[1] for _ in range(3)]
    finally:
        Bn.debug_attention_wait_cycles(0)
    assert set(seen) <= {0, 2} and set(seen[:3]) == {2}, seen
    out, e = call()
    assert e == 0
    C.assert_within(out, ref, tol)
