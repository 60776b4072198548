"""Calls that take their workspace from torch's allocator, captured: the memory stays the graph's."""
import pytest
import torch

from quantized_moe_expert_dequant_gb300 import binding as Bn
from tests import attention_cases as C
from tests import sparse_cases as S
from tests.test_gpu_pages import random_bounds

pytestmark = pytest.mark.gpu


def calls():
    """name -> (call that takes and returns out, outputs wanted)."""
    i32 = dict(dtype=torch.int32, device="cuda")
    b = C.batch(1, [1] * 60, [(37 * i) % 900 for i in range(60)], 8, 2, 128, 16, torch.bfloat16)
    cache = Bn.KvCache(b.k, b.v)
    pages = S.random_lists(b, 7, 4)
    sparse = lambda out, **kw: Bn.sparse_attention(cache, b.q, b.cu, b.ctx, b.table, pages, out=out, **kw)
    cu, none = torch.tensor([0, 60], **i32), torch.tensor([0], **i32)
    prefix = lambda out, **kw: Bn.prefix_attention(cache, b.q, b.cu, b.ctx, b.table, cu, none, 1, out=out,
                                                   **kw)
    c = C.batch(2, [40], [16 * 300], 8, 2, 128, 16, torch.bfloat16)
    bnd, ccache = random_bounds(c, 3), Bn.KvCache(c.k, c.v)
    select = lambda out, **kw: Bn.select_pages(ccache, bnd, c.q, c.cu, c.ctx, c.table, 20, out=out, **kw)
    return {"sparse": (sparse, torch.empty_like(b.q)), "prefix": (prefix, torch.empty_like(b.q)),
            "select": (select, torch.empty((40, 2, 20), **i32))}


@pytest.mark.parametrize("name", ["sparse", "prefix", "select"])
def test_a_graph_keeps_its_workspace(name):
    call, out = calls()[name]
    want = call(out).clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(out)
    # whatever was free is written over
    junk = [torch.full((1 << 22,), float("nan"), device="cuda") for _ in range(40)]
    for _ in range(2):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    del junk


@pytest.mark.parametrize("name", ["sparse", "prefix", "select"])
def test_two_graphs_at_once(name):
    (call, a), b = calls()[name], None
    want, b = call(a).clone(), torch.empty_like(a)
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    for g, out in zip(graphs, (a, b)):
        with torch.cuda.graph(g):
            for _ in range(5):
                call(out)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    a.zero_(), b.zero_()
    torch.cuda.synchronize()
    for _ in range(10):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, want) and torch.equal(b, want)


@pytest.mark.parametrize("name", ["sparse", "prefix", "select"])
def test_behind_other_work_and_joined_streams(name):
    """The kernels are set up while what is before them in the stream runs, whatever that is: a fill, a copy, another
    stream's event, also in a graph."""
    call, out = calls()[name]
    want = call(out).clone()
    big, side = torch.zeros(1 << 27, dtype=torch.uint8, device="cuda"), torch.cuda.Stream()
    held = torch.empty_like(out)

    def step():
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            big.fill_(1)
        out.zero_()
        main.wait_stream(side)
        call(out)
        held.copy_(out)
        out.fill_(3)
        call(out)

    step()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(held, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    out.zero_(), held.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(held, want)
