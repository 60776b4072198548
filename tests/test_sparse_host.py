"""What the calls that do not read the whole cache refuse, on the host: every call here is refused before
anything is enqueued (or has nothing to enqueue), so that the addresses are never read."""
import ctypes

import pytest
import torch

from quantized_moe_expert_dequant_gb300 import binding as Bn
from tests.test_attention_host import BAD_CACHE, INV, L, UNS, attention, cache  # noqa: F401

BIG = 1 << 40
ref = ctypes.byref


def calls(L, c, a, **kw):
    """Every call and workspace question with the same cache and arguments."""
    n = ctypes.c_int64(7)
    rcs = {
        "bounds": L.moe_page_bounds(ref(c), ref(a), 0x8000, None),
        "select_ws": L.moe_select_pages_workspace(ref(c), ref(a), ref(n)),
        "select": L.moe_select_pages(ref(c), ref(a), 0x8000, 4, 1, 1, 0x9000, 0x10000, BIG, None),
        "sparse_ws": L.moe_sparse_attention_workspace(ref(c), ref(a), 4, ref(n)),
        "sparse": L.moe_sparse_attention(ref(c), ref(a), 0x9000, 4, 0x10000, BIG, None),
        "prefix_ws": L.moe_prefix_attention_workspace(ref(c), ref(a), 1, 1, ref(n)),
        "prefix": L.moe_prefix_attention(ref(c), ref(a), 0x8000, 0x9000, 1, None, 1, 0x10000, BIG,
                                         None),
    }
    assert n.value == 7
    return rcs


@pytest.mark.parametrize("kw,rc", BAD_CACHE + [(dict(page_size=p), UNS) for p in (8, 24, 48, 2048)])
def test_caches(L, kw, rc):
    assert set(calls(L, cache(**kw), attention()).values()) == {rc}


@pytest.mark.parametrize("kw,rc", [
    (dict(n_seqs=-1), INV), (dict(n_rows=-1), INV), (dict(cu_q=None), INV),
    (dict(ctx_len=None), INV), (dict(page_table=None), INV), (dict(table_width=0), INV),
    (dict(table_stride=3), INV), (dict(cu_q=0x3002), INV), (dict(device_error=0x9001), INV)])
def test_batches(L, kw, rc):
    assert set(calls(L, cache(), attention(**kw)).values()) == {rc}


@pytest.mark.parametrize("kw,rc", [
    (dict(n_q_heads=0), INV), (dict(n_q_heads=12), INV), (dict(n_q_heads=8 * 65), UNS),
    (dict(q=None), INV), (dict(q=0x1008), INV), (dict(q_row_stride=4), INV)])
def test_queries(L, kw, rc):
    c, a, n = cache(), attention(**kw), ctypes.c_int64()
    assert L.moe_select_pages_workspace(ref(c), ref(a), ref(n)) == rc
    assert L.moe_select_pages(ref(c), ref(a), 0x8000, 4, 1, 1, 0x9000, 0x10000, BIG, None) == rc
    assert L.moe_sparse_attention(ref(c), ref(a), 0x9000, 4, 0x10000, BIG, None) == rc
    assert L.moe_prefix_attention(ref(c), ref(a), 0x8000, 0x9000, 1, None, 1, 0x10000, BIG, None) == rc


@pytest.mark.parametrize("kw,rc", [
    (dict(out=None), INV), (dict(out=0x2004), INV), (dict(out_head_stride=-8), INV),
    (dict(scale=0.0), INV), (dict(scale=float("nan")), INV)])
def test_outputs(L, kw, rc):
    c, a = cache(), attention(**kw)
    assert L.moe_sparse_attention(ref(c), ref(a), 0x9000, 4, 0x10000, BIG, None) == rc
    assert L.moe_prefix_attention(ref(c), ref(a), 0x8000, 0x9000, 1, None, 1, 0x10000, BIG, None) == rc


def test_arguments(L):
    c, a, n = cache(), attention(), ctypes.c_int64()
    for bounds in (None, 0x8008):
        assert L.moe_page_bounds(ref(c), ref(a), bounds, None) == INV
    sel = lambda **k: L.moe_select_pages(
        ref(c), ref(a), *{**dict(bounds=0x8000, n=4, sink=1, recent=1, pages=0x9000, ws=0x10000,
                                 size=BIG), **k}.values(), None)
    for kw in (dict(bounds=None), dict(bounds=0x8008), dict(n=1), dict(n=0), dict(sink=-1),
               dict(recent=0), dict(sink=4), dict(sink=2 ** 31 - 1, recent=2), dict(pages=None),
               dict(pages=0x9002), dict(ws=0x10008), dict(size=-1)):
        assert sel(**kw) == INV, kw
    assert L.moe_select_pages_workspace(ref(c), ref(a), None) == INV
    wide = attention(table_width=65537, table_stride=65537)
    assert L.moe_select_pages_workspace(ref(c), ref(wide), ref(n)) == UNS
    assert L.moe_select_pages(ref(c), ref(wide), 0x8000, 4, 1, 1, 0x9000, 0x10000, BIG, None) == UNS
    for pages, k, ws, size in ((None, 4, 0x10000, BIG), (0x9002, 4, 0x10000, BIG),
                               (0x9000, 0, 0x10000, BIG), (0x9000, 4, 0x10008, BIG),
                               (0x9000, 4, 0x10000, -1)):
        assert L.moe_sparse_attention(ref(c), ref(a), pages, k, ws, size, None) == INV
    assert L.moe_sparse_attention_workspace(ref(c), ref(a), 4, None) == INV
    many = attention(n_q_heads=8 * 33)
    assert L.moe_sparse_attention(ref(c), ref(many), 0x9000, 4, 0x10000, BIG, None) == UNS
    assert L.moe_sparse_attention_workspace(ref(c), ref(many), 4, ref(n)) == UNS
    pre = lambda **k: L.moe_prefix_attention(
        ref(c), ref(a), *{**dict(cu=0x8000, len=0x9000, groups=1, mask=None, max_q=1, ws=0x10000,
                                 size=BIG), **k}.values(), None)
    for kw, rc in ((dict(cu=None), INV), (dict(len=None), INV), (dict(cu=0x8002), INV),
                   (dict(len=0x9001), INV), (dict(groups=-1), INV), (dict(mask=0x1004), INV),
                   (dict(max_q=0), INV), (dict(max_q=65), UNS), (dict(ws=0x10008), INV),
                   (dict(size=-1), INV), (dict(groups=2 ** 31 - 1), UNS)):
        assert pre(**kw) == rc, kw
    assert L.moe_prefix_attention_workspace(ref(c), ref(a), 1, 1, None) == INV


def test_null_and_empty_calls(L):
    c = cache()
    n = ctypes.c_int64(7)
    for args in ((None, ref(attention())), (ref(c), None)):
        assert L.moe_page_bounds(*args, 0x8000, None) == INV
        assert L.moe_select_pages(*args, 0x8000, 4, 1, 1, 0x9000, 0x10000, BIG, None) == INV
        assert L.moe_sparse_attention(*args, 0x9000, 4, 0x10000, BIG, None) == INV
        assert L.moe_prefix_attention(*args, 0x8000, 0x9000, 1, None, 1, 0x10000, BIG, None) == INV
    for a in (attention(n_rows=0, q=None, out=None), attention(n_seqs=0)):
        assert L.moe_page_bounds(ref(c), ref(a), 0x8000, None) == Bn.MOE_OK
        assert L.moe_select_pages(ref(c), ref(a), None, 4, 1, 1, None, None, 0, None) == Bn.MOE_OK
        assert L.moe_sparse_attention(ref(c), ref(a), None, 4, None, 0, None) == Bn.MOE_OK
        assert L.moe_prefix_attention(ref(c), ref(a), None, None, 1, None, 1, None, 0, None) == Bn.MOE_OK
        for f, more in ((L.moe_select_pages_workspace, ()), (L.moe_sparse_attention_workspace, (4,)),
                        (L.moe_prefix_attention_workspace, (1, 1))):
            assert f(ref(c), ref(a), *more, ref(n)) == Bn.MOE_OK and n.value == 0


def test_bounds_go_without_queries(L):
    """q, out, the query heads and the scale are not looked at: with everything else right, only the missing
    bounds are refused."""
    a = attention(q=0x1001, out=None, n_q_heads=0, q_row_stride=3, scale=float("nan"))
    assert L.moe_page_bounds(ref(cache()), ref(a), None, None) == INV
    a.n_rows = 0
    assert L.moe_page_bounds(ref(cache()), ref(a), 0x8000, None) == Bn.MOE_OK


@pytest.mark.parametrize("kind", ["prefix", "select", "sparse", "bounds"])
def test_every_call_is_made_with_the_caches_gpu_current(monkeypatch, kind):
    """What a call asks, allocates and launches goes by the cache's GPU.  (No GPU here: the library, the current
    device, the allocator and the tensors' place are stand-ins.)"""
    now, calls, held = [0], [], []

    class Device:
        def __init__(self, dev):
            self.dev = dev

        def __enter__(self):
            self.before, now[0] = now[0], self.dev

        def __exit__(self, *e):
            now[0] = self.before

    class OnGpu1(torch.Tensor):
        def get_device(self):
            return 1

    def entry(fn):
        def call(*args):
            calls.append((fn, now[0]))
            if fn.endswith("_workspace"):
                args[-1]._obj.value = 64
            return Bn.MOE_OK
        return call

    def alloc(n, stream):
        held.append(n)
        calls.append((n, now[0]))
        return 4096

    monkeypatch.setattr(Bn, "_entry", entry)
    for name, f in (("_cuda_getDevice", lambda: now[0]), ("_cuda_getCurrentRawStream", lambda dev: 0),
                    ("_cuda_cudaCachingAllocator_raw_alloc", alloc),
                    ("_cuda_cudaCachingAllocator_raw_delete", lambda p: held.pop())):
        monkeypatch.setattr(torch._C, name, f, raising=False)
    monkeypatch.setattr(torch.cuda, "device", Device)
    t = lambda *shape, dtype=torch.int32: torch.zeros(shape, dtype=dtype).as_subclass(OnGpu1)
    bf16 = torch.bfloat16
    c = type("Cache", (), dict(_dev=1, head_dim=64, n_pages=3, n_kv_heads=8, page_size=16, dtype=bf16, _c=b"",
                               device="cpu", _shape=(3, 8, 16, 64, 0), _bounds=(3, 8, 2, 64), _sizes={}))()
    q, batch = t(1, 8, 64, dtype=bf16), (t(2), t(1), t(1, 4))
    bounds = t(3, 8, 2, 64, dtype=bf16)
    if kind == "prefix":
        Bn.prefix_attention(c, q, *batch, t(2), t(1), max_q=1, out=t(1, 8, 64, dtype=bf16))
    elif kind == "select":
        Bn.select_pages(c, bounds, q, *batch, n_select=4, out=t(1, 8, 4))
    elif kind == "sparse":
        Bn.sparse_attention(c, q, *batch, t(1, 8, 4), out=t(1, 8, 64, dtype=bf16))
    else:
        Bn.page_bounds(c, bounds, *batch, n_rows=1)
    name = {"prefix": "moe_prefix_attention", "select": "moe_select_pages",
            "sparse": "moe_sparse_attention", "bounds": "moe_page_bounds"}[kind]
    asked = [] if kind == "bounds" else [(name + "_workspace", 1), (64, 1)]
    assert calls == asked + [(name, 1)] and now == [0] and held == []


def test_the_binding_checks_shapes():
    t = lambda *shape, dtype=torch.int32: torch.zeros(shape, dtype=dtype)
    bf16 = torch.bfloat16
    c = type("Cache", (), dict(_dev=-1, head_dim=64, n_pages=3, n_kv_heads=2, page_size=16, dtype=bf16, _c=b"",
                               device="cpu", _shape=(3, 2, 16, 64, 0), _bounds=(3, 2, 2, 64), _sizes={}))()
    q, batch, bounds = t(1, 4, 64, dtype=bf16), (t(2), t(1), t(1, 4)), t(3, 2, 2, 64, dtype=bf16)
    for f in (lambda: Bn.page_bounds(c, t(3, 2, 64, dtype=bf16), *batch, n_rows=1),
              lambda: Bn.page_bounds(c, bounds.half(), *batch, n_rows=1),
              lambda: Bn.page_bounds(c, bounds, t(1), *batch[1:], n_rows=1),
              lambda: Bn.page_bounds(c, bounds, batch[0].long(), *batch[1:], n_rows=1),
              lambda: Bn.select_pages(c, bounds, t(1, 4, 32, dtype=bf16), *batch, n_select=4),
              lambda: Bn.select_pages(c, bounds, q.half(), *batch, n_select=4),
              lambda: Bn.select_pages(c, bounds, q, *batch, n_select=4, out=t(1, 2, 5)),
              lambda: Bn.select_pages(c, bounds[:2], q, *batch, n_select=4, out=t(1, 2, 4)),
              lambda: Bn.sparse_attention(c, q, *batch, t(1, 3, 4)),
              lambda: Bn.sparse_attention(c, q, *batch, t(1, 8)),
              lambda: Bn.sparse_attention(c, q, *batch, t(1, 2, 4).long()),
              lambda: Bn.prefix_attention(c, q, *batch, t(1), t(1), max_q=1),
              lambda: Bn.prefix_attention(c, q, *batch, t(2), t(1).long(), max_q=1),
              lambda: Bn.prefix_attention(c, q, *batch, t(2), t(1), max_q=1, tree_mask=t(1))):
        with pytest.raises(ValueError):
            f()
