"""What the attention calls refuse, on the host: addresses here are never read, since every call is
refused before anything is enqueued (or has nothing to enqueue)."""
import ctypes

import pytest
import torch

from quantized_moe_expert_dequant_gb300 import binding as Bn

INV, UNS = Bn.MOE_ERR_INVALID_ARG, Bn.MOE_ERR_UNSUPPORTED


def _struct(*groups):
    return type("Struct", (ctypes.Structure,), {"_fields_": [
        (n, t) for names, t in groups for n in names.split()]})


# the structs as the header declares them, field by field
KvCacheStruct = _struct(("k v", ctypes.c_void_p),
                        ("page_stride head_stride token_stride", ctypes.c_int64),
                        ("n_pages page_size n_kv_heads head_dim dtype", ctypes.c_int32))
NormRopeStruct = _struct(
    ("q k v", ctypes.c_void_p),
    ("q_row_stride q_head_stride k_row_stride k_head_stride v_row_stride v_head_stride",
     ctypes.c_int64), ("q_out", ctypes.c_void_p),
    ("q_out_row_stride q_out_head_stride", ctypes.c_int64),
    ("q_weight k_weight inv_freq positions slots device_error", ctypes.c_void_p),
    ("n_tokens n_q_heads rot_dim interleaved in_dtype", ctypes.c_int32), ("eps", ctypes.c_float))
AttentionStruct = _struct(
    ("q out", ctypes.c_void_p),
    ("q_row_stride q_head_stride out_row_stride out_head_stride", ctypes.c_int64),
    ("cu_q ctx_len page_table", ctypes.c_void_p), ("table_stride", ctypes.c_int64),
    ("table_width n_seqs n_rows n_q_heads", ctypes.c_int32), ("scale", ctypes.c_float),
    ("device_error", ctypes.c_void_p))


@pytest.fixture(scope="module")
def L():
    import __graft_entry__
    __graft_entry__.build()
    return Bn.lib()


def cache(**kw):
    base = dict(k=0x1000, v=0x2000, page_stride=8192, head_stride=1024, token_stride=64, n_pages=4,
                page_size=16, n_kv_heads=8, head_dim=64, dtype=Bn.DTYPE_BF16)
    base.update(kw)
    return KvCacheStruct(**base)


def rope(**kw):
    base = dict(q=0x1000, k=0x2000, v=0x3000, q_out=0x4000, positions=0x5000, slots=0x6000,
                inv_freq=0x7000, n_tokens=1, n_q_heads=8, rot_dim=64, interleaved=0,
                in_dtype=Bn.DTYPE_F32, eps=1e-6)
    base.update(kw)
    return NormRopeStruct(**base)


def attention(**kw):
    base = dict(q=0x1000, out=0x2000, cu_q=0x3000, ctx_len=0x4000, page_table=0x5000,
                table_stride=4, table_width=4, n_seqs=1, n_rows=1, n_q_heads=8, scale=0.125)
    base.update(kw)
    return AttentionStruct(**base)


BAD_CACHE = [
    (dict(k=None), INV), (dict(v=None), INV), (dict(k=0x1008), INV), (dict(v=0x2002), INV),
    (dict(page_stride=-8), INV), (dict(head_stride=4), INV), (dict(token_stride=65), INV),
    (dict(n_pages=0), INV), (dict(page_size=0), INV), (dict(n_kv_heads=0), INV),
    (dict(dtype=Bn.DTYPE_F32), INV), (dict(dtype=9), INV), (dict(head_dim=96), UNS),
    (dict(n_pages=2 ** 30, page_size=16), UNS),
]


@pytest.mark.parametrize("kw,rc", BAD_CACHE)
def test_caches(L, kw, rc):
    c, n = cache(**kw), ctypes.c_int64(7)
    ref = ctypes.byref
    assert L.moe_qk_norm_rope(ref(c), ref(rope()), None) == rc
    assert L.moe_prompt_attention(ref(c), ref(attention()), None, 0, None) == rc
    assert L.moe_tree_attention(ref(c), ref(attention()), None, 1, None, 0, None) == rc
    assert L.moe_tree_attention_workspace(ref(c), ref(attention()), 1, ref(n)) == rc
    assert L.moe_prompt_attention_workspace(ref(c), ref(attention()), ref(n)) == rc
    assert n.value == 7


@pytest.mark.parametrize("kw,rc", [
    (dict(n_tokens=-1), INV), (dict(n_q_heads=0), INV), (dict(rot_dim=-16), INV),
    (dict(rot_dim=80), INV), (dict(rot_dim=24), UNS), (dict(eps=-1.0), INV),
    (dict(eps=float("nan")), INV), (dict(eps=2.0), INV), (dict(in_dtype=Bn.DTYPE_F16), UNS),
    (dict(in_dtype=7), UNS), (dict(interleaved=2), INV), (dict(q=None), INV), (dict(k=None), INV),
    (dict(v=None), INV), (dict(q_out=None), INV), (dict(slots=None), INV),
    (dict(positions=None), INV), (dict(inv_freq=None), INV), (dict(q=0x1004), INV),
    (dict(q_out=0x4008), INV), (dict(q_weight=0x8008), INV), (dict(inv_freq=0x7004), INV),
    (dict(slots=0x6001), INV), (dict(device_error=0x9002), INV), (dict(q_row_stride=2), INV),
    (dict(k_head_stride=-4), INV), (dict(q_out_row_stride=4), INV), (dict(n_q_heads=70000), UNS),
])
def test_norm_rope(L, kw, rc):
    assert L.moe_qk_norm_rope(ctypes.byref(cache()), ctypes.byref(rope(**kw)), None) == rc


@pytest.mark.parametrize("kw,rc", [
    (dict(n_seqs=-1), INV), (dict(n_rows=-1), INV), (dict(n_q_heads=0), INV),
    (dict(n_q_heads=12), INV), (dict(n_q_heads=8 * 65), UNS), (dict(q=None), INV),
    (dict(out=None), INV), (dict(cu_q=None), INV), (dict(ctx_len=None), INV),
    (dict(page_table=None), INV), (dict(table_width=0), INV), (dict(table_stride=3), INV),
    (dict(scale=0.0), INV), (dict(scale=-1.0), INV), (dict(scale=float("nan")), INV),
    (dict(scale=float("inf")), INV), (dict(q=0x1008), INV), (dict(out=0x2004), INV),
    (dict(q_row_stride=4), INV), (dict(out_head_stride=-8), INV), (dict(cu_q=0x3002), INV),
    (dict(device_error=0x9001), INV),
])
def test_attention(L, kw, rc):
    c, a, n = cache(), attention(**kw), ctypes.c_int64()
    ref = ctypes.byref
    assert L.moe_prompt_attention(ref(c), ref(a), None, 0, None) == rc
    assert L.moe_tree_attention(ref(c), ref(a), None, 1, None, 0, None) == rc
    assert L.moe_tree_attention_workspace(ref(c), ref(a), 1, ref(n)) == rc
    assert L.moe_prompt_attention_workspace(ref(c), ref(a), ref(n)) == rc


@pytest.mark.parametrize("page", [8, 24, 48, 2048])
def test_page_sizes_of_attention(L, page):
    c = cache(page_size=page)
    assert L.moe_prompt_attention(ctypes.byref(c), ctypes.byref(attention()), None, 0,
                                  None) == UNS
    assert L.moe_tree_attention(ctypes.byref(c), ctypes.byref(attention()), None, 1, None, 0,
                                None) == UNS


def test_tree_arguments(L):
    ref = ctypes.byref
    c, a, n = cache(), attention(), ctypes.c_int64()
    for max_q, rc in ((0, INV), (-1, INV), (65, UNS)):
        assert L.moe_tree_attention(ref(c), ref(a), None, max_q, None, 0, None) == rc
        assert L.moe_tree_attention_workspace(ref(c), ref(a), max_q, ref(n)) == rc
    assert L.moe_tree_attention_workspace(ref(c), ref(a), 1, None) == INV
    assert L.moe_prompt_attention_workspace(ref(c), ref(a), None) == INV
    assert L.moe_prompt_attention(ref(c), ref(a), 0x1008, 1 << 40, None) == INV
    assert L.moe_prompt_attention(ref(c), ref(a), None, -1, None) == INV
    assert L.moe_tree_attention(ref(c), ref(a), 0x1004, 1, None, 0, None) == INV   # mask address
    assert L.moe_tree_attention(ref(c), ref(a), None, 1, 0x1008, 1 << 40, None) == INV
    assert L.moe_tree_attention(ref(c), ref(a), None, 1, None, -1, None) == INV


def test_null_and_empty_calls(L):
    ref = ctypes.byref
    assert L.moe_qk_norm_rope(None, ref(rope()), None) == INV
    assert L.moe_qk_norm_rope(ref(cache()), None, None) == INV
    assert L.moe_prompt_attention(None, ref(attention()), None, 0, None) == INV
    assert L.moe_prompt_attention(ref(cache()), None, None, 0, None) == INV
    assert L.moe_tree_attention(ref(cache()), None, None, 1, None, 0, None) == INV
    none = dict(q=None, k=None, v=None, q_out=None, slots=None, positions=None)
    assert L.moe_qk_norm_rope(ref(cache()), ref(rope(n_tokens=0, **none)), None) == Bn.MOE_OK
    a = attention(n_rows=0, q=None, out=None)
    assert L.moe_prompt_attention(ref(cache()), ref(a), None, 0, None) == Bn.MOE_OK
    assert L.moe_tree_attention(ref(cache()), ref(a), None, 1, None, 0, None) == Bn.MOE_OK


def test_the_binding_checks_tensors():
    x = torch.zeros((2, 2, 16, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        Bn.KvCache(x, x)                                   # not on a GPU
    meta = torch.zeros((2, 2, 16, 64), dtype=torch.bfloat16, device="meta")
    with pytest.raises(ValueError):
        Bn.KvCache(meta, meta)


@pytest.mark.parametrize("pack,S", [(Bn._pack_kv_cache, KvCacheStruct),
                                    (Bn._pack_norm_rope, NormRopeStruct),
                                    (Bn._pack_attention, AttentionStruct)])
def test_packed_bytes_have_the_layout_of_the_struct(pack, S):
    vals = [i + 1 for i in range(len(S._fields_))]
    b = pack(*vals)
    s = S.from_buffer_copy(b + bytes(max(0, ctypes.sizeof(S) - len(b))))
    assert [getattr(s, n) for n, _ in S._fields_] == vals


def test_wait_limits(L):
    assert L.moe_debug_attention_wait_cycles(-1) == INV
    assert L.moe_debug_attention_wait_cycles(1000) == Bn.MOE_OK
    assert L.moe_debug_attention_wait_cycles(0) == Bn.MOE_OK


@pytest.mark.parametrize("kind", ["tree", "prompt"])
def test_every_call_is_made_with_the_caches_gpu_current(monkeypatch, kind):
    """The workspace's size goes by the current GPU's SMs, as the launch does.  (No GPU here: the library,
    the current device and the tensors' place are stand-ins.)"""
    now, calls = [0], []

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

    monkeypatch.setattr(Bn, "_entry", entry)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: now[0], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0, raising=False)
    monkeypatch.setattr(torch.cuda, "device", Device)
    t = lambda *shape, dtype=torch.int32: torch.zeros(shape, dtype=dtype).as_subclass(OnGpu1)
    c = type("Cache", (), dict(_dev=1, head_dim=64, dtype=torch.bfloat16, _c=b"", device="cpu"))()
    q = t(1, 8, 64, dtype=torch.bfloat16)
    args = (c, q, t(2), t(1), t(1, 4))
    out = t(1, 8, 64, dtype=torch.bfloat16)
    if kind == "tree":
        Bn.tree_attention(*args, max_q=1, out=out)
    else:
        Bn.prompt_attention(*args, out=out)
    name = f"moe_{kind}_attention"
    assert calls == [(name + "_workspace", 1), (name, 1)] and now == [0]
