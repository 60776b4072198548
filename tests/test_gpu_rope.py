"""Norms, rotation and the write into the cache (moe_qk_norm_rope) against the formula in fp64, and
the three attention operators one after the other as a decoder layer uses them."""
import pytest
import torch

from quantized_moe_expert_dequant_gb300 import binding as Bn
from tests import attention_cases as C

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def inputs(seed, T, Hq, Hkv, D, dt_in, dt, R):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn((T, Hq + 2 * Hkv, D), generator=g) * 3).to(dt_in).cuda()
    w = [(1 + 0.2 * torch.randn(D, generator=g)).to(dt).cuda() for _ in range(2)]
    f = 1e4 ** (-torch.arange(0, R, 2, dtype=torch.float64) / max(R, 1)) if R else None
    return x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], w, None if f is None else f.cuda()


def check(T, Hq, Hkv, D, dt_in, dt, R, interleaved, norm, page=16, pos0=0, eps=1e-6, seed=0,
          token_major=False):
    q, k, v, w, f = inputs(seed + T, T, Hq, Hkv, D, dt_in, dt, R)
    n_pages = -(-T // page) + 2
    g = torch.Generator().manual_seed(seed)
    slots = torch.randperm(n_pages * page, generator=g)[:T].to(torch.int32)
    if T > 3:
        slots[2] = -1
    slots = slots.cuda()
    pos = (torch.arange(T, dtype=torch.int32) * 7 + pos0).cuda()
    shape = (n_pages, page, Hkv, D) if token_major else (n_pages, Hkv, page, D)
    kc = torch.full(shape, 3.0, dtype=dt, device="cuda")
    vc = torch.full(shape, 3.0, dtype=dt, device="cuda")
    if token_major:
        kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
    out = torch.full((T, Hq, D), 3.0, dtype=dt, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    wq, wk = w if norm else (None, None)
    Bn.qk_norm_rope(Bn.KvCache(kc, vc), q, k, v, pos, slots, f, wq, wk, eps, interleaved,
                    q_out=out, device_error=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    live = slots >= 0
    ref, tol = C.norm_rope(q, wq, pos, f, eps, interleaved, dt)
    C.assert_within(out[live], ref[live], tol[live], "q")
    assert bool((out[~live] == 3).all())
    ref, tol = C.norm_rope(k, wk, pos, f, eps, interleaved, dt)
    at = slots[live].long()
    flat = lambda c: c.transpose(1, 2).reshape(-1, Hkv, D)
    C.assert_within(flat(kc)[at], ref[live], tol[live], "k")
    assert torch.equal(flat(vc)[at], v.to(dt)[live])
    rest = torch.ones(n_pages * page, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert bool((flat(kc)[rest] == 3).all() and (flat(vc)[rest] == 3).all())


@pytest.mark.parametrize("dt_in,dt", [(F32, BF16), (BF16, BF16), (F32, F16), (F16, F16)])
@pytest.mark.parametrize("D,R", [(64, 64), (64, 16), (128, 128), (128, 96), (128, 0)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_types_and_rotations(dt_in, dt, D, R, interleaved, norm):
    check(37, 5, 3, D, dt_in, dt, R, interleaved, norm, pos0=11)


@pytest.mark.parametrize("T", [1, 2, 3, 8, 33, 1000])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (32, 8), (12, 2), (7, 7), (96, 8)])
def test_tokens_and_heads(T, Hq, Hkv):
    check(T, Hq, Hkv, 128, F32, BF16, 128, False, True, page=64)
    check(T, Hq, Hkv, 64, F16, F16, 32, True, False, page=7, token_major=True)


@pytest.mark.parametrize("pos0", [0, 1000003, 2 ** 31 - 300, -250])
def test_far_positions(pos0):
    check(40, 4, 2, 128, F32, BF16, 128, False, True, pos0=pos0)


def test_zero_and_tiny_heads():
    """A head of zeros stays zeros (eps > 0); small heads are brought to the same size by the norm."""
    q, k, v, w, f = inputs(5, 4, 4, 2, 64, F32, BF16, 64)
    q[1] = 0
    q[2] *= 1e-6
    kc = torch.zeros((1, 2, 16, 64), dtype=BF16, device="cuda")
    pos = torch.arange(4, dtype=torch.int32, device="cuda")
    out = Bn.qk_norm_rope(Bn.KvCache(kc, kc.clone()), q, k, v, pos, pos, f, w[0], w[1], 1e-10)
    ref, tol = C.norm_rope(q, w[0], pos, f, 1e-10, False, BF16)
    C.assert_within(out, ref, tol)
    assert not bool(out[1].any())


def test_in_place_and_one_norm():
    q, k, v, w, f = inputs(6, 21, 6, 2, 128, BF16, BF16, 128)
    pos = torch.arange(21, dtype=torch.int32, device="cuda")
    kc = torch.zeros((2, 2, 16, 128), dtype=BF16, device="cuda")
    cache = Bn.KvCache(kc, kc.clone())
    ref, tol = C.norm_rope(q, w[0], pos, f, 1e-6, False, BF16)
    other = Bn.qk_norm_rope(cache, q, k, v, pos, pos, f, w[0], None)
    same = Bn.qk_norm_rope(cache, q, k, v, pos, pos, f, w[0], None, q_out=q)
    assert same.data_ptr() == q.data_ptr() and torch.equal(same, other)
    C.assert_within(q, ref, tol)
    ref, tol = C.norm_rope(k, None, pos, f, 1e-6, False, BF16)
    C.assert_within(kc.transpose(1, 2).reshape(-1, 2, 128)[:21], ref, tol)


def test_bad_slots_are_reported():
    q, k, v, w, f = inputs(7, 5, 4, 2, 64, BF16, BF16, 64)
    kc = torch.full((2, 2, 16, 64), 3.0, dtype=BF16, device="cuda")
    vc = kc.clone()
    pos = torch.arange(5, dtype=torch.int32, device="cuda")
    slots = torch.tensor([0, 32, 1, 2 ** 31 - 1, 31], dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = Bn.qk_norm_rope(Bn.KvCache(kc, vc), q, k, v, pos, slots, f, device_error=err)
    torch.cuda.synchronize()
    assert int(err) == 1
    ref, tol = C.norm_rope(q, None, pos, f, 0, False, BF16)
    C.assert_within(out, ref, tol)
    flat = vc.transpose(1, 2).reshape(-1, 2, 64)
    assert torch.equal(flat[[0, 1, 31]], v[[0, 2, 4]]) and bool((flat[2:31] == 3).all())


def test_the_binding_refuses_other_tensors():
    q, k, v, w, f = inputs(9, 5, 4, 2, 64, BF16, BF16, 64)
    kc = torch.zeros((1, 2, 16, 64), dtype=BF16, device="cuda")
    cache = Bn.KvCache(kc, kc.clone())
    n = torch.arange(5, dtype=torch.int32, device="cuda")
    good = dict(q=q, k=k, v=v, positions=n, slots=n, inv_freq=f)
    Bn.qk_norm_rope(cache, **good)
    bad = [dict(k=k[:4]), dict(k=k.half()), dict(v=v.cpu()), dict(v=v[:, :1]), dict(slots=n[:4]),
           dict(slots=n.long()), dict(slots=n.cpu()), dict(positions=n[:4]), dict(q=q.double()),
           dict(q=q[..., :32]), dict(inv_freq=f.float()), dict(q_weight=w[0].float()),
           dict(k_weight=w[1][:32]), dict(q_out=torch.empty_like(q).half()),
           dict(q=q.transpose(1, 2).contiguous().transpose(1, 2)),
           dict(slots=torch.zeros(10, dtype=torch.int32, device="cuda")[::2])]
    for kw in bad:
        with pytest.raises(ValueError):
            Bn.qk_norm_rope(cache, **{**good, **kw})


def test_no_tokens():
    q, k, v, w, f = inputs(8, 0, 4, 2, 64, BF16, BF16, 64)
    kc = torch.zeros((1, 2, 16, 64), dtype=BF16, device="cuda")
    e = torch.zeros(0, dtype=torch.int32, device="cuda")
    assert Bn.qk_norm_rope(Bn.KvCache(kc, kc.clone()), q, k, v, e, e, f).shape == (0, 4, 64)


@pytest.mark.parametrize("Hq,Hkv,D,dtype", [(8, 2, 128, BF16), (6, 6, 64, F16)])
def test_prompt_chunk_draft_and_token_of_one_text(Hq, Hkv, D, dtype):
    """Two texts go through prompt, chunk, tree and single tokens; every output equals attention of
    the whole text so far, formed from the queries, keys and values the first operator gave."""
    page, eps = 16, 1e-6
    steps = [([50, 20], "prompt"), ([33, 70], "prompt"), ([6, 3], "tree"), ([1, 1], "tree")]
    g = torch.Generator().manual_seed(D)
    n_pages = 40
    kc = torch.full((n_pages, Hkv, page, D), float("nan"), dtype=dtype, device="cuda")
    cache = Bn.KvCache(kc, kc.clone())
    order = torch.randperm(n_pages, generator=g).to(torch.int32)
    table = order.view(2, 20).cuda()
    f = 1e6 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D).cuda()
    w = [(1 + 0.2 * torch.randn(D, generator=g)).to(dtype).cuda() for _ in range(2)]
    ctx = [0, 0]
    for lens, kind in steps:
        T = sum(lens)
        x = (torch.randn((T, Hq + 2 * Hkv, D), generator=g) * 2).cuda()
        pos = torch.cat([torch.arange(n) + c for n, c in zip(lens, ctx)]).to(torch.int32)
        seq = torch.repeat_interleave(torch.arange(2), torch.tensor(lens))
        slots = table.cpu()[seq, pos.long() // page] * page + pos % page
        q = Bn.qk_norm_rope(cache, x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], pos.cuda(),
                            slots.cuda(), f, w[0], w[1], eps)
        cu = torch.tensor([0, lens[0], T], dtype=torch.int32, device="cuda")
        ctx_t = torch.tensor(ctx, dtype=torch.int32, device="cuda")
        if kind == "prompt":
            out = Bn.prompt_attention(cache, q, cu, ctx_t, table)
        else:
            out = Bn.tree_attention(cache, q, cu, ctx_t, table, max(lens))
        b = C.Batch(cache.k, cache.v, q, cu, ctx_t, table, lens, ctx)
        ref, tol = b.reference(D ** -0.5)
        C.assert_within(out, ref, tol, kind)
        ctx = [c + n for c, n in zip(ctx, lens)]
