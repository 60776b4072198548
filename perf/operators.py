"""The attention half of a decoder layer: what is measured of it, and its plain form.

Three operators stand between the q/k/v projections and the output projection:

  norm_rope  RMS norm of every query and key head and the position rotation in one pass; queries
             go to a buffer, keys and values to their slots in the pages of a cache
  tree       attention of a few drafted tokens per sequence (a tree; one token is a tree of one)
             over the pages of the cache
  prompt     causal attention of whole prompts, or of chunks behind a cached prefix, packed one
             after the other, over the pages of the cache

Lengths are written as texts ("5,9,1"), one number a sequence, so that a case is plain values.
"""
import math

import torch

own = False

DEVICE = "cuda" if torch.cuda.is_available() else "cpu"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
EPS = 1e-6


def _norm_rope(name, tokens, heads, kv_heads, dim, page, dtype, in_dtype, norm=True, rot=None,
               interleaved=False, pos0=0, theta=1e6):
    return {"name": name, "op": "norm_rope", "tokens": tokens, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "page": page, "dtype": dtype, "in_dtype": in_dtype,
            "norm": norm, "rot": rot or dim, "interleaved": interleaved, "pos0": pos0,
            "theta": theta}


def _attn(name, op, lens, ctx, heads, kv_heads, dim, page, dtype):
    return {"name": name, "op": op, "lens": ",".join(map(str, lens)),
            "ctx": ",".join(map(str, ctx)), "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "page": page, "dtype": dtype}


def _ints(text):
    return [int(v) for v in text.split(",")]


def listed():
    return [
        # one decoded token, straight from the fp32 outputs of the projections: latency alone
        _norm_rope("norm_rope_token", 1, 32, 8, 128, 64, "bf16", "f32", pos0=4000),
        # the tokens of a verified draft: a small batch far into long texts
        _norm_rope("norm_rope_batch", 33, 32, 8, 128, 16, "bf16", "f32", pos0=900001),
        # an old-style model: no norm, half of each head rotated in neighbouring pairs, odd count
        _norm_rope("norm_rope_partial", 3001, 12, 2, 64, 32, "f16", "f16", norm=False, rot=32,
                   interleaved=True, theta=1e4),
        # a whole prompt of the largest model
        _norm_rope("norm_rope_prompt", 8192, 32, 8, 128, 64, "bf16", "bf16"),
        # one user, one token: the latency of a decode step
        _attn("tree_token", "tree", [1], [3999], 32, 8, 128, 64, "bf16"),
        # a served batch, one token each, contexts of every length
        _attn("tree_batch", "tree", [1] * 32,
              [(37 + 1009 * i * i) % 15991 + 1 for i in range(32)], 32, 8, 128, 64, "bf16"),
        # drafts of several sizes, small pages, grouped heads that are no power of two
        _attn("tree_draft", "tree", [32, 7, 64, 1, 24, 16, 33, 48],
              [4100, 517, 2048, 9000, 63, 0, 3333, 6001], 12, 2, 128, 16, "f16"),
        # drafts behind very long contexts
        _attn("tree_long", "tree", [8, 8, 5, 8], [131000, 131064, 100003, 65536], 32, 8, 128, 64,
              "bf16"),
        # one short question
        _attn("prompt_short", "prompt", [100], [0], 32, 8, 128, 64, "bf16"),
        # many prompts of a served batch, packed
        _attn("prompt_packed", "prompt", [(61 + 577 * i * i) % 1999 + 1 for i in range(16)],
              [0] * 16, 12, 2, 128, 16, "f16"),
        # chunks behind prefixes that the cache holds, narrow heads, none shared
        _attn("prompt_chunk", "prompt", [1024, 2000], [16001, 4096], 16, 16, 64, 32, "bf16"),
        # one long document
        _attn("prompt_long", "prompt", [8192], [0], 32, 8, 128, 128, "bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_rope", "tree", "prompt"])
    heads, kv_heads = rng.choice([(32, 8), (12, 2), (16, 16), (32, 4), (8, 1), (28, 4), (5, 1)])
    dim, page = rng.choice([64, 128]), rng.choice([16, 32, 64, 128])
    dtype = rng.choice(["bf16", "f16"])
    if op == "norm_rope":
        tokens = _log_int(rng, 1, 8192)
        c = _norm_rope("", tokens, heads, kv_heads, dim, page, dtype,
                       rng.choice(["f32", dtype]), rng.random() < 0.7, rng.choice([dim, dim // 2]),
                       rng.random() < 0.4, rng.choice([0, _log_int(rng, 1, 1000000)]),
                       rng.choice([1e4, 1e6]))
        while work(c)["bytes"] > work(listed()[3])["bytes"]:
            c["tokens"] //= 2
    elif op == "tree":
        n = _log_int(rng, 1, 64)
        top = rng.choice([1, 1, 8, 64])
        lens = [rng.randint(1, top) if top > 1 else 1 for _ in range(n)]
        if n > 2 and rng.random() < 0.3:
            lens[rng.randrange(n)] = 0
        far = _log_int(rng, 16, 131072)
        ctx = [rng.choice([0, rng.randint(0, far), far]) if rng.random() < 0.2
               else rng.randint(far // 8, far) for _ in range(n)]
        cap = 4 * 131072 * 8 * 128
        while n * (max(ctx) + 64) * kv_heads * dim > cap:
            ctx = [v // 2 for v in ctx]
        c = _attn("", "tree", lens, ctx, heads, kv_heads, dim, page, dtype)
    else:
        n = _log_int(rng, 1, 16)
        far = _log_int(rng, 8, 8192)
        lens = [_log_int(rng, 1, far) for _ in range(n)]
        lens[rng.randrange(n)] = far
        if n > 2 and rng.random() < 0.3:
            lens[rng.randrange(n)] = 0
        ctx = [0] * n
        if rng.random() < 0.3:
            ctx = [rng.randint(0, 8192) for _ in range(n)]
        cap = 32 * 8192 * 8192
        while (n * heads * max(lens) * (max(lens) + max(ctx)) > cap
               or _pairs(lens, ctx) * heads * dim > _pairs([8192], [0]) * 32 * 128):
            lens, ctx = [(v + 1) // 2 for v in lens], [v // 2 for v in ctx]
        c = _attn("", "prompt", lens, ctx, heads, kv_heads, dim, page, dtype)
    c.pop("name")
    return c


def _pairs(lens, ctx):
    """Visible (query, position) pairs of causal sequences."""
    return sum(n * c + n * (n + 1) // 2 for n, c in zip(lens, ctx))


def work(case):
    h, g, d = case["heads"], case["kv_heads"], case["dim"]
    w = SIZE[case["dtype"]]
    if case["op"] == "norm_rope":
        t = case["tokens"]
        n = t * (h + 2 * g) * d
        return {"bytes": n * (SIZE[case["in_dtype"]] + w) + 8 * t, "flops": 10 * t * (h + g) * d}
    lens, ctx = _ints(case["lens"]), _ints(case["ctx"])
    rows = sum(lens)
    keys = sum(n + c for n, c in zip(lens, ctx) if n)
    pairs = _pairs(lens, ctx) if case["op"] == "prompt" else sum(
        n * (n + c) for n, c in zip(lens, ctx))
    return {"bytes": (2 * keys * g + 2 * rows * h) * d * w, "flops": 4 * pairs * h * d}


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE).manual_seed(seed)
    h, g, d, ps, dt = (case[k] for k in ("heads", "kv_heads", "dim", "page", "dtype"))
    dt = TYPES[dt]

    def normal(*shape, dtype=dt, scale=1.0):
        x = torch.randn(shape, generator=gen, device=DEVICE, dtype=torch.float32)
        return x.mul_(scale).to(dtype)

    def perm(n):
        return torch.randperm(n, generator=gen, device=DEVICE)

    s = {"op": case["op"], "h": h, "g": g, "d": d, "page": ps, "dtype": dt}
    if case["op"] == "norm_rope":
        t, rot, it = case["tokens"], case["rot"], TYPES[case["in_dtype"]]
        n_pages = -(-t // ps) + 3
        s["k_pages"], s["v_pages"] = normal(n_pages, g, ps, d), normal(n_pages, g, ps, d)
        # one row holds the three projections of a token, heads of a few times their norm
        s["qkv"] = normal(t, h + 2 * g, d, dtype=it, scale=3.0)
        ar = torch.arange(t, device=DEVICE)
        s["slots"] = (perm(n_pages)[ar // ps] * ps + ar % ps).to(torch.int32)
        first = torch.randint(0, 1000, (1,), generator=gen, device=DEVICE)
        s["positions"] = (ar + first + case["pos0"]).to(torch.int32)
        s["inv_freq"] = case["theta"] ** (
            -torch.arange(0, rot, 2, device=DEVICE, dtype=torch.float64) / rot)
        s["q_weight"] = (1 + normal(d, dtype=torch.float32, scale=0.2)).to(dt)
        s["k_weight"] = (1 + normal(d, dtype=torch.float32, scale=0.2)).to(dt)
        if not case["norm"]:
            s["q_weight"] = s["k_weight"] = None
        s["rot"], s["interleaved"] = rot, case["interleaved"]
        return s
    lens, ctx = _ints(case["lens"]), _ints(case["ctx"])
    n, rows = len(lens), sum(lens)
    pages = [-(-(a + b) // ps) for a, b in zip(lens, ctx)]
    width, used = max(pages), sum(pages)
    # pages in no order, as a cache hands them out; those that no sequence has hold old values
    s["k_pages"], s["v_pages"] = normal(used + 2, g, ps, d), normal(used + 2, g, ps, d)
    order = perm(used + 2)
    table = torch.zeros((n, width), dtype=torch.int32, device=DEVICE)
    at = 0
    for i, p in enumerate(pages):
        table[i, :p] = order[at:at + p].to(torch.int32)
        at += p
    s["page_table"] = table
    cu = [0]
    for v in lens:
        cu.append(cu[-1] + v)
    s["cu_q"] = torch.tensor(cu, dtype=torch.int32, device=DEVICE)
    s["ctx"] = torch.tensor(ctx, dtype=torch.int32, device=DEVICE)
    s["q"] = normal(rows, h, d, scale=1.5)
    s["scale"] = d ** -0.5
    s["max_q"], s["max_kv"] = max(lens), max(a + b for a, b in zip(lens, ctx))
    s["mask"] = None
    if case["op"] == "tree":
        # bit j of a row's mask: it sees drafted token j; a token sees its ancestors and itself
        import random
        r = random.Random(seed)
        bits = []
        for v in lens:
            tree = []
            for j in range(v):
                up = r.randint(max(-1, j - 4), j - 1)
                tree.append((tree[up] if up >= 0 else 0) | 1 << j)
            bits += [b - (1 << 64) if b >> 63 else b for b in tree]
        s["mask"] = torch.tensor(bits, dtype=torch.int64, device=DEVICE)
    return s


def _plain_norm_rope(s):
    h, g, d, rot = s["h"], s["g"], s["d"], s["rot"]
    x = s["qkv"].float()
    qk, v = x[:, :h + g], x[:, h + g:]
    if s["q_weight"] is not None:
        w = torch.cat([s["q_weight"].float().expand(h, d), s["k_weight"].float().expand(g, d)])
        qk = qk * torch.rsqrt(qk.square().mean(-1, keepdim=True) + EPS) * w
    angle = s["positions"].double()[:, None] * s["inv_freq"]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    if s["interleaved"]:
        a, b = qk[..., 0:rot:2], qk[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = qk[..., :rot // 2], qk[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    qk = torch.cat([turned, qk[..., rot:]], -1).to(s["dtype"])
    slot = s["slots"].long()
    page, at = slot // s["page"], slot % s["page"]
    s["k_pages"][page, :, at] = qk[:, h:]
    s["v_pages"][page, :, at] = v.to(s["dtype"])
    return {"q": qk[:, :h].contiguous(), "k": s["k_pages"], "v": s["v_pages"]}


def _plain_attention(s):
    h, g, d, mq, mk = s["h"], s["g"], s["d"], s["max_q"], s["max_kv"]
    cu, ctx, rows = s["cu_q"].long(), s["ctx"].long(), s["q"].shape[0]
    n = ctx.numel()
    take = (cu[:-1, None] + torch.arange(mq, device=cu.device)).clamp(max=rows - 1)
    q = s["q"].float()[take].view(n, mq, g, h // g, d).permute(0, 2, 1, 3, 4)
    q = q.reshape(n, g, mq * (h // g), d)
    pages = s["page_table"].long()
    k = s["k_pages"][pages].permute(0, 2, 1, 3, 4).reshape(n, g, -1, d)[:, :, :mk].float()
    v = s["v_pages"][pages].permute(0, 2, 1, 3, 4).reshape(n, g, -1, d)[:, :, :mk].float()
    score = (q @ k.transpose(-1, -2)).mul_(s["scale"]).view(n, g, mq, h // g, mk)
    place = torch.arange(mk, device=cu.device) - ctx[:, None]
    if s["mask"] is None:
        seen = place[:, None] <= torch.arange(mq, device=cu.device)[:, None]
    else:
        bit = (s["mask"][take][..., None] >> place[:, None].clamp(0, 63)) & 1
        seen = (place[:, None] < 0) | ((bit == 1) & (place[:, None] < 64))
        seen &= place[:, None] < (cu[1:] - cu[:-1])[:, None, None]
    score.masked_fill_(~seen[:, None, :, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    score.sub_(top.masked_fill(top == -math.inf, 0.0)).exp_()
    total = score.sum(-1, keepdim=True)
    out = score.view(n, g, -1, mk) @ v
    out = (out.view(n, g, mq, h // g, d) / total.clamp_min(1e-30)).to(s["dtype"])
    out = out.permute(0, 2, 1, 3, 4).reshape(n, mq, h, d)
    row = torch.arange(rows, device=cu.device)
    seq = torch.searchsorted(cu, row, right=True) - 1
    return out[seq, row - cu[seq]]


_binding = None


def _framework():
    global _binding
    if _binding is None:
        from quantized_moe_expert_dequant_gb300 import binding
        _binding = binding
    return _binding


def _own_run(s):
    B = _framework()
    if "cache" not in s:
        s["cache"] = B.KvCache(s["k_pages"], s["v_pages"])
    if s["op"] == "norm_rope":
        h, g, x = s["h"], s["g"], s["qkv"]
        q = B.qk_norm_rope(s["cache"], x[:, :h], x[:, h:h + g], x[:, h + g:], s["positions"],
                           s["slots"], s["inv_freq"], q_weight=s["q_weight"],
                           k_weight=s["k_weight"], eps=EPS, interleaved=s["interleaved"])
        return {"q": q, "k": s["k_pages"], "v": s["v_pages"]}
    if s["op"] == "tree":
        return B.tree_attention(s["cache"], s["q"], s["cu_q"], s["ctx"], s["page_table"],
                                max_q=s["max_q"], tree_mask=s["mask"], scale=s["scale"])
    return B.prompt_attention(s["cache"], s["q"], s["cu_q"], s["ctx"], s["page_table"],
                              scale=s["scale"])


def run(state):
    if own:
        return _own_run(state)
    return _plain_norm_rope(state) if state["op"] == "norm_rope" else _plain_attention(state)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm_rope":
        h, g, d, rot = s["h"], s["g"], s["d"], s["rot"]
        parts = []
        for x, w in ((s["qkv"][:, :h], s["q_weight"]), (s["qkv"][:, h:h + g], s["k_weight"])):
            y = x.double()
            if w is not None:
                y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / d + EPS) * w.double()
            first = torch.arange(rot // 2, device=DEVICE)
            first, second = (2 * first, 2 * first + 1) if s["interleaved"] else (
                first, first + rot // 2)
            turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEVICE),
                               torch.outer(s["positions"].double(), s["inv_freq"]))[:, None]
            z = torch.complex(y[..., first], y[..., second]) * turn
            y = y.clone()
            y[..., first], y[..., second] = z.real, z.imag
            parts.append(y)
        k, v = s["k_pages"].double(), s["v_pages"].double()
        for pages, rows in ((k, parts[1]), (v, s["qkv"][:, h + g:].double())):
            flat = pages.transpose(1, 2).reshape(-1, g, d)
            flat[s["slots"].long()] = rows
            pages.copy_(flat.view(pages.shape[0], s["page"], g, d).transpose(1, 2))
        return {"q": parts[0], "k": k, "v": v}
    lens, ctx = _ints(case["lens"]), _ints(case["ctx"])
    per = s["h"] // s["g"]
    if sum(4 * a * (a + b) * s["h"] * s["d"] for a, b in zip(lens, ctx)) > 5e12:
        return None
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEVICE)
    at = 0
    for i, (a, b) in enumerate(zip(lens, ctx)):
        if a == 0:
            continue
        used = s["page_table"][i, :-(-(a + b) // s["page"])].long()
        if s["mask"] is None:
            hidden = torch.ones((a, a), dtype=torch.bool, device=DEVICE).triu(1)
        else:
            m = s["mask"][at:at + a].cpu().tolist()
            hidden = torch.tensor([[not (x >> j) & 1 for j in range(a)] for x in m], device=DEVICE)
        for head in range(s["h"]):
            k = s["k_pages"][used, head // per].reshape(-1, s["d"])[:a + b].double()
            v = s["v_pages"][used, head // per].reshape(-1, s["d"])[:a + b].double()
            e = s["q"][at:at + a, head].double() @ k.T * s["scale"]
            e[:, b:][hidden] = -math.inf
            out[at:at + a, head] = torch.softmax(e, -1) @ v
        at += a
    return out
