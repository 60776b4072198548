"""Attention over a cache of pages that does not read all of it for every token: what is measured of
it, and its plain form.

  prefix  attention of decoded or drafted tokens of a batch whose sequences share their first pages
          (a system prompt, a document): the shared pages are read once for all
  bounds  the least and the largest key of a page in every dimension, kept up as tokens are added
  select  for each token and key/value head the pages whose bounds allow the largest scores, among
          them always the first and the last
  sparse  attention of tokens over the pages that were selected for each of them

Lengths are written as texts ("5,9,1"), one number a sequence or group, so that a case is plain
values.
"""
import math
import random

import torch

own = False

DEVICE = "cuda" if torch.cuda.is_available() else "cpu"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
SIZE = 2  # bytes of an element of either
SINK, RECENT = 1, 2


def _text(values):
    return ",".join(map(str, values))


def _ints(text):
    return [int(v) for v in text.split(",")]


def _prefix(name, groups, prefix, lens, after, heads, kv_heads, dim, page, dtype):
    """groups: sequences of each; prefix: positions that a group shares; lens: drafted tokens of
    each sequence; after: positions between the prefix and those."""
    return {"name": name, "op": "prefix", "groups": _text(groups), "prefix": _text(prefix),
            "lens": _text(lens), "after": _text(after), "heads": heads, "kv_heads": kv_heads,
            "dim": dim, "page": page, "dtype": dtype}


def _rows(name, op, lens, ctx, heads, kv_heads, dim, page, dtype, select=0):
    return {"name": name, "op": op, "lens": _text(lens), "ctx": _text(ctx), "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "page": page, "dtype": dtype, "select": select}


def listed():
    spread = [(37 + 1009 * i * i) % 30991 + 1000 for i in range(32)]
    return [
        # four short answers behind a short system prompt: latency alone
        _prefix("prefix_few", [4], [512], [1] * 4, [9, 33, 70, 1], 12, 2, 128, 16, "f16"),
        # a served batch, one token each, behind one long system prompt
        _prefix("prefix_batch", [64], [8192], [1] * 64,
                [(61 + 577 * i * i) % 999 + 1 for i in range(64)], 32, 8, 128, 64, "bf16"),
        # drafts of several sizes in three groups, one of them a sequence alone; ragged prefixes;
        # heads that are not shared
        _prefix("prefix_groups", [24, 7, 1], [4096, 2016, 130], [1 + i % 8 for i in range(32)],
                [(29 + 131 * i * i) % 700 for i in range(32)], 16, 16, 64, 32, "f16"),
        # questions about one book, drafts of eight tokens
        _prefix("prefix_book", [32], [65536], [8] * 32, [100 * i for i in range(32)], 32, 8, 128,
                64, "bf16"),
        # one new token for each sequence of a batch: only its last page changes
        _rows("bounds_token", "bounds", [1] * 32, spread, 32, 8, 128, 64, "bf16"),
        # the pages of prompts that have just been written, one of them behind a prefix
        _rows("bounds_prompt", "bounds", [8192, 1001, 37], [0, 77, 5000], 12, 2, 64, 16, "f16"),
        # one user far into a long text
        _rows("select_token", "select", [1], [131000], 32, 8, 128, 64, "bf16", 32),
        # a served batch, contexts of every length
        _rows("select_batch", "select", [1] * 32, spread, 32, 8, 128, 64, "bf16", 32),
        # the next chunk of a long document, small pages
        _rows("select_chunk", "select", [500, 12], [32001, 9000], 12, 2, 64, 16, "f16", 100),
        # one user: 32 of 2047 pages
        _rows("sparse_token", "sparse", [1], [131000], 32, 8, 128, 64, "bf16", 32),
        # a served batch, some contexts shorter than what may be selected
        _rows("sparse_batch", "sparse", [1] * 32, spread, 32, 8, 128, 64, "bf16", 32),
        # the next chunk of a long document, narrow heads, small pages
        _rows("sparse_chunk", "sparse", [500, 12], [32001, 9000], 12, 2, 64, 16, "f16", 100),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _largest(op):
    found = [work(c) for c in listed() if c["op"] == op]
    return {k: max(w[k] for w in found) for k in ("bytes", "flops")}


def draw(rng):
    op = rng.choice(["prefix", "prefix", "bounds", "select", "sparse"])
    heads, kv_heads = rng.choice([(32, 8), (12, 2), (16, 16), (32, 4), (8, 1), (28, 4), (5, 1)])
    dim, page = rng.choice([64, 128]), rng.choice([16, 32, 64, 128])
    dtype = rng.choice(["bf16", "f16"])
    top = _largest(op)
    if op == "prefix":
        groups = [_log_int(rng, 1, 64) for _ in range(rng.choice([1, 1, 2, 5]))]
        n = sum(groups)
        prefix = [_log_int(rng, 16, 65536) for _ in groups]
        most = rng.choice([1, 1, 8, 24])
        lens = [rng.randint(1, most) for _ in range(n)]
        if n > 2 and rng.random() < 0.3:
            lens[rng.randrange(n)] = 0
        far = _log_int(rng, 4, 4096)
        after = [rng.choice([0, far]) if rng.random() < 0.2 else rng.randint(0, far)
                 for _ in range(n)]
        while True:
            c = _prefix("", groups, prefix, lens, after, heads, kv_heads, dim, page, dtype)
            w = work(c)
            # (what the plain form holds at a time counts too)
            if (w["flops"] <= top["flops"] and w["bytes"] <= top["bytes"]
                    and n * max(lens) * heads * (max(prefix) + max(after)) <= 2 ** 30):
                break
            prefix, after = [max(v // 2, 16) for v in prefix], [v // 2 for v in after]
            lens = [(v + 1) // 2 for v in lens]
    else:
        chunk = rng.random() < 0.4
        n = _log_int(rng, 1, 4 if chunk else 64)
        most = _log_int(rng, 2, 8192 if op == "bounds" else 512) if chunk else 1
        lens = [rng.randint(1, most) for _ in range(n)]
        if n > 2 and rng.random() < 0.3:
            lens[rng.randrange(n)] = 0
        far = _log_int(rng, 16 * page if op == "select" else 16, 131072)
        ctx = [rng.choice([0, far]) if rng.random() < 0.2 else rng.randint(far // 8, far)
               for _ in range(n)]
        longest = rng.randrange(n)
        ctx[longest], lens[longest] = far, max(lens[longest], 1)
        select = SINK + RECENT + _log_int(rng, 1, 4096 // page)
        while True:
            if op == "select":  # (nothing to select from otherwise)
                select = min(select, max(SINK + RECENT + 1, ctx[longest] // page // 2))
            c = _rows("", op, lens, ctx, heads, kv_heads, dim, page, dtype,
                      0 if op == "bounds" else select)
            w = work(c)
            held = sum(a + b for a, b in zip(lens, ctx)) * kv_heads * dim
            if (w["flops"] <= top["flops"] and w["bytes"] <= top["bytes"]
                    and held <= 33 * 32768 * 8 * 128):
                break
            ctx, lens = [v // 2 for v in ctx], [(v + 1) // 2 for v in lens]
    c.pop("name")
    return c


def _shared(case):
    """Positions on shared pages: whole pages of each group's prefix."""
    return [v // case["page"] * case["page"] for v in _ints(case["prefix"])]


def _contexts(case):
    """Of a prefix case: positions before the drafted tokens, and of these on shared pages."""
    ctx, shared, after = [], [], _ints(case["after"])
    for n, pre, p in zip(_ints(case["groups"]), _ints(case["prefix"]), _shared(case)):
        for _ in range(n):
            shared.append(p)
            ctx.append(pre + after[len(ctx)])
    return ctx, shared


def work(case):
    h, g, d, ps = case["heads"], case["kv_heads"], case["dim"], case["page"]
    lens = _ints(case["lens"])
    rows = sum(lens)
    if case["op"] == "prefix":
        ctx, shared = _contexts(case)
        keys = sum(_shared(case)) + sum(n + c - p for n, c, p in zip(lens, ctx, shared) if n)
        pairs = sum(n * (n + c) for n, c in zip(lens, ctx))
        return {"bytes": (2 * keys * g + 2 * rows * h) * d * SIZE, "flops": 4 * pairs * h * d}
    ctx = _ints(case["ctx"])
    if case["op"] == "bounds":
        keys = pages = 0
        for n, c in zip(lens, ctx):
            if n:
                keys += n + c % ps
                pages += (c + n - 1) // ps - c // ps + 1
        return {"bytes": (keys + 2 * pages) * g * d * SIZE, "flops": 2 * keys * g * d}
    k = case["select"]
    seen = [[(c + i) // ps + 1 for i in range(n)] for n, c in zip(lens, ctx)]
    if case["op"] == "select":
        pages = sum(max(s) for s in seen if s)
        return {"bytes": (2 * pages * g + rows * h) * d * SIZE + 4 * rows * g * k,
                "flops": 4 * sum(map(sum, seen)) * g * d}
    listed_pages = sum(min(k, p) for s in seen for p in s)
    union = sum(min(max(s), sum(min(k, p) for p in s)) for s in seen if s)
    return {"bytes": (2 * union * ps * g + 2 * rows * h) * d * SIZE + 4 * listed_pages * g,
            "flops": 4 * listed_pages * ps * h * d}


def _normal(gen, shape, dtype, scale=1.0):
    x = torch.randn(shape, generator=gen, device=DEVICE, dtype=torch.float32)
    return x.mul_(scale).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE).manual_seed(seed)
    h, g, d, ps = (case[k] for k in ("heads", "kv_heads", "dim", "page"))
    dt, op, lens = TYPES[case["dtype"]], case["op"], _ints(case["lens"])
    n, rows = len(lens), sum(lens)
    s = {"op": op, "h": h, "g": g, "d": d, "page": ps, "dtype": dt, "rows": rows, "max_q": max(lens)}
    if op == "prefix":
        ctx, shared = _contexts(case)
    else:
        ctx, shared = _ints(case["ctx"]), [0] * n
    need = [-(-(a + b) // ps) for a, b in zip(lens, ctx)]
    first = [v // ps for v in shared]  # pages that the sequence shares
    total = sum(a - b for a, b in zip(need, first))
    if op == "prefix":
        total += sum(v // ps for v in _shared(case))
    # pages in no order, as a cache hands them out; those that no sequence has hold old values
    order = torch.randperm(total + 2, generator=gen, device=DEVICE).to(torch.int32)
    table = torch.zeros((n, max(need)), dtype=torch.int32, device=DEVICE)
    at = 0
    if op == "prefix":
        seq = 0
        for count, p in zip(_ints(case["groups"]), _shared(case)):
            table[seq:seq + count, :p // ps] = order[at:at + p // ps]
            at += p // ps
            seq += count
    for i in range(n):
        m = need[i] - first[i]
        table[i, first[i]:need[i]] = order[at:at + m]
        at += m
    s["page_table"] = table
    cu = [0]
    for v in lens:
        cu.append(cu[-1] + v)
    s["cu_q"] = torch.tensor(cu, dtype=torch.int32, device=DEVICE)
    s["ctx"] = torch.tensor(ctx, dtype=torch.int32, device=DEVICE)
    s["max_kv"] = max(a + b for a, b in zip(lens, ctx))
    shape = (total + 2, g, ps, d)
    if op == "select":  # reads no keys, only their bounds
        s["k_pages"] = s["v_pages"] = torch.empty(shape, dtype=dt, device=DEVICE)
    else:
        # keys of a text: a direction that its page has, and the token's own
        s["k_pages"] = (_normal(gen, shape, dt, 0.8)
                        .add_(_normal(gen, (total + 2, g, 1, d), dt, 0.6)))
        s["v_pages"] = _normal(gen, shape, dt) if op != "bounds" else s["k_pages"]
    if op in ("bounds", "select"):
        middle = _normal(gen, (total + 2, g, d), torch.float32, 0.6)
        reach = 0.8 * (ps ** 0.2 + 0.3 * torch.rand((total + 2, g, 2, d), generator=gen,
                                                    device=DEVICE))
        sign = torch.tensor([-1.0, 1.0], device=DEVICE)[:, None]
        s["bounds"] = (middle[:, :, None] + sign * reach).to(dt)
    if op != "bounds":
        s["q"] = _normal(gen, (rows, h, d), dt, 1.5)
    s["scale"], s["select"] = d ** -0.5, case.get("select", 0)
    s["mask"] = None
    if op == "prefix":
        groups = _ints(case["groups"])
        s["groups"], s["shared"] = groups, _shared(case)
        cu_group = [0]
        for v in groups:
            cu_group.append(cu_group[-1] + v)
        s["cu_group"] = torch.tensor(cu_group, dtype=torch.int32, device=DEVICE)
        s["prefix_len"] = torch.tensor(_ints(case["prefix"]), dtype=torch.int32, device=DEVICE)
        s["after"] = max([b + a - p for a, b, p in zip(lens, ctx, shared)])
        # bit j of a row's mask: it sees drafted token j; a token sees its ancestors and itself
        r = random.Random(seed)
        bits = []
        for v in lens:
            tree = []
            for j in range(v):
                up = r.randint(max(-1, j - 4), j - 1)
                tree.append((tree[up] if up >= 0 else 0) | 1 << j)
            bits += tree
        if max(lens) > 1:
            s["mask"] = torch.tensor(bits, dtype=torch.int64, device=DEVICE)
    if op == "sparse":
        # what a selection gives: the first page and the last, and between them pages that the
        # tokens of a sequence mostly agree about
        row = torch.arange(rows, device=DEVICE)
        seq = torch.searchsorted(s["cu_q"].long(), row, right=True) - 1
        last = (s["ctx"].long()[seq] + row - s["cu_q"].long()[seq]) // ps
        width, k = table.shape[1], case["select"]
        page = torch.arange(width, device=DEVICE)
        score = torch.randn((n, g, width), generator=gen, device=DEVICE)[seq]
        score += 0.7 * torch.randn((rows, g, width), generator=gen, device=DEVICE)
        score[..., :SINK] = 100.0
        end = last[:, None, None]
        score = torch.where((page > end - RECENT) & (page <= end), 200.0, score)
        score = score.masked_fill(page > end, -math.inf)
        top, at = score.topk(min(k, width), dim=-1)
        at = torch.where(top == -math.inf, 2 ** 31 - 1, at).sort(-1).values
        pages = torch.full((rows, g, k), -1, dtype=torch.int32, device=DEVICE)
        pages[..., :at.shape[-1]] = torch.where(at == 2 ** 31 - 1, -1, at).to(torch.int32)
        s["pages"] = pages
    return s


def _row_places(s):
    """Sequence and position of every row."""
    cu = s["cu_q"].long()
    row = torch.arange(s["rows"], device=cu.device)
    seq = torch.searchsorted(cu, row, right=True) - 1
    return seq, s["ctx"].long()[seq] + row - cu[seq]


def _softmax_parts(score):
    top = score.amax(-1, keepdim=True)
    p = score.sub_(top.masked_fill(top == -math.inf, 0.0)).exp_()
    return p, p.sum(-1, keepdim=True).clamp_min(1e-30)


def _plain_prefix(s):
    h, g, d, mq, ps = s["h"], s["g"], s["d"], s["max_q"], s["page"]
    cu, ctx, rows, per = s["cu_q"].long(), s["ctx"].long(), s["rows"], s["h"] // s["g"]
    out = torch.empty((rows, h, d), dtype=s["dtype"], device=cu.device)
    tokens, seq = torch.arange(mq, device=cu.device), 0
    for count, shared in zip(s["groups"], s["shared"]):
        a, b = seq, seq + count
        seq = b
        start, n_q = cu[a:b], cu[a + 1:b + 1] - cu[a:b]
        take = (start[:, None] + tokens).clamp(max=rows - 1)
        q = s["q"].float()[take].view(count, mq, g, per, d).permute(2, 0, 1, 3, 4)
        pages = s["page_table"][a, :shared // ps].long()  # once for the group
        kp = s["k_pages"][pages].permute(1, 0, 2, 3).reshape(g, shared, d).float()
        vp = s["v_pages"][pages].permute(1, 0, 2, 3).reshape(g, shared, d).float()
        first = (q.reshape(g, -1, d) @ kp.transpose(1, 2)).view(g, count, mq * per, shared)
        pages = s["page_table"][a:b, shared // ps:].long()
        ko = s["k_pages"][pages].permute(2, 0, 1, 3, 4).reshape(g, count, -1, d)[:, :, :s["after"]]
        vo = s["v_pages"][pages].permute(2, 0, 1, 3, 4).reshape(g, count, -1, d)[:, :, :s["after"]]
        m = ko.shape[2]
        rest = q.reshape(g, count, mq * per, d) @ ko.float().transpose(2, 3)
        place = shared + torch.arange(m, device=cu.device) - ctx[a:b, None]
        if s["mask"] is None:
            seen = place[:, None] <= tokens[:, None]
        else:
            bit = (s["mask"][take][..., None] >> place[:, None].clamp(0, 63)) & 1
            seen = (place[:, None] < 0) | ((bit == 1) & (place[:, None] < 64))
        seen = seen & (place < n_q[:, None])[:, None]
        rest.view(g, count, mq, per, m).masked_fill_(~seen[None, :, :, None], -math.inf)
        p, total = _softmax_parts(torch.cat([first, rest], -1).mul_(s["scale"]))
        o = (p[..., :shared].reshape(g, count * mq * per, shared) @ vp).view(g, count, mq * per, d)
        o = (o + p[..., shared:] @ vo.float()) / total
        o = o.view(g, count, mq, per, d).permute(1, 2, 0, 3, 4).reshape(count, mq, h, d)
        used = tokens < n_q[:, None]
        out[take[used]] = o[used].to(s["dtype"])
    return out


def _plain_bounds(s):
    ps, cu, ctx = s["page"], s["cu_q"].long(), s["ctx"].long()
    end = ctx + cu[1:] - cu[:-1]
    page = torch.arange(s["page_table"].shape[1], device=cu.device)
    new = ((page + 1) * ps > ctx[:, None]) & (page * ps < end[:, None]) & (end > ctx)[:, None]
    seq, page = new.nonzero(as_tuple=True)
    held = s["page_table"][seq, page].long()
    inside = page[:, None] * ps + torch.arange(ps, device=cu.device) < end[seq, None]
    k = s["k_pages"][held].float()
    hidden = ~inside[:, None, :, None]
    s["bounds"][held, :, 0] = k.masked_fill(hidden, math.inf).amin(2).to(s["dtype"])
    s["bounds"][held, :, 1] = k.masked_fill(hidden, -math.inf).amax(2).to(s["dtype"])
    return s["bounds"]


def _plain_select(s):
    g, d, ps, k, mq, rows = s["g"], s["d"], s["page"], s["select"], s["max_q"], s["rows"]
    cu, tokens = s["cu_q"].long(), torch.arange(s["max_q"], device=s["cu_q"].device)
    take = (cu[:-1, None] + tokens).clamp(max=rows - 1)
    used = tokens < (cu[1:] - cu[:-1])[:, None]
    last = ((s["ctx"].long()[:, None] + tokens) // ps)[:, None, :, None]
    pages = torch.full((rows, g, k), -1, dtype=torch.int32, device=cu.device)
    # in 64 bits: the order of two pages may hang on the last bit
    q = s["q"].double().view(rows, g, -1, d)
    up, down = q.clamp(min=0).sum(2), q.clamp(max=0).sum(2)
    both = torch.cat([down, up], -1)[take].transpose(1, 2)  # [n, g, mq, 2 d], as (least, largest)
    limit = s["bounds"][s["page_table"].long()].double()  # [n, pages, g, 2, d]
    score = both @ limit.permute(0, 2, 3, 4, 1).reshape(len(cu) - 1, g, 2 * d, -1)
    page = torch.arange(score.shape[-1], device=cu.device)
    score[..., :SINK] = math.inf
    score.masked_fill_(page > last - RECENT, math.inf).masked_fill_(page > last, -math.inf)
    # stable: of equal scores the lower page
    top, at = score.sort(dim=-1, descending=True, stable=True)
    top, at = top[..., :k], at[..., :k]
    at = torch.where(top == -math.inf, 2 ** 31 - 1, at).sort(-1).values
    at = torch.where(at == 2 ** 31 - 1, -1, at).to(torch.int32).transpose(1, 2)
    pages[take[used], :, :at.shape[-1]] = at[used]
    return pages


def _plain_sparse(s):
    h, g, d, ps = s["h"], s["g"], s["d"], s["page"]
    seq, position = _row_places(s)
    out = torch.empty((s["rows"], h, d), dtype=s["dtype"], device=seq.device)
    head = torch.arange(g, device=seq.device)[:, None]
    step = max(1, 2 ** 28 // (g * s["select"] * ps * d))  # rows at a time
    for a in range(0, s["rows"], step):
        pages = s["pages"][a:a + step].long()
        held = s["page_table"][seq[a:a + step, None, None], pages.clamp(min=0)].long()
        n = pages.shape[0]
        k = s["k_pages"][held, head].reshape(n, g, -1, d).float()
        v = s["v_pages"][held, head].reshape(n, g, -1, d).float()
        at = pages[..., None] * ps + torch.arange(ps, device=seq.device)
        seen = (pages[..., None] >= 0) & (at <= position[a:a + step, None, None, None])
        q = s["q"][a:a + step].float().view(n, g, -1, d)
        score = (q @ k.transpose(2, 3)).mul_(s["scale"])
        p, total = _softmax_parts(score.masked_fill_(~seen.view(n, g, 1, -1), -math.inf))
        out[a:a + step] = (p @ v / total).view(n, h, d).to(s["dtype"])
    return out


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
    batch = s["cu_q"], s["ctx"], s["page_table"]
    if s["op"] == "prefix":
        return B.prefix_attention(s["cache"], s["q"], *batch, s["cu_group"], s["prefix_len"],
                                  max_q=s["max_q"], tree_mask=s["mask"], scale=s["scale"])
    if s["op"] == "bounds":
        return B.page_bounds(s["cache"], s["bounds"], *batch, n_rows=s["rows"])
    if s["op"] == "select":
        return B.select_pages(s["cache"], s["bounds"], s["q"], *batch, n_select=s["select"],
                              sink=SINK, recent=RECENT)
    return B.sparse_attention(s["cache"], s["q"], *batch, s["pages"], scale=s["scale"])


def run(state):
    if own:
        return _own_run(state)
    return {"prefix": _plain_prefix, "bounds": _plain_bounds, "select": _plain_select,
            "sparse": _plain_sparse}[state["op"]](state)


def exact(case, seed):
    s = prepare(case, seed)
    h, g, d, ps = s["h"], s["g"], s["d"], s["page"]
    per, lens = h // g, _ints(case["lens"])
    cu, ctx = s["cu_q"].tolist(), s["ctx"].tolist()
    table = s["page_table"].long()
    if case["op"] == "prefix":
        out = torch.zeros((s["rows"], h, d), dtype=torch.float64, device=DEVICE)
        for i, n in enumerate(lens):
            if n == 0:
                continue
            a, c = cu[i], ctx[i]
            used = table[i, :-(-(n + c) // ps)]
            hidden = torch.ones((n, n), dtype=torch.bool, device=DEVICE).triu(1)
            if s["mask"] is not None:
                bits = s["mask"][a:a + n].tolist()
                hidden = torch.tensor([[not (x >> j) & 1 for j in range(n)] for x in bits],
                                      device=DEVICE)
            for head in range(g):
                k = s["k_pages"][used, head].reshape(-1, d)[:n + c].double()
                v = s["v_pages"][used, head].reshape(-1, d)[:n + c].double()
                q = s["q"][a:a + n, head * per:(head + 1) * per].double()
                e = torch.einsum("nhd,kd->hnk", q, k) * s["scale"]
                e[:, :, c:].masked_fill_(hidden, -math.inf)
                o = torch.einsum("hnk,kd->nhd", torch.softmax(e, -1), v)
                out[a:a + n, head * per:(head + 1) * per] = o
        return out
    if case["op"] == "bounds":
        out, want = s["bounds"].double(), []
        for i, n in enumerate(lens):
            want += [(i, j, min(ps, ctx[i] + n - j * ps))
                     for j in range(ctx[i] // ps, (ctx[i] + n - 1) // ps + 1) if n]
        index = table.tolist()
        for size in {w[2] for w in want}:  # pages filled alike
            held = torch.tensor([index[i][j] for i, j, m in want if m == size], device=DEVICE)
            k = s["k_pages"][held, :, :size].double()
            out[held] = torch.stack([k.min(2).values, k.max(2).values], 2)
        return out
    if case["op"] == "select":
        k = case["select"]
        pages = torch.full((s["rows"], g, k), -1, dtype=torch.int32, device=DEVICE)
        for i, n in enumerate(lens):
            for r in range(0, n, 16):
                m = min(16, n - r)
                count = (ctx[i] + r + m - 1) // ps + 1
                limit = s["bounds"][table[i, :count]].double()
                rows = slice(cu[i] + r, cu[i] + r + m)
                q = s["q"][rows].double().view(m, g, per, d)
                score = torch.zeros((m, g, count), dtype=torch.float64, device=DEVICE)
                for head in range(per):
                    x = q[:, :, head, None]
                    for c in range(0, count, 512):
                        lo, hi = (limit[c:c + 512, :, e].transpose(0, 1) for e in (0, 1))
                        score[:, :, c:c + 512] += torch.maximum(x * lo, x * hi).sum(-1)
                for t in range(m):
                    own_count = (ctx[i] + r + t) // ps + 1
                    forced = [j for j in range(own_count)
                              if j < SINK or j >= own_count - RECENT]
                    free = torch.arange(SINK, max(own_count - RECENT, SINK), device=DEVICE)
                    left = min(k - len(forced), len(free))
                    if left <= 0:
                        chosen = torch.tensor(forced, device=DEVICE).expand(g, -1)
                    else:
                        best = score[t][:, free].sort(dim=-1, descending=True, stable=True).indices
                        chosen = torch.cat([torch.tensor(forced, device=DEVICE).expand(g, -1),
                                            free[best[:, :left]]], 1).sort(-1).values
                    pages[cu[i] + r + t, :, :chosen.shape[1]] = chosen.to(torch.int32)
        return pages
    out = torch.zeros((s["rows"], h, d), dtype=torch.float64, device=DEVICE)
    lists = s["pages"].tolist()
    for i, n in enumerate(lens):
        for r in range(cu[i], cu[i] + n):
            limit = ctx[i] + r - cu[i] + 1
            for head in range(g):
                used = torch.tensor([j for j in lists[r][head] if j >= 0], device=DEVICE)
                at = (used[:, None] * ps + torch.arange(ps, device=DEVICE)).flatten()
                keep = at < limit
                k = s["k_pages"][table[i, used], head].reshape(-1, d)[keep].double()
                v = s["v_pages"][table[i, used], head].reshape(-1, d)[keep].double()
                q = s["q"][r, head * per:(head + 1) * per].double()
                out[r, head * per:(head + 1) * per] = torch.softmax(q @ k.T * s["scale"], -1) @ v
    return out
