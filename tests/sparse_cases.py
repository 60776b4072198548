"""References of the calls that go by pages (bounds, selection, attention over listed pages): the
definitions in fp64 over plain lists."""
from __future__ import annotations

import torch

from tests import attention_cases as C


def bounds(b, before):
    """What the bounds are after a call for batch b, from those before."""
    out = before.clone()
    ps = b.k.shape[2]
    for i, (n, c) in enumerate(zip(b.lens, b.ctxs)):
        if n == 0:
            continue
        for j in range(c // ps, (c + n - 1) // ps + 1):
            page = int(b.table[i, j])
            k = b.k[page, :, :min(ps, c + n - j * ps)]
            out[page, :, 0] = k.amin(1)
            out[page, :, 1] = k.amax(1)
    return out


def scores(b, bnd, i, r, h, pages):
    """Exact scores of the first pages of sequence i for row r and key/value head h."""
    per = b.q.shape[1] // b.k.shape[1]
    q = b.q[r, h * per:(h + 1) * per].double()
    lim = bnd[b.table[i, :pages].long(), h].double()
    return torch.maximum(q[:, None] * lim[None, :, 0], q[:, None] * lim[None, :, 1]).sum((0, 2))


def select(b, bnd, n_select, sink, recent):
    rows, Hkv, ps = b.q.shape[0], b.k.shape[1], b.k.shape[2]
    out = torch.full((rows, Hkv, n_select), -7, dtype=torch.int32)
    at = 0
    for i, (n, c) in enumerate(zip(b.lens, b.ctxs)):
        for r in range(n):
            pages = (c + r) // ps + 1
            for h in range(Hkv):
                if pages <= n_select:
                    chosen = list(range(pages))
                else:
                    s = scores(b, bnd, i, at + r, h, pages).tolist()
                    free = sorted(range(sink, pages - recent), key=lambda j: (-s[j], j))
                    chosen = sorted(list(range(sink)) + list(range(pages - recent, pages))
                                    + free[:n_select - sink - recent])
                out[at + r, h] = torch.tensor(chosen + [-1] * (n_select - len(chosen)))
        at += n
    return out


def attention(b, pages, scale):
    """(out, tolerance) fp64 [rows, Hq, D] of rows over their listed pages [rows, Hkv, n]."""
    rows, Hq, D = b.q.shape
    Hkv, ps = b.k.shape[1], b.k.shape[2]
    per = Hq // Hkv
    out = torch.zeros((rows, Hq, D), dtype=torch.float64, device=b.q.device)
    tol = torch.zeros_like(out)
    lists = pages.tolist()
    at = 0
    for i, (n, c) in enumerate(zip(b.lens, b.ctxs)):
        for r in range(n):
            seen = c + r + 1
            for h in range(Hkv):
                own = lists[at + r][h][:(seen - 1) // ps + 1]
                pos = [j * ps + o for j in own if 0 <= j <= (seen - 1) // ps
                       for o in range(min(ps, seen - j * ps))]
                p = torch.tensor(pos, dtype=torch.long, device=b.q.device)
                pg = b.table[i].long()[p // ps]
                k, v = b.k[pg, h, p % ps], b.v[pg, h, p % ps]
                mask = torch.ones((per, len(pos)), dtype=torch.bool, device=b.q.device)
                o, t = C.attention(b.q[at + r, h * per:(h + 1) * per], k, v, mask, scale)
                out[at + r, h * per:(h + 1) * per], tol[at + r, h * per:(h + 1) * per] = o, t
        at += n
    return out, tol


def random_lists(b, n_select, seed, sink=1, recent=1):
    """Lists as a selection gives them, at random."""
    gen = torch.Generator().manual_seed(seed)
    rows, Hkv, ps = b.q.shape[0], b.k.shape[1], b.k.shape[2]
    out = torch.full((rows, Hkv, n_select), -1, dtype=torch.int32)
    at = 0
    for n, c in zip(b.lens, b.ctxs):
        for r in range(n):
            pages = (c + r) // ps + 1
            for h in range(Hkv):
                if pages <= n_select:
                    own = list(range(pages))
                else:
                    free = torch.randperm(pages - sink - recent, generator=gen) + sink
                    own = sorted(list(range(sink)) + free[:n_select - sink - recent].tolist()
                                 + list(range(pages - recent, pages)))
                out[at + r, h, :len(own)] = torch.tensor(own, dtype=torch.int32)
        at += n
    return out.to(b.q.device)
