"""Inputs and fp64 references of the attention operators (norm and rotation, trees, prompts).

References are the formulas in fp64 over plain lists of positions; they share nothing with the
kernels.  ``attention`` also returns, per output element, how far a kernel may be off:

  u       half a step of the 16-bit type (2^-8 bf16, 2^-11 fp16)
  A       sum_j w_j |v_j|, w the softmax weights
  u |out|           the output's rounding
  u A               each weight p_j is rounded to the 16-bit type before it meets v_j; the kernels
                    may sum p_j before or after that rounding, so the divisor is off by u too: u |out|
  2 e A             e: error of a score's exponent, in numerator and divisor.  A score is a
                    sum of D products in fp32 (one truncation, 2^-23, each), then scaled,
                    shifted (exponents of size x: 2^-23 x) and raised by ex2.approx (2^-22)
  2 n 2^-23 A       sums of n weights and weighted values in fp32
  n 2^-25 max|v|    fp16 only: weights below 2^-14 are subnormal (the divisor is at least about 1);
                    2^-25 is `least`, smaller where the kernels form larger weights
"""
from __future__ import annotations

import dataclasses
import math

import torch

UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def attention(q, k, v, seen, scale, n_sum=None, least=2.0 ** -25):
    """q [R, D], k and v [N, D], seen bool [R, N] -> (out, tolerance) fp64 [R, D]; least: half of fp16's
    least step, relative to a weight that the divisor holds."""
    dt = q.dtype
    u = UNIT[dt]
    qd, kd, vd = q.double(), k.double(), v.double()
    s = (qd @ kd.T) * scale
    s = s.masked_fill(~seen, -math.inf)
    top = s.amax(-1, keepdim=True) if s.shape[1] else torch.full((s.shape[0], 1), -math.inf,
                                                                dtype=torch.float64,
                                                                device=s.device)
    safe = top.masked_fill(top == -math.inf, 0.0)
    p = torch.exp(s - safe)
    l = p.sum(-1, keepdim=True).clamp_min(1e-300)
    w = p / l
    out = w @ vd
    A = w @ vd.abs()
    D, n = q.shape[1], k.shape[0]
    size = (qd.abs() @ kd.abs().T).amax() * scale if n else 0.0
    e = float(size) * (D * 2.0 ** -23 + 4 * 2.0 ** -23) + 2.0 ** -21
    tol = 2 * u * out.abs() + A * (u + 2 * e + 2 * (n + 8) * 2.0 ** -23) + 1e-12
    if dt == torch.float16 and n:
        tol = tol + n * least * vd.abs().amax() + 2.0 ** -25
    return out, tol


@dataclasses.dataclass
class Batch:
    k: torch.Tensor           # [pages, Hkv, page, D]
    v: torch.Tensor
    q: torch.Tensor           # [rows, Hq, D]
    cu: torch.Tensor
    ctx: torch.Tensor
    table: torch.Tensor
    lens: list
    ctxs: list

    def keys(self, i, h):
        n = self.lens[i] + self.ctxs[i]
        ps = self.k.shape[2]
        used = self.table[i, :-(-n // ps)].long()
        D = self.k.shape[3]
        return (self.k[used, h].reshape(-1, D)[:n], self.v[used, h].reshape(-1, D)[:n])

    def reference(self, scale, masks=None, **kw):
        """(out, tol) fp64 [rows, Hq, D]; masks: a list of ints per row, or None: causal."""
        rows, Hq, D = self.q.shape[0], self.q.shape[1], self.q.shape[2]
        G = Hq // self.k.shape[1]
        out = torch.zeros((rows, Hq, D), dtype=torch.float64, device=self.q.device)
        tol = torch.zeros_like(out)
        at = 0
        for i, (n, c) in enumerate(zip(self.lens, self.ctxs)):
            if n == 0:
                continue
            seen = torch.ones((n, c + n), dtype=torch.bool)
            if masks is None:
                seen[:, c:] = torch.ones((n, n), dtype=torch.bool).tril()
            else:
                seen[:, c:] = torch.tensor([[bool(masks[at + r] >> j & 1) for j in range(n)]
                                            for r in range(n)])
            seen = seen.to(self.q.device)
            for h in range(Hq):
                k, v = self.keys(i, h // G)
                out[at:at + n, h], tol[at:at + n, h] = attention(
                    self.q[at:at + n, h], k, v, seen, scale, **kw)
            at += n
        return out, tol


def batch(seed, lens, ctxs, Hq, Hkv, D, page, dtype, extra_pages=2, pad_rows=0, device="cuda",
          stale=float("nan"), q_scale=1.5, token_major=False):
    """Sequences on pages in no order; whatever no sequence owns holds `stale`."""
    gen = torch.Generator(device="cpu").manual_seed(seed)
    need = [-(-(n + c) // page) for n, c in zip(lens, ctxs)]
    n_pages = sum(need) + extra_pages
    order = torch.randperm(n_pages, generator=gen)
    table = torch.full((len(lens), max(max(need), 1)), -1, dtype=torch.int32)
    shape = (n_pages, page, Hkv, D) if token_major else (n_pages, Hkv, page, D)
    k = torch.full(shape, stale, dtype=dtype)
    v = torch.full(shape, stale, dtype=dtype)
    if token_major:
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    at = 0
    for i, (n, c) in enumerate(zip(lens, ctxs)):
        for j in range(need[i]):
            pg = int(order[at])
            at += 1
            table[i, j] = pg
            m = min(page, n + c - j * page)
            k[pg, :, :m] = torch.randn((Hkv, m, D), generator=gen).to(dtype)
            v[pg, :, :m] = torch.randn((Hkv, m, D), generator=gen).to(dtype)
    cu = torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32)
    q = (torch.randn((sum(lens) + pad_rows, Hq, D), generator=gen) * q_scale).to(dtype)
    if device == "cuda":
        kd = torch.empty_strided(k.shape, k.stride(), dtype=dtype, device=device)
        vd = torch.empty_strided(k.shape, k.stride(), dtype=dtype, device=device)
        kd.copy_(k)
        vd.copy_(v)
        k, v = kd, vd
    t = lambda x: x.to(device)
    return Batch(k, v, t(q), t(cu), t(torch.tensor(ctxs, dtype=torch.int32)), t(table),
                 list(lens), list(ctxs))


def assert_within(got, ref, tol, what=""):
    d = (got.double() - ref).abs()
    bad = ~(d <= tol)
    assert not bool(bad.any()), (
        f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((d / tol).nan_to_num(9e9).max()):.3g} "
        f"tolerances at {bad.nonzero()[0].tolist()}: {got[tuple(bad.nonzero()[0])]} for "
        f"{ref[tuple(bad.nonzero()[0])]}")


def norm_rope(x, w, pos, inv_freq, eps, interleaved, dtype):
    """x [T, H, D] -> (y, tolerance) fp64: the norm (w not None), the rotation (inv_freq not None),
    one rounding.  The fp32 path has at most about 32 roundings per element before it (sum of 128
    squares in runs of 16, square root, division, two products, the turn), and sine and cosine
    are off by the angle's rounding (pi 2^-24) and 2 ulp: below 6e-7 together."""
    y = x.double()
    if w is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * w.double()
    size = y.abs()
    if inv_freq is not None:
        R = 2 * inv_freq.numel()
        i = torch.arange(R // 2, device=x.device)
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
        t = pos.double()[:, None, None] * inv_freq
        ya, yb = y[..., a], y[..., b]
        z = y.clone()
        z[..., a] = ya * t.cos() - yb * t.sin()
        z[..., b] = yb * t.cos() + ya * t.sin()
        size = size.clone()
        size[..., a] = ya.abs() + yb.abs()
        size[..., b] = ya.abs() + yb.abs()
        y = z
    tiny = 2.0 ** -25 if dtype == torch.float16 else 1e-38
    return y, UNIT[dtype] * y.abs() * (1 + 1e-5) + size * (32 * 2.0 ** -24 + 6e-7) + tiny
