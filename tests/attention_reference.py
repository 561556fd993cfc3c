"""Attention and its gradient in 64 bits, with bounds on what a kernel that
sums in 32 bits may differ by.

Bounds, per value: a score x = scale q . k of D float32 products is off by
ex = scale (D + 2) 2^-24 |q| |k|, its exponential by a relative 2 ex + 2^-22
(the exponent's own rounding and the exponential's last bits), and a sum of n
terms by n 2^-24 of the terms' magnitudes.  With bf16 inputs probabilities (and
dS) may be rounded to bf16, 2^-8 of each term, and the stored out that the
gradient reads is rounded, 2^-8 of each value.  The result's own rounding, half
a step, comes on top.  What lies below the smallest normal number, 2^-126, may be
taken as zero, a probability as well as a product with one: 2^-126 times what
it is multiplied with, and 2^-126 for the product.
"""

import math

import torch

U = 2.0 ** -24
TINY = 2.0 ** -126
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def attend(q, k, v, scale, causal, dout=None):
    """One sequence: q, dout [m, H, D], k, v [n, Hk, D] of the call's dtype.
    A dict of float64 results and another of the bounds on them."""
    half = HALF[q.dtype]
    rounded = half if q.dtype == torch.bfloat16 else 0.0
    m, heads, d = q.shape
    n, kvh, _ = k.shape
    g = heads // kvh
    q64, k64, v64 = (t.double().transpose(0, 1).contiguous() for t in (q, k, v))
    k64, v64 = k64.repeat_interleave(g, 0), v64.repeat_interleave(g, 0)
    kt, vt = k64.transpose(1, 2).contiguous(), v64.transpose(1, 2).contiguous()
    x = scale * torch.matmul(q64, kt)
    if causal:
        seen = torch.arange(n, device=q.device)[None] <= torch.arange(m, device=q.device)[:, None] + n - m
        x = x.masked_fill(~seen, -math.inf)
    lse = torch.logsumexp(x, -1) if n else torch.full((heads, m), -math.inf, dtype=torch.float64, device=q.device)
    p = torch.exp(x - torch.where(torch.isinf(lse), 0.0, lse)[..., None])
    out = torch.matmul(p, v64)
    ex = scale * (d + 2) * U * q64.norm(dim=-1)[..., None] * (k64.norm(dim=-1)[:, None] if n else 0.0)
    worst = ex.amax(-1, keepdim=True) if n else ex.sum(-1, keepdim=True)
    ep = 2 * (ex + worst) + 2 * 2.0 ** -22 + n * U  # a probability's relative error, its row's sum included
    res = {"out": out, "lse": lse}
    tol = {"out": torch.matmul(p * (ep + rounded + n * U) + TINY, v64.abs()) + half * out.abs() + (n + 1) * TINY,
           "lse": worst.squeeze(-1) + (n + 4) * U + 2.0 ** -22 + 2.0 ** -22 * torch.nan_to_num(lse, neginf=0.0).abs()}
    if dout is not None:
        do = dout.double().transpose(0, 1).contiguous()
        dp = torch.matmul(do, vt)
        dot = (do * out).sum(-1, keepdim=True)
        ds = p * (dp - dot)
        edp = (d + 2) * U * do.norm(dim=-1)[..., None] * (v64.norm(dim=-1)[:, None] if n else 0.0)
        edot = (do.abs() * (tol["out"] + d * U * out.abs())).sum(-1, keepdim=True)
        es = (ep + 2.0 ** -22) * ds.abs() + p * (edp + edot + 4 * U * (dp.abs() + dot.abs())) + rounded * ds.abs()
        es = es + TINY * (dp.abs() + dot.abs() + 1.0)

        def over_group(t):
            return t.view(kvh, g, n, d).sum(1)

        res["dq"] = scale * torch.matmul(ds, k64)
        tol["dq"] = scale * torch.matmul(es + n * U * ds.abs(), k64.abs()) + half * res["dq"].abs()
        dst, pt, est = (t.transpose(1, 2).contiguous() for t in (ds, p, es))
        ept = (p * (ep + rounded) + TINY).transpose(1, 2).contiguous()
        res["dk"] = scale * over_group(torch.matmul(dst, q64))
        tol["dk"] = scale * over_group(torch.matmul(est + g * m * U * dst.abs(), q64.abs())) + half * res["dk"].abs()
        res["dv"] = over_group(torch.matmul(pt, do))
        tol["dv"] = over_group(torch.matmul(ept + g * m * U * pt, do.abs())) + half * res["dv"].abs()
        for name, terms in (("dq", n), ("dk", g * m), ("dv", g * m)):
            tol[name] = tol[name] + (terms + 1) * TINY
    rows_first = {name: t.transpose(0, 1) for name, t in res.items()}
    return rows_first, {name: t.transpose(0, 1) for name, t in tol.items()}


def close(got, want, tol, what):
    """got is within tol of want, infinities equal."""
    same = got.double() == want
    err = torch.where(same, 0.0, (got.double() - want).abs())
    bad = ~(err <= tol)
    assert not bad.any(), (what, int(bad.sum()), float((err / tol)[bad].max()), err[bad][:4].tolist(), tol[bad][:4].tolist())
