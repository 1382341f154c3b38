"""Plain 64-bit forms of the tuning operators (CPU, torch) and what their errors may be.

An fp32 addition is taken at one unit in the last place (2^-23: the matrix cores are not
assumed to round to nearest), products of 16-bit numbers are exact.

The transposed product.  With Smax_r the row's largest scale and e_r its exponent, the kernel's
weights are S (u - z) 2^-e_r (two fp32 roundings, 2^-23) in one fp16 part (half a step: 2^-12,
or half a subnormal step: 2^-25 of 2^e_r <= Smax_r) or in two (the second is half a step off
what the first leaves, 2^-24; 2^-23 with the fp32 roundings: together 2^-22).  An element of
dy that fp16 does not hold is off by half a subnormal step, 2^-25 where the row's largest
dy 2^e is at least 2^14: 2^-39 of it.  d_row + 64 additions (64: pieces, scaling)."""
from __future__ import annotations

import torch

from oracle import gptq_oracle as o
from serving_helpers import BF, F32, HF, out_rounding, zero_parts  # noqa: F401

U = 2.0 ** -23


def segments(offsets, n):
    """(expert, first row, end) as the operators take the offsets: clamped, never falling."""
    if offsets is None:
        return [(0, 0, n)]
    run, out = min(max(int(offsets[0]), 0), n), []
    for e, v in enumerate(offsets[1:]):
        end = max(run, min(max(int(v), 0), n))
        out.append((e, run, end))
        run = end
    return out


def layer_parts(q):
    """(Smax, 2^e) of every row."""
    S = q.scales.cpu().double().abs().amax(1)
    e = torch.floor(torch.log2(torch.where(S > 0, S, 1.0)))
    return S, 2.0 ** e


def weight_rel(t):
    """Relative error of a weight of the transposed product by the output's type."""
    return 2.0 ** -12 + U if t == BF else 2.0 ** -22


def back_reference(q, What, dy, out_t):
    """dx and its bound, one expert."""
    dy = dy.cpu().double()
    S, p2 = layer_parts(q)
    ref, mag = dy @ What, dy.abs() @ What.abs()
    bound = ((What.shape[0] + 64) * U + weight_rel(out_t)) * mag
    bound += 2.0 ** -25 * (dy.abs() @ S)[:, None]
    bound += 2.0 ** -39 * (dy.abs() * p2).amax(1)[:, None] * (What.abs() / p2[:, None]).sum(0)[None]
    return ref, bound


def head_reference(q, What, x, p, ids, w, T, grad_t, zero_mag=None):
    """(loss, its bound, dx, its bound) of tokens with entries ``ids`` (-1: none) of weights ``p``
    (rows add up to 1; dp: their errors), w = 0 where masked.

    A logit is off by (d + 64) additions of what its products add up, and half a step of 1 / T
    and of the division by it.  lse is off by the largest of the row's logits' errors and by exp
    and the sums: 2^-18 (exp's argument z - max is half a step off, 2^-24 of at most 64 where
    exp counts; exp 2^-22; 40 additions and one rescaling per span).  A softmax value is off by
    its logit's and lse's errors and 2^-20 of it more, exp(z - max) is taken in fp16 (one part
    2^-12, two 2^-23; at least half a subnormal step of 2^-14 2^(e_max - e))."""
    x = x.cpu().double()
    n, d = x.shape
    V = What.shape[0]
    z = (x @ What.t()) / T
    dz = ((d + 64) * U * zero_parts(q, x) / T + 2 * U * z.abs())
    lse = torch.logsumexp(z, 1)
    dlse = dz.amax(1) + 2.0 ** -18
    there = ids >= 0
    at = ids.clamp(min=0)
    zj, dzj = torch.gather(z, 1, at), torch.gather(dz, 1, at)
    pj = torch.where(there, p, 0.0)
    lp = torch.where(pj > 0, torch.log(torch.where(pj > 0, pj, 1.0)), 0.0)
    gap = torch.where(pj > 0, lp - zj + lse[:, None], 0.0)
    kl = (pj * gap).sum(1)
    dp = 2.0 ** -20 if p.shape[1] > 1 else 0.0        # teacher's logits / T half a step off, below 16
    loss = w * T * T * kl
    bound = w * T * T * ((pj * (dzj + dp * (gap.abs() + 1))).sum(1) + dlse) + U * loss.abs()
    qv = torch.exp(z - lse[:, None])
    g = qv.clone()
    g.scatter_add_(1, at, -pj)
    dx = (w * T)[:, None] * (g @ What)
    S, p2 = layer_parts(q)
    a_rel = 2.0 ** -12 if grad_t == BF else U
    rel = dz + dlse[:, None] + 2.0 ** -20 + a_rel + weight_rel(grad_t) + (V + 64) * U
    bdx = (qv * rel) @ What.abs() + 2.0 ** -25 * (qv @ S)[:, None]
    bdx += 2.0 ** -38 * p2.max() * (What.abs() / p2[:, None]).sum(0)[None]
    k = ids.shape[1]
    own = torch.zeros_like(qv)
    own.scatter_add_(1, at, pj * (dp + (k + 70) * U))
    bdx += (own + (k + 70) * U * g.abs()) @ What.abs()
    bdx = (w * T)[:, None] * bdx
    return loss, bound, dx, bdx


def teacher_weights(ids, top, T, vocab):
    """p of the entries in 64 bits, ids with -1 where there is none, and which tokens have one."""
    ids, top = ids.cpu().long(), top.cpu().double()
    ids = torch.where((ids >= 0) & (ids < vocab), ids, -1)
    v = torch.where(ids >= 0, top / T, -float("inf"))
    live = v.amax(1) > -float("inf")
    p = torch.softmax(torch.where(live[:, None], v, 0.0), 1)
    return torch.where(ids >= 0, p, 0.0), ids, live
