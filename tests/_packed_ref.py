"""Plain 64-bit attention of packed sequences and its gradient, from the formulas of include/fa.h,
with bounds for rounding, for the tests.  torch on the CPU; nothing of the package."""
from __future__ import annotations

import math

import torch


def seen(n, m, causal):
    """[n, m]: query i sees key j."""
    i, j = torch.arange(n)[:, None], torch.arange(m)[None]
    return j <= i + m - n if causal else torch.ones(n, m, dtype=torch.bool)


def sequences(new, keys):
    a = b = 0
    for n, m in zip(new, keys):
        yield slice(a, a + n), slice(b, b + m), n, m
        a, b = a + n, b + m


def _heads(x, G):
    return x.double().repeat_interleave(G, 1).transpose(0, 1)  # [H, T, d]


def forward(q, k, v, new, keys, causal, scale, half_step, tiny):
    """(o, lse, bound of o, bound of lse) of rows packed without gaps.

    Bounds, with e = half_step (the inputs' type) and w the weights relative to their sum:
    a score is off by d roundings of 2^-23 of its terms (fp32 accumulation), s, and the exponential
    by 2^-21 and 2^-23 of its argument; a weight for the product by e (or `tiny` / 2 where subnormal);
    the sums over m keys by m 2^-23; the result by e, or `tiny` / 2 below the normal numbers."""
    Hq, d = q.shape[1:]
    G = Hq // k.shape[1]
    o, ob = torch.zeros(q.shape, dtype=torch.float64), torch.zeros(q.shape, dtype=torch.float64)
    lse, lb = torch.full(q.shape[:2], -math.inf, dtype=torch.float64), torch.zeros(q.shape[:2], dtype=torch.float64)
    for rows, cols, n, m in sequences(new, keys):
        if n == 0 or m == 0:
            continue
        Q, K, V = q[rows].double().transpose(0, 1), _heads(k[cols], G), _heads(v[cols], G)
        mask = seen(n, m, causal)
        x = (Q @ K.transpose(1, 2) * scale).masked_fill(~mask, -math.inf)
        l = torch.logsumexp(x, -1, keepdim=True)
        p = torch.where(mask, torch.exp(x - torch.where(l == -math.inf, 0.0, l)), 0.0)
        y = p @ V
        s = (Q.abs() @ K.abs().transpose(1, 2) * scale).masked_fill(~mask, 0.0) * (d * 2.0 ** -23)
        off = s + 2.0 ** -21 + torch.where(mask, (x - x.amax(-1, keepdim=True)).abs().nan_to_num(0, 0, 0) * 2.0 ** -23, 0.0)
        most = (p * off).sum(-1, keepdim=True)  # of the sum of the weights
        b = (p * (off + half_step + m * 2.0 ** -23 + most)) @ V.abs() + tiny / 2 * m * V.abs().amax(1, keepdim=True)
        o[rows], ob[rows] = y.transpose(0, 1), (b + half_step * (y.abs() + b) + tiny / 2).transpose(0, 1)
        lse[rows] = l[..., 0].T
        lb[rows] = (most + m * 2.0 ** -23 + 2.0 ** -20 + 2.0 ** -22 * l.abs().nan_to_num(0, 0, 0))[..., 0].T
    return o, lse, ob, lb


def backward(q, k, v, o, do, lse, new, keys, causal, scale, half_step, tiny):
    """((dq, dk, dv), their bounds) for given o and lse.

    A weight is off by what its score, the saved LSE (2^-24 of it) and the exponential are; it is
    rounded by e for dV; dP and D by d roundings of 2^-23 of their terms; dS by e for dK, dQ
    (or `tiny` / 2 where subnormal); sums by their length times 2^-23; results by e, or, below the
    normal numbers, where they are multiples of `tiny`, by half of that."""
    Hq, d = q.shape[1:]
    Hk = k.shape[1]
    G = Hq // Hk
    grads = [torch.zeros(x.shape, dtype=torch.float64) for x in (q, k, v)]
    bounds = [torch.zeros(x.shape, dtype=torch.float64) for x in (q, k, v)]
    e, f = half_step, 2.0 ** -23
    for rows, cols, n, m in sequences(new, keys):
        if n == 0 or m == 0:
            continue
        Q, O, dO = (x[rows].double().transpose(0, 1) for x in (q, o, do))
        K, V, L = _heads(k[cols], G), _heads(v[cols], G), lse[rows].double().T[..., None]
        mask = seen(n, m, causal) & (L > -math.inf)
        x = Q @ K.transpose(1, 2) * scale
        p = torch.where(mask, torch.exp(x - torch.where(L == -math.inf, 0.0, L)), 0.0)
        dp, D = dO @ V.transpose(1, 2), (dO * O).sum(-1, keepdim=True)
        ds = p * (dp - D)
        s = Q.abs() @ K.abs().transpose(1, 2) * scale * (d * f)
        off = s + 2.0 ** -21 + (x.abs() + L.abs().nan_to_num(0, 0, 0)) * f
        dpb = (dO.abs() @ V.abs().transpose(1, 2) + (dO * O).abs().sum(-1, keepdim=True)) * (d * f)
        dsb = p * ((off + e) * (dp - D).abs() + (1 + off) * dpb)
        found = [ds @ K * scale, ds.transpose(1, 2) @ Q * scale, p.transpose(1, 2) @ dO]
        slack = [((dsb + ds.abs() * m * f) @ K.abs() + tiny / 2 * m * K.abs().amax(1, keepdim=True)) * scale,
                 ((dsb + ds.abs() * n * G * f).transpose(1, 2) @ Q.abs() + tiny / 2 * n * Q.abs().amax(1, keepdim=True)) * scale,
                 (p * (off + e + n * G * f)).transpose(1, 2) @ dO.abs() + tiny / 2 * n * dO.abs().amax(1, keepdim=True)]
        for i, at in enumerate((rows, cols, cols)):
            y, b = found[i].transpose(0, 1), slack[i].transpose(0, 1)
            if i:
                y, b = y.unflatten(1, (Hk, G)).sum(2), b.unflatten(1, (Hk, G)).sum(2)
            grads[i][at], bounds[i][at] = y, b + e * (y.abs() + b) + tiny / 2
    return grads, bounds
