"""The operators of gemm_serving.h from their definition in 64 bits, with bounds
on how far a kernel that rounds where the documentation says may be from it.

Log probabilities.  An exponent t = a (z - m) is formed with three roundings (a, the
difference, the product) and exp2 is off by one unit, so a term of the sum is off by
(3 |t| ln2 / 2 + 1) 2^-23 of itself; in the mean over the terms, weighted by p, that is
(1.5 D + 1) 2^-23 with D = sum p |d|.  A lane sums n / 64 terms on four chains that are
joined per 32, the lanes' sums and the moves to larger maxima (each of one unit and of
its exponent's rounding; what a move shrinks below its own size no longer counts, so
the exponents that count add up to few) take some tens of roundings more.  Twice the
sum of these is allowed: sum_error(n, D).  L = ln s adds one unit of L, the distance
d_token two roundings; the entropy weighs the terms' errors with |d|.

Mixture of experts.  The first product's sums are off by sum_bound(K) S as in
linear_ref, the activation by act_bound and 1.13 of its argument's error, the product
with the gate by both factors' errors.  h is stored as two bf16 values, which keep 2^-16
of it (each conversion is off by half a step, 2^-8 and then 2^-8 of the rest), or in
fp32; the smallest numbers of bf16's lower half are 2^-133.  The second product adds
sum_bound of its magnitudes, the weighting and the sums over experts and waves some
roundings of the terms' magnitudes (16 are allowed for).
"""
from __future__ import annotations

import math

import torch

from tests.linear_ref import act64, act_bound, half_step, slope64, sum_bound, worst  # noqa: F401

U = 2.0 ** -23


def sum_error(n, spread):
    return 2 * U * (n / 256 + 40 + 2 * spread)


def ranks(z, top):
    """Places of the largest values of each row: falling, equal ones by place, NaN with -infinity."""
    key = torch.where(torch.isnan(z), torch.full_like(z, -math.inf), z)
    return torch.sort(-key, dim=1, stable=True)[1][:, :top]


def log_probs(logits, tokens, top, scale):
    """{name: (value, bound)} in float64 on the CPU; top_ids whole numbers."""
    z = logits.cpu().double()
    rows, n = z.shape
    m = torch.where(torch.isnan(z), torch.full_like(z, -math.inf), z).max(dim=1, keepdim=True).values
    empty = torch.isneginf(z).all(dim=1, keepdim=True)
    bad = (torch.isnan(z) | torch.isposinf(z)).any(dim=1, keepdim=True)
    base = torch.where(empty | bad, torch.zeros_like(m), m)
    d = torch.where(bad, torch.zeros_like(z), scale * (z - base))
    e = torch.exp(d)
    s = e.sum(dim=1, keepdim=True)
    L = torch.log(s)
    p = torch.where(empty, torch.zeros_like(e), e / s)
    pd = torch.where(p > 0, p * d, torch.zeros_like(p))
    spread = pd.abs().sum(dim=1, keepdim=True)
    H = torch.where(empty, torch.zeros_like(L), L - pd.sum(dim=1, keepdim=True))
    rel = sum_error(n, spread)
    Lerr = rel + U * L.abs().nan_to_num(0, 0, 0)
    nan = torch.full_like(m, math.nan)
    found = {"L": (torch.where(bad, nan, L), Lerr + 1e-37),
             "entropy": (torch.where(bad, nan, H), Lerr + 2 * rel * (1 + spread) + 1e-37),
             "m": (torch.where(bad, nan, m), torch.full_like(m, 1e-300))}

    def at(place):
        dist = torch.gather(d, 1, place)
        value = torch.where(empty, torch.full_like(dist, -math.inf), dist - L)
        return torch.where(bad, nan, value), Lerr + 2 * U * (dist.abs().nan_to_num(0, 0, 0) + L.abs().nan_to_num(0, 0, 0))

    if tokens is not None:
        t = tokens.cpu().long()[:, None]
        held = (t >= 0) & (t < n)
        value, bound = at(torch.where(held, t, torch.zeros_like(t)))
        found["logprob"] = torch.where(held, value, torch.zeros_like(value)), bound + 1e-37
    if top:
        place = ranks(z, top)
        found["top_ids"] = place
        found["top_logprobs"] = at(place)
    return found


def log_probs_grad(logits, tokens, stats, entropy, dlogprob, dentropy, scale):
    """(value, bound) of the gradient for the given stats and entropy."""
    z, st = logits.cpu().double(), stats.cpu().double()
    rows, n = z.shape
    zero = torch.zeros(rows, 1, dtype=torch.float64)
    m, L = st[:, :1], st[:, 1:]
    H = entropy.cpu().double()[:, None] if entropy is not None else zero
    t = tokens.cpu().long()[:, None] if tokens is not None else torch.full((rows, 1), -1)
    held = (t >= 0) & (t < n)
    g = torch.where(held, dlogprob.cpu().double()[:, None], zero) if dlogprob is not None else zero
    h = dentropy.cpu().double()[:, None] if dentropy is not None else zero
    none = ((g == 0) & (h == 0)) | torch.isneginf(m)
    logp = scale * (z - m) - L
    p = torch.exp(logp)
    hit = torch.arange(n)[None, :] == torch.where(held, t, torch.full_like(t, -1))
    info = torch.where(p > 0, p * (logp + H), torch.zeros_like(p))
    dz = scale * (torch.where(hit, g, zero) - g * p - h * info)
    dz = torch.where(none, torch.zeros_like(dz), dz)
    # p: exponent a (z - m) - L log2(e), each part rounded, and exp2
    size = (scale * (z - m)).abs() + L.abs()
    size = torch.where(p > 0, size, torch.zeros_like(size))
    err = scale * p * 4 * U * ((g.abs() + h.abs() * (size + H.abs())) * (2 + size) + h.abs() * (size + H.abs() + 1))
    err = torch.where(none, torch.zeros_like(err), err)
    err = err + torch.where(hit, 4 * U * scale * g.abs(), zero)
    hs = half_step(logits.dtype)
    return dz, err + hs * (dz.abs() + err) + 1e-37


def moe_layer(x, up, down, ids, weights, act, residual, gated, transb, out_dtype):
    """(value, bound), float64 on the CPU."""
    x64 = x.cpu().double()
    ids, weights = ids.cpu().long(), weights.cpu().double()
    y = torch.zeros_like(x64)
    err, mag = torch.zeros_like(x64), torch.zeros_like(x64)
    keep = 2.0 ** -16 if x.dtype == torch.bfloat16 else 0.0
    for e in range(up.shape[0]):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if t.numel() == 0:
            continue
        u, d = up[e].cpu().double(), down[e].cpu().double()
        if transb:
            u, d = u.T, d.T
        z, s = x64[t] @ u, x64[t].abs() @ u.abs()
        zerr = sum_bound(x.shape[1]) * s
        if gated:
            n = z.shape[1] // 2
            a = act64(z[:, :n], act)
            aerr = 1.13 * zerr[:, :n] + (act_bound(z[:, :n]) if act not in ("none", "relu") else 0)
            h = a * z[:, n:]
            herr = aerr * (z[:, n:].abs() + zerr[:, n:]) + a.abs() * zerr[:, n:] + U * h.abs()
        else:
            h = act64(z, act)
            herr = 1.13 * zerr + (act_bound(z) if act not in ("none", "relu") else 0)
        herr = herr + keep * (h.abs() + herr) + 2.0 ** -130
        m = (h.abs() + herr) @ d.abs()
        w = weights[t, j][:, None]
        y.index_add_(0, t, w * (h @ d))
        err.index_add_(0, t, w.abs() * (herr @ d.abs() + sum_bound(d.shape[0]) * m))
        mag.index_add_(0, t, w.abs() * m)
    err = err + 16 * U * mag
    if residual is not None:
        r = residual.cpu().double()
        y = y + r
        err = err + U * (y.abs() + r.abs())
    hs = half_step(out_dtype)
    return y, err + hs * (y.abs() + err) + 1e-37


def adapter_linear(x, w, a, b, ids, scales, bias, act, residual, transb, out_dtype):
    """(value, bound) of the layer with adapters, float64 on the CPU.

    t = scale x . a^T is off by sum_bound(K) of its magnitudes, a rounding for the
    scale and one per part of K (8 at most); bf16 products read it as two bf16 values,
    which keep 2^-16 of it.  The layer's sum has K + rank terms."""
    x64 = x.cpu().double()
    w64 = (w.T if transb else w).cpu().double()
    z, s = x64 @ w64, x64.abs() @ w64.abs()
    carried = torch.zeros_like(z)     # t's error through b
    keep = 2.0 ** -16 if x.dtype == torch.bfloat16 else 0.0
    ids = ids.cpu().long()
    for i in range(a.shape[0]):
        rows = torch.nonzero(ids == i)[:, 0]
        if rows.numel() == 0:
            continue
        a64, b64 = a[i].cpu().double(), b[i].cpu().double()
        f = float(scales[i]) if scales is not None else 1.0
        t, m = f * (x64[rows] @ a64.T), abs(f) * (x64[rows].abs() @ a64.abs().T)
        terr = (sum_bound(x.shape[1]) + 10 * U) * m + keep * t.abs()
        z[rows] += t @ b64.T
        s[rows] += (t.abs() + terr) @ b64.abs().T
        carried[rows] = terr @ b64.abs().T
    err = carried + sum_bound(x.shape[1] + 2 * a.shape[1]) * s
    if bias is not None:
        v = bias.cpu().double()
        z = z + v
        err = err + U * (s + v.abs())
    y = act64(z, act)
    err = 1.13 * err + (act_bound(z) if act not in ("none", "relu") else 0)
    if residual is not None:
        r = residual.cpu().double()
        y = y + r
        err = err + U * (y.abs() + r.abs())
    hs = half_step(out_dtype)
    return y, err + hs * (y.abs() + err) + 1e-37
