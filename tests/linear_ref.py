"""The linear layers' definition in 64 bits, with bounds on how far a kernel
that rounds where the documentation says may be from it.

Bounds.  bf16 products are exact in fp32 and fp32 products round once; a sum of
K terms in fp32, in any order, is off by at most K 2^-24 (1 + o(1)) times the
sum S of the terms' magnitudes.  The kernels' matrix instructions may round
inside, so twice that is allowed: sum_bound(K) S.  The activations and their
slopes are formed from the hardware's exp2 and reciprocal (1 ulp each) and a
rounded exponent, which makes sigmoid(x) off by at most (|x| + 4) 2^-23
(1 - sigmoid) relative; since z^2 q (1 - q) < 1 and |z| q (1 - q) < 0.3, the
activations are off by less than 2^-21 (1 + |z|).  The error function is a
polynomial within 1.5e-7 of it and half of that, times z, is less than 2^-23 |z|.
Twice the former is allowed: act_bound.  |act'| < 1.13, so an error in z grows by less than
that.  An output in a narrower type adds half a step of it (eps / 2 relative).
"""
from __future__ import annotations

import math

import torch

ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def sum_bound(k):
    return 2.0 * (k + 8) * 2.0 ** -24


def act_bound(z):
    return 2.0 ** -20 * (1 + z.abs())


def act64(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu":
        return z * 0.5 * torch.erfc(-z / math.sqrt(2))
    if act == "gelu_tanh":
        return z * torch.sigmoid(math.sqrt(8 / math.pi) * (z + 0.044715 * z ** 3))
    if act == "silu":
        return z * torch.sigmoid(z)
    return z


def slope64(z, act):
    if act == "relu":
        return (z > 0).double()
    if act == "gelu":
        return 0.5 * torch.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        r = math.sqrt(8 / math.pi)
        q = torch.sigmoid(r * (z + 0.044715 * z ** 3))
        return q + z * q * (1 - q) * r * (1 + 3 * 0.044715 * z ** 2)
    if act == "silu":
        q = torch.sigmoid(z)
        return q + z * q * (1 - q)
    return torch.ones_like(z)


def oriented(w, transb):
    return (w.transpose(-1, -2) if transb else w).cpu().double()


def forward(x, w, bias, act, residual, alpha, transb, out_dtype):
    """(z, y, bound of z, bound of y) of one group's rows, in float64."""
    x, w = x.cpu().double(), oriented(w, transb)
    z, s = alpha * (x @ w), abs(alpha) * (x.abs() @ w.abs())
    err = sum_bound(x.shape[1]) * s
    if bias is not None:
        b = bias.cpu().double()
        z = z + b
        err = err + 2.0 ** -23 * (s + b.abs())
    y = act64(z, act)
    yerr = 1.13 * err + (act_bound(z) if act not in ("none", "relu") else 0)
    if residual is not None:
        r = residual.cpu().double()
        y = y + r
        yerr = yerr + 2.0 ** -23 * (y.abs() + r.abs())
    h = half_step(out_dtype)
    return z, y, err + h * (z.abs() + err) + 1e-37, yerr + h * (y.abs() + yerr) + 1e-37


def backward(dy, x, w, act, pre, alpha, transb, out_dtype):
    """{name: (value, bound)} for dx, dw and dbias of one group's rows."""
    h, hin = half_step(out_dtype), half_step(dy.dtype)
    x64, w64, dy64 = x.cpu().double(), oriented(w, transb), dy.cpu().double()
    dz, derr = dy64, torch.zeros_like(dy64)
    if act != "none":
        z = pre.cpu().double()
        dz = dy64 * slope64(z, act)
        derr = dy64.abs() * (act_bound(z) if act != "relu" else 0) + 2.0 ** -23 * dz.abs()
    rounded = derr if act == "none" else derr + hin * (dz.abs() + derr)   # as the products read it
    mag = dz.abs() + rounded
    a = abs(alpha)
    found = {
        "dx": (alpha * (dz @ w64.T), a * (rounded @ w64.abs().T + sum_bound(dz.shape[1]) * (mag @ w64.abs().T))),
        "dw": (alpha * (x64.T @ dz), a * (x64.abs().T @ rounded + sum_bound(x.shape[0]) * (x64.abs().T @ mag))),
    }
    if transb:
        found["dw"] = tuple(t.T for t in found["dw"])
    found = {k: (v, e + h * (v.abs() + e) + 1e-37) for k, (v, e) in found.items()}
    found["dbias"] = (dz.sum(0), derr.sum(0) + sum_bound(dz.shape[0]) * (dz.abs() + derr).sum(0) + 1e-37)
    return found


def worst(got, want, bound):
    """Largest error over its bound (infinite where a NaN appears or is lost)."""
    if got.numel() == 0:
        return 0.0
    got = got.cpu().double()
    assert got.shape == want.shape, (got.shape, want.shape)
    ratio = (got - want).abs() / bound
    ratio = torch.where(torch.isnan(want) & torch.isnan(got), torch.zeros_like(ratio), ratio)
    return float(torch.nan_to_num(ratio, nan=math.inf).max())
