"""How exact the linear layers are where a choice of types decides it.

The other tests' bound for gelu (linear_ref.act_bound, 2^-20 (1 + |z|)) holds for
both fits of the normal distribution: Phi(-|z|) off by 2.2e-6 of itself (bf16 outputs)
is at most 0.17 * 2.2e-6 < 2^-21 in z Phi(z), and the roundings, counted below, stay
under 2^-21 (1 + |z|)."""
from __future__ import annotations

import pytest
import torch

import dense_gemm_03_amd as dg
from tests import linear_ref as ref


def bf16(*shape, seed, scale=1.0):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=gen) * scale).bfloat16().cuda()


@pytest.mark.gpu
@pytest.mark.parametrize("transb", [False, True])
@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
def test_float32_operands_keep_dz_in_float32(cuda, act, transb):
    """bf16 values handed over as float32 with bf16 gradients: dz is not rounded
    between the activation and the products (linear_ref.backward's bound for
    float32 operands has no bf16 rounding of dz), only dx and dw at the end."""
    m, n, k, offsets = 300, 200, 136, [0, 90, 90, 300]
    x, dy, z = bf16(m, k, seed=1), bf16(m, n, seed=2), bf16(m, n, seed=3, scale=2.0)
    w = bf16(3, *((n, k) if transb else (k, n)), seed=4, scale=k ** -0.5)
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    kw = dict(act=act, pre=z, transb=transb, out_dtype=torch.bfloat16)
    dense = dg.linear_grad(dy.float(), x.float(), w[0].float(), **kw)
    grouped = dg.grouped_linear_grad(dy.float(), x.float(), w.float(), off, **kw)
    cases = [(slice(0, m), w[0], dense)] + [
        (slice(lo, hi), w[g], (grouped[0][lo:hi], grouped[1][g], grouped[2][g]))
        for g, (lo, hi) in enumerate(zip(offsets[:-1], offsets[1:]))]
    for at, weights, got in cases:
        want = ref.backward(dy[at].float(), x[at].float(), weights.float(), act, z[at], 1.0, transb, torch.bfloat16)
        for name, g in zip(("dx", "dw", "dbias"), got):
            assert ref.worst(g, *want[name]) <= 1.0, name


def points(rows, cols, lo, hi, seed):
    gen = torch.Generator().manual_seed(seed)
    return torch.rand(rows, cols, generator=gen) * (hi - lo) + lo


def gelu_bound(z):
    """Of Phi(z) in float32, relative, in half steps u = 2^-24.  |z| >= 1: t G(t)
    e^(-z^2 / 2), t = 1 / (1 + 0.28 |z|).  The exponent's argument has three roundings
    (z^2, the constant, the product), which is 1.5 z^2 u in e, and exp2 is off by one
    unit, 2 u.  t is off by 3 u (the sum, and 1 unit of the reciprocal) and Phi
    by at most 2.7 times that (d ln / d ln t, largest at |z| = 1): 8.1 u.  Horner's
    rule and the coefficients: 4 u.  Two products: 2 u.  The fit, 9e-8: 1.5 u.
    Together 17.6 u + 1.5 z^2 u.  |z| < 1: 1/2 + z Q(z^2), z Q at most 2.15 Phi
    and off by 4 u, and the sum: 9.6 u."""
    return (18 + 1.5 * z * z) * 2.0 ** -24


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [8, 300])
@pytest.mark.parametrize("span", [(-12.0, -3.0), (-3.0, -1.0), (-1.0, 1.0), (1.0, 9.0)], ids=str)
def test_gelu_of_float32_layers(cuda, rows, span):
    """y = gelu(z) with float32 outputs is right to a few units in the last place
    of y itself, in the tail too, through every entry and the reduce of slices."""
    z = points(rows, 64, *span, seed=rows)
    z64 = z.double()
    want = z64 * 0.5 * torch.erfc(-z64 / 2 ** 0.5)
    eye = torch.eye(64, device="cuda")      # sums of one term: z as it is
    for cfg in [-1, *range(dg.gemm_linear_num_configs(dg.GEMM_DTYPE_F32))]:
        for split in (1, 2):
            if cfg >= 0 and not dg.gemm_linear_config_forms(dg.GEMM_DTYPE_F32, cfg) & 1:
                continue
            dg.gemm_linear_force_config(cfg, split)
            try:
                y = dg.linear(z.cuda(), eye, act="gelu")
            finally:
                dg.gemm_linear_force_config()
            # one more half step for z Phi
            err = (y.cpu().double() - want).abs() / ((gelu_bound(z64) + 2.0 ** -24) * want.abs() + 1e-36)
            assert float(err.max()) <= 1.0, (cfg, split, float(err.max()))


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [8, 1200])
def test_gelu_slope_of_float32_layers(cuda, rows):
    """dz = gelu'(z) = Phi(z) + z phi(z): each term within the bound of Phi
    (phi shares its exponential), and the half steps of the sum and of dz."""
    z = points(rows, 72, -12.0, 9.0, seed=rows)
    z64 = z.double()
    cdf = 0.5 * torch.erfc(-z64 / 2 ** 0.5)
    dens = z64.abs() * torch.exp(-z64 * z64 / 2) / (2 * torch.pi) ** 0.5
    p = dg.LinearParams(0, 0, 0, 0, dg.GEMM_ACT_GELU, 1.0, rows, 72, 0, 0, 1, 72, 72, 0, 72, 0, 0)
    need = dg.gemm_linear_act_grad_workspace_size(p)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    dz, dbias = torch.empty(rows, 72, device="cuda"), torch.empty(72, device="cuda")
    dy, pre = torch.ones(rows, 72, device="cuda"), z.cuda()
    assert dg.gemm_linear_act_grad(p, dy.data_ptr(), 72, pre.data_ptr(), None, dz.data_ptr(), 72, dbias.data_ptr(),
                                   ws.data_ptr(), need, torch.cuda.current_stream().cuda_stream) == dg.GEMM_OK
    want = cdf + torch.sign(z64) * dens
    bound = (gelu_bound(z64) + 2.0 ** -23) * (cdf + dens) + 1e-36
    assert float(((dz.cpu().double() - want).abs() / bound).max()) <= 1.0


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [8, 300])
def test_gelu_of_bf16_layers(cuda, rows):
    """bf16 outputs of any size, the tail's too, are the value rounded once: half a
    step, and the bound of Phi with the coarser fit that bf16 takes, 2.2e-6 (37 u)
    and, for |z| < 1 where t counts 2.9 times, 0.6 u more."""
    z = points(rows, 64, -9.0, 9.0, seed=rows).bfloat16()
    z64 = z.double()
    want = z64 * 0.5 * torch.erfc(-z64 / 2 ** 0.5)
    eye = torch.eye(64, device="cuda", dtype=torch.bfloat16)
    code = dg.GEMM_DTYPE_BF16
    for cfg in [-1, *range(dg.gemm_linear_num_configs(code))]:
        for split in (1, 2):
            if cfg >= 0 and not dg.gemm_linear_config_forms(code, cfg) & 1:
                continue
            dg.gemm_linear_force_config(cfg, split)
            try:
                y = dg.linear(z.cuda(), eye, act="gelu", out_dtype=torch.bfloat16)
            finally:
                dg.gemm_linear_force_config()
            near = gelu_bound(z64) + 38 * 2.0 ** -24
            bound = (ref.half_step(torch.bfloat16) * (1 + near) + near) * want.abs() + 1e-36
            assert float(((y.cpu().double() - want).abs() / bound).max()) <= 1.0, (cfg, split)
