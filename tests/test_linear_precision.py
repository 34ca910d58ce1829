"""How exact the linear layers are where a choice of types decides it."""
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
