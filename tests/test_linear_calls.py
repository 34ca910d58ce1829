"""What a call of the linear layers may be handed: views, aliases, streams,
threads, and the largest sizes.  The host's part of it runs without a GPU."""
from __future__ import annotations

import pytest
import torch

import dense_gemm_03_amd as dg
from dense_gemm_03_amd import layers


# ------------------------------------------------------------------ views --

def strided_weights():
    """Weights of one input (or, transposed, one output) whose values are not
    side by side."""
    wide = torch.arange(1, 49, dtype=torch.float32).reshape(2, 24)
    return [("1 x N, every second column", wide[:1, ::2], 0),
            ("column of a wide matrix, transposed", wide.reshape(12, 4)[:, :1].t(), 0),
            ("groups of 1 x N", wide[:, ::2].unsqueeze(1), 2)]


@pytest.mark.parametrize("name,w,groups", strided_weights(), ids=[c[0] for c in strided_weights()])
def test_one_row_of_weights_has_to_be_contiguous(name, w, groups):
    assert w.shape[-2] == 1 and w.shape[-1] == 12 and w.stride(-1) != 1
    for transb in (False, True):
        with pytest.raises(ValueError):
            layers._weights(w, groups, transb)
    tight = w.contiguous()
    assert layers._weights(tight, groups, False) == (1, 12, 12, 12 if groups else 0)
    assert layers._weights(tight, groups, True) == (12, 1, 12, 12 if groups else 0)


@pytest.mark.gpu
def test_one_row_of_weights_on_the_gpu(cuda):
    x = torch.ones(3, 1, device="cuda")
    for name, w, groups in strided_weights():
        w = torch.empty_strided(w.shape, w.stride(), device="cuda").copy_(w)
        off = torch.tensor([0, 1, 3], dtype=torch.int32, device="cuda")
        forward = (lambda v: dg.grouped_linear(x, v, off)) if groups else (lambda v: dg.linear(x, v))
        with pytest.raises(ValueError):
            forward(w)
        with pytest.raises(ValueError):   # nor as the gradient's place
            dy = torch.ones(3, 12, device="cuda")
            if groups:
                dg.grouped_linear_grad(dy, x, w.contiguous(), off, dw=w)
            else:
                dg.linear_grad(dy, x, w.contiguous(), dw=w)
        rows = [0, 1, 1] if groups else [0, 0, 0]
        want = torch.stack([w.reshape(-1, 12)[g] for g in rows])
        assert torch.equal(forward(w.contiguous()), want)
