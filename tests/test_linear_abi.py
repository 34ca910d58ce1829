"""The linear layers' C ABI and host logic without a GPU: exported symbols,
argument checks, workspace sizes, and the formulas the GPU tests hold the
kernels to (activations against torch's, slopes against differences)."""
from __future__ import annotations

import ctypes
import os
import re

import pytest
import torch

import dense_gemm_03_amd as dg
from dense_gemm_03_amd import layers
from tests import linear_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BAD = dg.GEMM_ERR_INVALID_ARG


def params(**kw):
    """Parameters of a valid layer: 100 rows, 64 inputs, 48 outputs, bf16."""
    p = dict(dtype=1, dtype_y=1, dtype_bias=0, transw=0, act=dg.GEMM_ACT_SILU, alpha=1.0, rows=100, N=48, K=64,
             groups=0, ldx=64, ldw=48, ldy=48, ldr=48, ldp=48, stride_w=0, stride_bias=0)
    p.update(kw)
    return dg.LinearParams(**p)


def test_exports_the_headers_symbols():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "gemm_linear.h")).read(), flags=re.S)
    names = set(re.findall(r"^\s*(?:const\s+)?\w+\s*\*?\s*(gemm_linear\w*)\s*\(", text, re.M))
    assert names == set(layers.SIGNATURES)
    lib = ctypes.CDLL(dg.LIB_PATH)
    for name in names:
        assert hasattr(lib, name), name


P = 1 << 20     # stands in for a 16-byte aligned device address: refused calls read nothing
BAD_PARAMS = [dict(dtype=2), dict(dtype_y=-1), dict(dtype_bias=7), dict(transw=2), dict(act=5), dict(act=-1),
              dict(rows=-1), dict(N=-1), dict(K=-1), dict(groups=-1), dict(rows=1 << 31), dict(groups=1 << 20)]


def forward(p, x=P, w=P, off=P, bias=P, res=P, pre=P, y=P, ws=P, nbytes=1 << 40):
    return dg.gemm_linear(p, x, w, off, bias, res, pre, y, ws, nbytes)


@pytest.mark.parametrize("kw", BAD_PARAMS, ids=str)
def test_bad_parameters(kw):
    p = params(**kw)
    assert forward(p) == BAD
    assert dg.gemm_linear_act_grad(p, P, 48, P, P, P, 48, P, P, 1 << 40) == BAD
    assert dg.gemm_linear_weight_grad(p, P, P, P, 0, 0.0, P, P, 1 << 40) == BAD
    for size in (dg.gemm_linear_workspace_size, dg.gemm_linear_act_grad_workspace_size,
                 dg.gemm_linear_weight_grad_workspace_size):
        assert size(p) == BAD
    assert dg.gemm_linear_select_config(p) == BAD


def test_null_parameters():
    assert dg.gemm_linear(None, P, P, P, P, P, P, P, P, 1 << 40) == BAD
    assert dg.gemm_linear_workspace_size(None) == BAD


def test_bad_forward_arguments():
    for kw in (dict(ldx=63), dict(ldw=47), dict(ldy=47), dict(ldr=47), dict(ldp=47), dict(transw=1, ldw=63),
               dict(groups=3, stride_w=64 * 48 - 1, stride_bias=48), dict(groups=3, stride_w=64 * 48, stride_bias=47)):
        assert forward(params(**kw)) == BAD, kw
    for kw in (dict(x=None), dict(w=None), dict(y=None), dict(x=P + 1), dict(w=P + 1), dict(y=P + 1), dict(res=P + 1),
               dict(pre=P + 1), dict(bias=P + 2)):
        assert forward(params(), **kw) == BAD, kw
    grouped = params(groups=3, stride_w=64 * 48, stride_bias=48)
    assert forward(grouped, off=None) == BAD
    assert forward(grouped, off=P + 2) == BAD
    split = params(rows=1, K=8192, N=64, ldx=8192, ldw=64, ldy=64, ldr=64, ldp=64)
    need = dg.gemm_linear_workspace_size(split)
    if need:
        assert forward(split, ws=None) == BAD
        assert forward(split, nbytes=need - 1) == BAD
        assert forward(split, ws=P + 8) == BAD


def test_bad_gradient_arguments():
    act = lambda p=params(rows=2000), dy=P, ldd=48, pre=P, off=P, dz=P, lddz=48, db=P, ws=P, n=1 << 40: \
        dg.gemm_linear_act_grad(p, dy, ldd, pre, off, dz, lddz, db, ws, n)  # noqa: E731
    grouped = params(groups=3, stride_w=64 * 48)
    need = dg.gemm_linear_act_grad_workspace_size(params(rows=2000))
    assert need > 0
    for kw in (dict(dy=None), dict(ldd=47), dict(lddz=47), dict(pre=None), dict(dy=P + 1), dict(dz=P + 1),
               dict(pre=P + 1), dict(db=P + 2), dict(ws=None), dict(n=need - 1), dict(p=grouped, off=None),
               dict(p=params(ldp=47))):
        assert act(**kw) == BAD, kw
    wg = lambda p=params(), x=P, dz=P, off=P, dt=0, dw=P, ws=P, n=1 << 40: \
        dg.gemm_linear_weight_grad(p, x, dz, off, dt, 0.0, dw, ws, n)  # noqa: E731
    for kw in (dict(x=None), dict(dz=None), dict(dw=None), dict(p=params(ldy=47)), dict(dt=2), dict(dw=P + 2), dict(x=P + 1),
               dict(dz=P + 1), dict(p=grouped, off=None), dict(p=params(ldw=47)), dict(p=params(ldx=63)),
               dict(p=params(groups=2, stride_w=10))):
        assert wg(**kw) == BAD, kw


def grad(p=None, o=None, dy=P, x=P, w=P, off=P, pre=P, dx=P, dw=P, db=P, ws=P, n=1 << 40):
    return dg.gemm_linear_grad(p or params(), o or outputs(), dy, x, w, off, pre, dx, dw, db, ws, n)


def outputs(**kw):
    o = dict(dtype_dx=0, dtype_dw=0, beta=0.0, lddx=64, lddw=48, stride_dw=64 * 48)
    o.update(kw)
    return dg.LinearGradOutputs(**o)


def test_bad_backward_arguments():
    groups = dict(groups=3, stride_w=64 * 48)
    need = dg.gemm_linear_grad_workspace_size(params(), outputs())
    assert need >= 100 * 48 * 2
    for kw in BAD_PARAMS:
        assert grad(params(**kw)) == BAD, kw
        assert dg.gemm_linear_grad_workspace_size(params(**kw), outputs()) == BAD, kw
    for kw in (dict(dy=None), dict(x=None), dict(w=None), dict(pre=None), dict(dy=P + 1), dict(x=P + 1), dict(w=P + 1),
               dict(pre=P + 1), dict(dx=P + 2), dict(dw=P + 2), dict(db=P + 2), dict(ws=None), dict(ws=P + 8),
               dict(n=need - 1), dict(o=outputs(dtype_dx=2)), dict(o=outputs(dtype_dw=-1)), dict(o=outputs(lddx=63)),
               dict(o=outputs(lddw=47)), dict(p=params(ldx=63)), dict(p=params(ldw=47)), dict(p=params(ldy=47)),
               dict(p=params(ldp=47)), dict(p=params(**groups), off=None), dict(p=params(**groups), off=P + 2),
               dict(p=params(**groups), o=outputs(stride_dw=64 * 48 - 1)),
               dict(p=params(transw=1, ldw=64), o=outputs(lddw=63))):
        assert grad(**kw) == BAD, kw
    assert dg.gemm_linear_grad(None, outputs(), P, P, P, P, P, P, P, P, P, 1 << 40) == BAD
    assert dg.gemm_linear_grad(params(), None, P, P, P, P, P, P, P, P, P, 1 << 40) == BAD
    assert dg.gemm_linear_grad_workspace_size(params(), None) == BAD
    # nothing asked for, nothing done
    assert grad(dx=None, dw=None, db=None, x=None, w=None, ws=None, n=0) == dg.GEMM_OK
    # a forced entry that lacks one of the forms is refused before anything runs
    rows = [c for c in range(dg.gemm_linear_num_configs(1)) if dg.gemm_linear_config_forms(1, c) != 7]
    assert rows
    dg.gemm_linear_force_config(rows[0])
    try:
        assert grad() == BAD
    finally:
        dg.gemm_linear_force_config()


def test_backward_scratch_covers_the_parts():
    for rows, N, K in ((1, 1, 1), (100, 48, 64), (2000, 333, 515), (40, 4096, 4096), (5000, 64, 8192)):
        for dtype in (0, 1):
            for t in (0, 1):
                for act in (0, 4):
                    lddz = N if act == 0 else -(-N // (4 << dtype)) * (4 << dtype)
                    p = params(dtype=dtype, rows=rows, N=N, K=K, transw=t, act=act, ldx=K, ldw=K if t else N, ldy=N,
                               ldp=N)
                    o = outputs(lddx=K, lddw=K if t else N)
                    dz = rows * lddz * (4 >> dtype) if act else 0
                    turned = params(dtype=dtype, dtype_y=0, rows=rows, N=K, K=N, transw=1 - t, act=0, ldx=lddz,
                                    ldw=K if t else N, ldy=K, ldr=0, ldp=0)
                    weight = params(dtype=dtype, rows=rows, N=N, K=K, transw=t, act=0, ldx=K, ldw=K if t else N,
                                    ldy=lddz)
                    size = lambda *which: dg.gemm_linear_grad_workspace_size(p, o, *which)  # noqa: E731
                    assert size(1, 0, 0) >= dz + dg.gemm_linear_workspace_size(turned)
                    assert size(0, 1, 0) >= dz + dg.gemm_linear_weight_grad_workspace_size(weight)
                    assert size(0, 0, 1) >= dg.gemm_linear_act_grad_workspace_size(p)
                    assert size(1, 1, 1) >= max(size(1, 0, 0), size(0, 1, 0), size(0, 0, 1))


def test_empty_calls_launch_nothing():
    assert forward(params(rows=0), x=None, y=None, ws=None, nbytes=0) == dg.GEMM_OK
    assert forward(params(N=0), w=None, y=None, ws=None, nbytes=0) == dg.GEMM_OK
    assert dg.gemm_linear_act_grad(params(rows=0), None, 48, None, None, None, 48, None, None, 0) == dg.GEMM_OK
    assert dg.gemm_linear_act_grad(params(N=0), None, 48, None, None, P, 48, P, None, 0) == dg.GEMM_OK
    assert dg.gemm_linear_weight_grad(params(K=0), None, P, None, 0, 0.0, None, None, 0) == dg.GEMM_OK


def test_the_dispatchers_entry_has_the_form():
    for dtype in (0, 1):
        n = dg.gemm_linear_num_configs(dtype)
        assert n >= 3 and dg.gemm_linear_config_name(dtype, n) is None
        assert dg.gemm_linear_config_forms(dtype, n) == BAD
        for rows in (0, 1, 5, 64, 200, 5000):
            for N, K in [(1, 1), (64, 4096), (4096, 64), (16384, 4096)]:
                for groups in (0, 1, 16, 300):
                    for t in (0, 1):
                        p = params(dtype=dtype, rows=rows, N=N, K=K, groups=groups, transw=t)
                        for wg in (0, 1):
                            cfg = dg.gemm_linear_select_config(p, wg)
                            assert cfg >= 0
                            assert dg.gemm_linear_config_forms(dtype, cfg) >> (2 if wg else t) & 1
    assert dg.gemm_linear_num_configs(3) == BAD


def test_forced_entry_without_the_form_is_refused():
    for dtype in (0, 1):
        for cfg in range(dg.gemm_linear_num_configs(dtype)):
            forms = dg.gemm_linear_config_forms(dtype, cfg)
            dg.gemm_linear_force_config(cfg)
            try:
                for form in range(3):
                    got = dg.gemm_linear_select_config(params(dtype=dtype, transw=form & 1), form == 2)
                    assert got == (cfg if forms >> form & 1 else BAD)
            finally:
                dg.gemm_linear_force_config()


def test_helpers_refuse_host_tensors():
    x, w = torch.zeros(4, 8), torch.zeros(8, 6)
    with pytest.raises(ValueError):
        dg.linear(x, w)
    with pytest.raises(ValueError):
        dg.linear_grad(torch.zeros(4, 6), x, w)
    with pytest.raises(ValueError):
        dg.grouped_linear(x, w, torch.zeros(2, dtype=torch.int32))


@pytest.mark.parametrize("act", ref.ACTS)
def test_formulas(act):
    """The reference activations are torch's, and their slopes the limits of
    difference quotients: a central difference with step h is off by at most
    h^2 / 6 times the third derivative (below 2 here) plus rounding."""
    f = torch.nn.functional
    theirs = {"none": lambda t: t, "relu": f.relu, "gelu": f.gelu, "silu": f.silu,
              "gelu_tanh": lambda t: f.gelu(t, approximate="tanh")}[act]
    z = torch.linspace(-8, 8, 1601, dtype=torch.float64) + 0.003
    assert torch.allclose(ref.act64(z, act), theirs(z), rtol=1e-12, atol=1e-14)
    h = 1e-4
    diff = (ref.act64(z + h, act) - ref.act64(z - h, act)) / (2 * h)
    assert float((diff - ref.slope64(z, act)).abs().max()) < h * h + 1e-10
