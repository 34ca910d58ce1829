"""The linear layers' kernels well past the first trip round their LDS stages:
summed axes of 5 to 19 k-tiles, odd and even, with and without a tail, for whole
tiles, halves and quarters, dense and grouped, all three products.  Operands are
small whole numbers, so every partial sum is exact in fp32 (at most 25 x 1300,
below 2^24) and the whole output has to equal the product in 64 bits, whatever
the order of the sums: a stage that is read too early, overwritten too early or
taken in a wrong place of k shows."""
from __future__ import annotations

import pytest
import torch

import dense_gemm_03_amd as dg
from tests.gpu_util import log

pytestmark = pytest.mark.gpu


def whole(*shape, seed, dtype=torch.bfloat16, pad=0):
    """Whole numbers from -5 to 5, rows `pad` elements further apart."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.randint(-5, 6, (*shape[:-1], shape[-1] + pad), generator=gen, device="cuda").to(dtype)
    return t[..., :shape[-1]]


def same(what, got, want):
    torch.cuda.synchronize()
    bad = int((got.double() != want).sum())
    assert bad == 0, "%s: %d of %d differ" % (what, bad, want.numel())


def entry(dtype, prefix):
    code = dg.GEMM_DTYPE_BF16 if dtype == torch.bfloat16 else dg.GEMM_DTYPE_F32
    names = [dg.gemm_linear_config_name(code, i) for i in range(dg.gemm_linear_num_configs(code))]
    found = [i for i, name in enumerate(names) if name.startswith(prefix)]
    assert len(found) == 1, (prefix, names)
    return found[0]


def dense(cfg, split, m, n, k, transb, dtype=torch.bfloat16, pad=0):
    """y (m x n) over k and dw (its orientation by transb) over k."""
    x = whole(m, k, seed=1, dtype=dtype, pad=pad)
    w = whole(*((n, k) if transb else (k, n)), seed=2, dtype=dtype, pad=pad)
    want = x.double() @ (w.double().t() if transb else w.double())
    xt, dz = whole(k, m, seed=3, dtype=dtype, pad=pad), whole(k, n, seed=4, dtype=dtype, pad=pad)
    grad = xt.double().t() @ dz.double()
    place = torch.empty((n, m) if transb else (m, n), dtype=dtype, device="cuda")   # stands for w: not read
    assert dg.gemm_linear_force_config(cfg, split) == 0
    try:
        same("y", dg.linear(x, w, transb=transb), want)
        dw = dg.linear_grad(dz, xt, place, transb=transb, need_dx=False, need_dbias=False)[1]
        same("dw", dw, grad.t() if transb else grad)
    finally:
        dg.gemm_linear_force_config()


# 256 x 256 tiles on 256 units, 32 per XCD: 143 tiles stay whole, 81 are cut into
# halves (and a last row of tiles into quarters), of 272 the last sixteen and of
# 9 all into quarters.
TILES = [(3300, 2800), (2100, 2060), (4250, 4096), (700, 600)]
SUMS = [320, 384, 392, 584, 1216]     # 5, 6, 6 + tail, 9 + tail, 19 k-tiles of 64


@pytest.mark.parametrize("transb", [False, True])
@pytest.mark.parametrize("k", SUMS)
@pytest.mark.parametrize("tiles", TILES, ids=str)
def test_large_tiles(cuda, tiles, k, transb):
    cfg = entry(torch.bfloat16, "bf16_256x256x64")
    for split in (1, 2):
        dense(cfg, split, *tiles, k, transb)


@pytest.mark.parametrize("pad", [1, 2, 8])
@pytest.mark.parametrize("tiles", TILES, ids=str)
def test_large_tiles_of_other_pitches(cuda, tiles, pad):
    """2-, 4- and 16-byte rows with something else behind them."""
    cfg = entry(torch.bfloat16, "bf16_256x256x64")
    for transb in (False, True):
        dense(cfg, 1, *tiles, 456, transb, pad=pad)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_every_entry(cuda, dtype):
    code = dg.GEMM_DTYPE_BF16 if dtype == torch.bfloat16 else dg.GEMM_DTYPE_F32
    for cfg in range(dg.gemm_linear_num_configs(code)):
        if dg.gemm_linear_config_forms(code, cfg) != 7:
            continue
        for k in (640, 1240):
            for split in (1, 3):
                for pad in (0, 1, 2):
                    log(dg.gemm_linear_config_name(code, cfg), k, split, pad)
                    for transb in (False, True):
                        dense(cfg, split, 600, 520, k, transb, dtype=dtype, pad=pad)


COUNTS = {
    "whole tiles and quarters": [512, 256, 300, 0, 770, 256, 1024, 129, 513, 1, 384, 640],
    "halves": [256, 512, 256, 768, 256],
}


@pytest.mark.parametrize("transb", [False, True])
@pytest.mark.parametrize("name", COUNTS)
@pytest.mark.parametrize("k", [320, 392, 584])
def test_groups_start_at_other_k_tiles(cuda, k, name, transb):
    """Group g starts at k-tile 8 g modulo their number (5, 6, 9: not 0)."""
    counts, n = COUNTS[name], 1100
    offsets = [3]
    for c in counts:
        offsets.append(offsets[-1] + c)
    rows, g = offsets[-1] + 7, len(counts)
    x = whole(rows, k, seed=1)
    w = whole(g, *((n, k) if transb else (k, n)), seed=2)
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    want = torch.full((rows, n), 7.0, dtype=torch.float64, device="cuda")
    for i in range(g):
        at = slice(offsets[i], offsets[i + 1])
        want[at] = x[at].double() @ (w[i].double().t() if transb else w[i].double())
    for split in (1, 2):
        assert dg.gemm_linear_force_config(entry(torch.bfloat16, "bf16_256x256x64"), split) == 0
        try:
            y = dg.grouped_linear(x, w, off, transb=transb, out=torch.full((rows, n), 7.0, device="cuda"))
        finally:
            dg.gemm_linear_force_config()
        same("y", y, want)


@pytest.mark.parametrize("transb", [False, True])
def test_long_groups_of_weight_gradients(cuda, transb):
    """dw over groups of 1 to 1216 rows, in whole tiles (12 of them per group)
    and in the pieces of a last round."""
    counts, n, k = [1216, 640, 5, 0, 392, 584, 64, 320, 129], 1000, 700
    offsets = [2]
    for c in counts:
        offsets.append(offsets[-1] + c)
    rows, g = offsets[-1] + 5, len(counts)
    x, dz = whole(rows, k, seed=1), whole(rows, n, seed=2)
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    place = torch.empty(g, *((n, k) if transb else (k, n)), dtype=torch.bfloat16, device="cuda")
    for split in (1, 2):
        assert dg.gemm_linear_force_config(entry(torch.bfloat16, "bf16_256x256x64"), split) == 0
        try:
            dw = dg.grouped_linear_grad(dz, x, place, off, transb=transb, need_dx=False, need_dbias=False)[1]
        finally:
            dg.gemm_linear_force_config()
        for i in range(g):
            at = slice(offsets[i], offsets[i + 1])
            want = x[at].double().t() @ dz[at].double()
            same("dw %d" % i, dw[i], want.t() if transb else want)
