"""Linear layers on the GPU against their definition in 64 bits: the product
with bias, activation and residual, dense and grouped by expert, and the
gradients, over types, orientations, every kernel of the table, sizes at the
edges of tiles, alignments, offsets that leave groups empty and rows to nobody,
streams and captured graphs.  The bounds are derived in linear_ref."""
from __future__ import annotations

import pytest
import torch

import dense_gemm_03_amd as dg
from tests import linear_ref as ref
from tests.gpu_util import log

pytestmark = pytest.mark.gpu

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def rand(*shape, dtype, seed, scale=1.0):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=gen, dtype=torch.float32) * scale).to(dtype).cuda()


def padded(t, extra, fill=float("nan")):
    """t with `extra` columns behind each row (a view with a longer pitch)."""
    if not extra:
        return t
    wide = torch.full((*t.shape[:-1], t.shape[-1] + extra), fill, dtype=t.dtype, device=t.device)
    wide[..., :t.shape[-1]] = t
    return wide[..., :t.shape[-1]]


def spans(offsets, rows):
    off = [min(max(o, 0), rows) for o in offsets]
    return [(a, max(a, b)) for a, b in zip(off[:-1], off[1:])]


def check(what, got, want, bound):
    torch.cuda.synchronize()
    r = ref.worst(got, want, bound)
    assert r <= 1.0, "%s: error %.3g of its bound" % (what, r)
    return r


def check_forward(dtype, rows, n, k, *, transb=False, act="none", bias=True, residual=False, pre=False,
                  alpha=1.0, out=None, offsets=None, pad=0, seed=1, x=None):
    dt, odt = DTYPES[dtype], DTYPES[out or dtype]
    groups = len(offsets) - 1 if offsets is not None else 0
    lead = (groups,) if groups else ()
    x = padded(rand(rows, k, dtype=dt, seed=seed), pad) if x is None else x
    w = padded(rand(*lead, *((n, k) if transb else (k, n)), dtype=dt, seed=seed + 1, scale=max(k, 1) ** -0.5), pad)
    b = rand(*lead, n, dtype=dt, seed=seed + 2) if bias else None
    r = padded(rand(rows, n, dtype=odt, seed=seed + 3), pad) if residual else None
    before = rand(rows, n, dtype=odt, seed=seed + 4)
    y = padded(before.clone(), pad, 7.0)
    z = padded(before.clone(), pad, 7.0) if pre else None
    kw = dict(bias=b, act=act, residual=r, alpha=alpha, transb=transb, pre=z, out=y)
    if groups:
        got = dg.grouped_linear(x, w, torch.tensor(offsets, dtype=torch.int32, device="cuda"), **kw)
    else:
        got = dg.linear(x, w, **kw)
    assert got is y
    torch.cuda.synchronize()
    want, bound = before.cpu().double(), torch.full((rows, n), 1e-300, dtype=torch.float64)
    zwant, zbound = want.clone(), bound.clone()
    for g, (lo, hi) in enumerate(spans(offsets, rows) if groups else [(0, rows)]):
        at = slice(lo, hi)
        zwant[at], want[at], zbound[at], bound[at] = ref.forward(
            x[at], w[g] if groups else w, (b[g] if groups else b) if bias else None, act,
            r[at] if residual else None, alpha, transb, odt)
    check("y", y, want, bound)
    if pre:
        check("pre", z, zwant, zbound)
    if pad and rows and n:     # the pitch behind the rows is left as it was
        assert bool((y.as_strided((rows, pad), (y.stride(0), 1), n) == 7.0).all())
    return y


def check_backward(dtype, rows, n, k, *, transb=False, act="none", alpha=1.0, out=None, offsets=None, pad=0,
                   seed=1, **kw):
    dt, odt = DTYPES[dtype], DTYPES[out or dtype]
    groups = len(offsets) - 1 if offsets is not None else 0
    lead = (groups,) if groups else ()
    x = padded(rand(rows, k, dtype=dt, seed=seed), pad)
    w = padded(rand(*lead, *((n, k) if transb else (k, n)), dtype=dt, seed=seed + 1, scale=max(k, 1) ** -0.5), pad)
    dy = padded(rand(rows, n, dtype=dt, seed=seed + 2), pad)
    z = padded(rand(rows, n, dtype=dt, seed=seed + 3, scale=2.0), pad) if act != "none" else None
    kw = dict(act=act, pre=z, alpha=alpha, transb=transb, out_dtype=odt, **kw)
    if groups:
        dx, dw, db = dg.grouped_linear_grad(dy, x, w, torch.tensor(offsets, dtype=torch.int32, device="cuda"), **kw)
    else:
        dx, dw, db = dg.linear_grad(dy, x, w, **kw)
    torch.cuda.synchronize()
    for g, (lo, hi) in enumerate(spans(offsets, rows) if groups else [(0, rows)]):
        at = slice(lo, hi)
        want = ref.backward(dy[at], x[at], w[g] if groups else w, act, z[at] if z is not None else None,
                            alpha, transb, odt)
        check("dx %d" % g, dx[at], *want["dx"])
        check("dw %d" % g, dw[g] if groups else dw, *want["dw"])
        check("dbias %d" % g, db[g] if groups else db, *want["dbias"])
    return dx, dw, db


SIZES = [(1, 1, 1), (1, 256, 64), (3, 100, 70), (17, 129, 33), (33, 64, 512), (64, 512, 1000), (65, 257, 96),
         (130, 384, 260), (300, 300, 200), (257, 520, 129), (600, 768, 320)]


@pytest.mark.parametrize("transb", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_forward_sizes(cuda, dtype, transb, size):
    m, n, k = size
    check_forward(dtype, m, n, k, transb=transb, act="silu", residual=True, pre=True, alpha=0.75)


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("act", ref.ACTS)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_forward_epilogues(cuda, dtype, act, out):
    for bias, residual, pre in [(False, False, False), (True, False, True), (False, True, False), (True, True, True)]:
        check_forward(dtype, 140, 200, 96, act=act, bias=bias, residual=residual, pre=pre, out=out)


@pytest.mark.parametrize("pad", [1, 2, 4, 8])
@pytest.mark.parametrize("transb", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_pitches(cuda, dtype, transb, pad):
    """Rows with a longer pitch: 2-, 4-, 8- and 16-byte aligned; what lies
    behind the rows (NaN in the inputs) is neither used nor written."""
    check_forward(dtype, 150, 256, 192, transb=transb, act="gelu", residual=True, pre=True, pad=pad)
    check_forward(dtype, 70, 96, 128, transb=transb, offsets=[0, 33, 33, 70], pad=pad)
    check_backward(dtype, 150, 256, 192, transb=transb, act="silu", pad=pad)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_every_kernel(cuda, dtype):
    """Every entry of the table in each of its forms, whole and in slices,
    with aligned rows and with odd ones, dense and grouped."""
    code = dg.GEMM_DTYPE_F32 if dtype == "f32" else dg.GEMM_DTYPE_BF16
    offsets = [2, 2, 150, 151, 151, 420, 511]
    try:
        for cfg in range(dg.gemm_linear_num_configs(code)):
            forms = dg.gemm_linear_config_forms(code, cfg)
            for split in (1, 3):
                for n, k in [(520, 384), (263, 331)]:
                    for off in (None, offsets):
                        log(dg.gemm_linear_config_name(code, cfg), split, n, k, off is not None)
                        assert dg.gemm_linear_force_config(cfg, split) == 0
                        for transb in (False, True):
                            if forms >> transb & 1:
                                check_forward(dtype, 515, n, k, transb=transb, act="silu", residual=True, pre=True,
                                              offsets=off)
                            if forms & 4:
                                check_weight_grad(dtype, 515, n, k, transb, off)
    finally:
        dg.gemm_linear_force_config()


def check_weight_grad(dtype, rows, n, k, transb, offsets):
    dt = DTYPES[dtype]
    groups = len(offsets) - 1 if offsets is not None else 0
    lead = (groups,) if groups else ()
    x, dz = rand(rows, k, dtype=dt, seed=5), rand(rows, n, dtype=dt, seed=6)
    w = torch.zeros(*lead, *((n, k) if transb else (k, n)), dtype=dt, device="cuda")
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda") if groups else None
    old = rand(*w.shape, dtype=torch.float32, seed=7)
    kw = dict(transb=transb, need_dx=False, need_dbias=False, dw=old.clone(), accumulate=True)
    _, dw, _ = dg.grouped_linear_grad(dz, x, w, off, **kw) if groups else dg.linear_grad(dz, x, w, **kw)
    for g, (lo, hi) in enumerate(spans(offsets, rows) if groups else [(0, rows)]):
        want, bound = ref.backward(dz[lo:hi], x[lo:hi], w[g] if groups else w, "none", None, 1.0, transb,
                                   torch.float32)["dw"]
        o = (old[g] if groups else old).cpu().double()
        check("dw %d" % g, dw[g] if groups else dw, want + o, bound + 2.0 ** -22 * (o.abs() + want.abs()))


def offsets_of(counts, before=0):
    out = [before]
    for c in counts:
        out.append(out[-1] + c)
    return out


# Tiles of 256 x 256 on 256 compute units, 32 per XCD: 143 tiles are whole ones,
# 81 are cut into halves, and quarters are what 9 tiles and the last of 272 give.
@pytest.mark.parametrize("transb", [False, True])
@pytest.mark.parametrize("size", [(3300, 2800, 72), (2100, 2060, 200), (4250, 4096, 136), (700, 600, 192)], ids=str)
def test_whole_tiles_halves_and_quarters(cuda, size, transb):
    m, n, k = size
    try:
        for split in (1, 2):
            assert dg.gemm_linear_force_config(0, split) == 0
            check_forward("bf16", m, n, k, transb=transb, act="silu", residual=True, pre=True)
            check_weight_grad("bf16", k, n, m, transb, None)
    finally:
        dg.gemm_linear_force_config()


GROUPS = {
    "last tiles of a few rows": [260, 512, 257, 1, 0, 300, 256, 770, 512, 3, 640, 129, 128, 127, 384],
    "only small tiles": [100, 7, 0, 128, 64] * 8,
    "one large": [3000, 1, 1, 1],
}


@pytest.mark.parametrize("transb", [False, True])
@pytest.mark.parametrize("name", GROUPS)
def test_quarters_of_groups(cuda, name, transb):
    offsets = offsets_of(GROUPS[name], 5)
    try:
        for n in (520, 2304):
            assert dg.gemm_linear_force_config(0) == 0
            check_forward("bf16", offsets[-1] + 9, n, 136, transb=transb, act="relu", residual=True, offsets=offsets)
    finally:
        dg.gemm_linear_force_config()


@pytest.mark.parametrize("groups", [5, 20, 70])
def test_weight_gradients_of_many_tiles(cuda, groups):
    """dw of groups with 9 tiles each: whole tiles, quarters in the last round
    (20), and more groups than a wave has lanes."""
    offsets = offsets_of([(37 * g) % 150 for g in range(groups)], 2)
    try:
        for split in (1, 2):
            assert dg.gemm_linear_force_config(0, split) == 0
            check_weight_grad("bf16", offsets[-1] + 3, 600, 520, False, offsets)
            check_weight_grad("bf16", offsets[-1] + 3, 600, 520, True, offsets)
    finally:
        dg.gemm_linear_force_config()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,n", [(1030, 40), (1500, 264), (8300, 2050), (8192, 2048)])
def test_bias_gradient_of_many_rows(cuda, dtype, rows, n):
    """Chunks of 16 and of 64 rows, one group and uneven ones."""
    for offsets in (None, offsets_of([rows // 3, 0, 1, rows // 2, 15], 4)):
        check_backward(dtype, rows, n, 24, act="silu", offsets=offsets)


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("transb", [False, True])
def test_gradients_against_differences(cuda, act, transb):
    """The directional derivative of L = <dy, y> along random signs v, from
    (L(+h) - L(-h)) / 2h at points that fp32 holds exactly.  It is off by h^2 / 6
    times the third derivative along v (those of the activations stay below 2),
    by the outputs' errors, each inside its bound, over h, and the gradient by
    its own bound."""
    m, n, k, h = 30, 40, 48, 2.0 ** -7
    exact = lambda *s, **kw: rand(*s, dtype=torch.bfloat16, **kw).float()  # noqa: E731
    at = dict(x=exact(m, k, seed=1), w=exact(*((n, k) if transb else (k, n)), seed=2, scale=k ** -0.5),
              b=exact(n, seed=3))
    dy = rand(m, n, dtype=torch.float32, seed=4)
    z = torch.empty(m, n, device="cuda")
    dg.linear(at["x"], at["w"], bias=at["b"], act=act, transb=transb, pre=z)
    got = dict(zip("xwb", dg.linear_grad(dy, at["x"], at["w"], act=act, pre=z, transb=transb)))
    bounds = ref.backward(dy, at["x"], at["w"], act, z, 1.0, transb, torch.float32)
    d, x64 = dy.cpu().double(), at["x"].cpu().double()
    w64 = (at["w"].t() if transb else at["w"]).cpu().double()
    for which, name in zip("xwb", ("dx", "dw", "dbias")):
        v = torch.sign(exact(*at[which].shape, seed=9) + 1e-30)
        ends, noise = [], 0.0
        for step in (h, -h):
            moved = dict(at)
            moved[which] = at[which] + step * v
            assert torch.equal(moved[which].double(), at[which].double() + step * v.double())
            y = dg.linear(moved["x"], moved["w"], bias=moved["b"], act=act, transb=transb)
            bound = ref.forward(moved["x"], moved["w"], moved["b"], act, None, 1.0, transb, torch.float32)[3]
            noise += float((d.abs() * bound).sum())
            ends.append(float((d * y.cpu().double()).sum()))
        v = v.cpu().double()
        along = {"x": lambda: v @ w64, "b": lambda: v.expand(m, n),
                 "w": lambda: x64 @ (v.t() if transb else v)}[which]()
        want = (ends[0] - ends[1]) / (2 * h)
        grad = float((got[which].cpu().double() * v).sum())
        limit = (float((d.abs() * along.abs() ** 3).sum()) * 2 * h * h / 6 + noise / (2 * h) +
                 float((bounds[name][1] * v.abs()).sum()))
        log("  %s: difference %.5f, gradient %.5f, limit %.3g" % (name, want, grad, limit))
        assert abs(grad - want) <= limit, name


OFFSETS = {
    "one group": [0, 90],
    "all in the middle": [0, 0, 90, 90],
    "single rows": [0, 1, 2, 3, 4, 5],
    "nobody": [0, 0, 0, 0],
    "rows outside": [7, 7, 40, 41, 80],
    "uneven": [0, 1, 34, 34, 67, 90],
}


@pytest.mark.parametrize("transb", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("name", OFFSETS)
def test_grouped(cuda, dtype, transb, name):
    check_forward(dtype, 90, 200, 72, transb=transb, act="gelu_tanh", residual=True, pre=True, offsets=OFFSETS[name])
    check_backward(dtype, 90, 200, 72, transb=transb, act="gelu_tanh", offsets=OFFSETS[name])


@pytest.mark.parametrize("groups", [64, 65, 200])
def test_many_groups(cuda, groups):
    """More groups than a wave has lanes, most of them small or empty."""
    gen = torch.Generator().manual_seed(groups)
    counts = torch.randint(0, 5, (groups,), generator=gen)
    counts[groups // 2] = 70
    offsets = [0] + torch.cumsum(counts, 0).tolist()
    for dtype in ("f32", "bf16"):
        check_forward(dtype, offsets[-1] + 3, 96, 64, act="silu", offsets=offsets)
        check_backward(dtype, offsets[-1] + 3, 96, 64, act="silu", offsets=offsets)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_offsets_outside_the_rows_are_clamped(cuda, dtype):
    """Offsets past the rows, negative or falling: what they leave of each
    group is computed, nothing outside the arrays is touched."""
    for offsets in ([-5, 20, 1000], [0, 30, 10, 10, 40], [50, 50, 1 << 30], [-7, -7, -3]):
        if offsets != [0, 30, 10, 10, 40]:     # there two groups claim the same rows
            check_forward(dtype, 50, 64, 48, offsets=offsets, act="relu")
        dt = DTYPES[dtype]
        off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
        g = len(offsets) - 1
        dx, dw, db = dg.grouped_linear_grad(rand(50, 64, dtype=dt, seed=1), rand(50, 48, dtype=dt, seed=2),
                                            rand(g, 48, 64, dtype=dt, seed=3), off)
        torch.cuda.synchronize()
        assert bool(torch.isfinite(dw).all()) and bool(torch.isfinite(db).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_offsets_that_claim_the_rows_many_times(cuda, dtype):
    """Falling offsets whose groups take all rows 300 times over: more tiles and
    chunks than offsets in order can have.  Guards around the outputs stay, and
    dw, whose blocks walk their own group only, is right."""
    dt, rows, n, k, g = DTYPES[dtype], 1200, 64, 48, 601
    off = torch.tensor([0, rows] * 301, dtype=torch.int32, device="cuda")
    x, dy = rand(rows, k, dtype=dt, seed=1), rand(rows, n, dtype=dt, seed=2)
    w = rand(1, k, n, dtype=dt, seed=3).expand(g, k, n).contiguous()
    whole = torch.full((rows + 8, n), 7.0, device="cuda")
    for cfg in range(dg.gemm_linear_num_configs(1 if dtype == "bf16" else 0)):
        if dg.gemm_linear_config_forms(1 if dtype == "bf16" else 0, cfg) & 1:
            dg.gemm_linear_force_config(cfg)
            try:
                dg.grouped_linear(x, w, off, out=whole[4:-4])
            finally:
                dg.gemm_linear_force_config()
            assert bool((whole[:4] == 7).all()) and bool((whole[-4:] == 7).all())
    dx, dw, db = dg.grouped_linear_grad(dy, x, w, off)
    want, bound = ref.backward(dy, x, w[0], "none", None, 1.0, False, torch.float32)["dw"]
    for i in (0, 300, 600):
        check("dw", dw[i], want, bound)
    assert not dw[1].any() and not dw[599].any()


@pytest.mark.parametrize("act", ref.ACTS)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_backward(cuda, dtype, act):
    for (m, n, k) in [(1, 64, 64), (2, 65, 33), (64, 128, 128), (65, 72, 200), (500, 260, 130)]:
        for transb in (False, True):
            check_backward(dtype, m, n, k, transb=transb, act=act, alpha=0.5)


def test_backward_parts_and_types(cuda):
    """Parts that are not asked for, and an input of another type for pre."""
    x, w = rand(40, 32, dtype=torch.bfloat16, seed=1), rand(32, 48, dtype=torch.bfloat16, seed=2)
    dy, z = rand(40, 48, dtype=torch.bfloat16, seed=3), rand(40, 48, dtype=torch.float32, seed=4)
    dx, dw, db = dg.linear_grad(dy, x, w, act="silu", pre=z)
    want = ref.backward(dy, x, w, "silu", z, 1.0, False, torch.float32)
    for name, got in (("dx", dx), ("dw", dw), ("dbias", db)):
        check(name, got, *want[name])
    for need in [(True, False, False), (False, True, False), (False, False, True), (False, False, False)]:
        part = dg.linear_grad(dy, x, w, act="silu", pre=z, need_dx=need[0], need_dw=need[1], need_dbias=need[2])
        for asked, whole, got in zip(need, (dx, dw, db), part):
            assert torch.equal(whole, got) if asked else got is None


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_empty(cuda, dtype):
    dt = DTYPES[dtype]
    e = lambda *s: torch.empty(*s, dtype=dt, device="cuda")  # noqa: E731
    assert dg.linear(e(0, 8), e(8, 16), bias=e(16)).shape == (0, 16)
    assert dg.linear(e(4, 8), e(8, 0)).shape == (4, 0)
    bias, res = rand(16, dtype=dt, seed=1), rand(4, 16, dtype=dt, seed=2)
    y = dg.linear(e(4, 0), e(0, 16), bias=bias, residual=res, act="relu", out_dtype=dt)   # no inputs: act(bias)
    want = (bias.double().clamp(min=0) + res.double())
    check("k = 0", y, want.cpu(), ref.half_step(dt) * want.abs().cpu() + 1e-30)
    dx, dw, db = dg.linear_grad(e(0, 16), e(0, 8), e(8, 16))
    assert dx.shape == (0, 8) and not dw.any() and not db.any()
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    dx, dw, db = dg.grouped_linear_grad(e(0, 16), e(0, 8), e(3, 8, 16), off, act="silu", pre=e(0, 16))
    assert dx.shape == (0, 8) and not dw.any() and not db.any() and db.shape == (3, 16)
    assert dg.grouped_linear(e(0, 8), e(3, 8, 16), off).shape == (0, 16)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_alpha_zero_does_not_read_the_operands(cuda, dtype):
    """alpha == 0: act(bias) + residual and zero gradients, whatever x and w
    hold, at pitches that would be copied to aligned rows otherwise."""
    dt = DTYPES[dtype]
    nan = lambda *s: torch.full(s, float("nan"), dtype=dt, device="cuda")  # noqa: E731
    bias = rand(301, dtype=dt, seed=1)
    y = dg.linear(nan(401, 501), nan(501, 301), bias=bias, act="relu", alpha=0.0, out_dtype=dt)
    assert torch.equal(y, torch.relu(bias).expand(401, 301))
    dx, dw, db = dg.linear_grad(rand(401, 301, dtype=dt, seed=2), nan(401, 501), nan(501, 301), alpha=0.0)
    assert not dx.any() and not dw.any() and bool(torch.isfinite(db).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", [(900, 1025, 1001), (520, 2047, 770), (2049, 515, 1030), (300, 4097, 2051)], ids=str)
def test_large_odd_sizes(cuda, dtype, size):
    """Rows below 16-byte alignment in products large enough to be copied to
    aligned rows first, dense and grouped, all three products."""
    m, n, k = size
    cuts = [0, m // 3, m // 3, m // 2, m - 7]
    for transb in (False, True):
        check_forward(dtype, m, n, k, transb=transb, act="silu", offsets=cuts)
        check_backward(dtype, m, n, k, transb=transb, act="gelu_tanh")
    check_forward(dtype, m, n, k, residual=True)
    check_backward(dtype, m, n, k, offsets=cuts)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_nan_and_infinity_stay_in_their_rows(cuda, dtype):
    """A NaN or an infinity in one row's input reaches that row's output only
    (and, in the gradients, its own group's), wherever a tile ends."""
    dt = DTYPES[dtype]
    rows, n, k = 100, 136, 80
    offsets = [0, 31, 64, 90]
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    w = rand(3, k, n, dtype=dt, seed=2)
    x = rand(rows, k, dtype=dt, seed=1)
    clean = dg.grouped_linear(x, w, off, act="silu", out=torch.zeros(rows, n, device="cuda"))
    bad = x.clone()
    bad[31, 5] = float("nan")
    bad[63] = float("inf")
    bad[90:] = float("nan")
    got = dg.grouped_linear(bad, w, off, act="silu", out=torch.zeros(rows, n, device="cuda"))
    keep = [r for r in range(rows) if r not in (31, 63)]
    assert torch.equal(got[keep], clean[keep])
    assert bool(torch.isnan(got[31]).all()) and not bool(torch.isfinite(got[63]).all())
    dy = rand(rows, n, dtype=dt, seed=3)
    dy[95] = float("nan")
    dx, dw, db = dg.grouped_linear_grad(dy, bad, w, off)
    assert bool(torch.isfinite(dw[0]).all()) and bool(torch.isfinite(dw[2]).all())
    assert bool(torch.isnan(dw[1][5]).all()) and bool(torch.isfinite(db).all())
    assert bool(torch.isfinite(dx[:90]).all())
    for act in ref.ACTS:      # a NaN before the activation stays one, forward and backward
        one = torch.full((1, 8), float("nan"), dtype=dt, device="cuda")
        eye = torch.eye(8, dtype=dt, device="cuda")
        assert bool(torch.isnan(dg.linear(one, eye, act=act)).all()), act
        if act != "none":
            dz = dg.linear_grad(torch.ones_like(one), torch.zeros_like(one), eye, act=act, pre=one, need_dw=False)[2]
            assert bool(torch.isnan(dz).all()), act
        if act != "none":    # far out the slopes are 0 and 1, not 0 x infinity
            far = torch.tensor([[-3e38, -1e20, -200.0, 200.0, 1e20, 3e38, float("inf"), float("-inf")]],
                               device="cuda").to(dt)
            slope = dg.linear_grad(torch.ones_like(far), torch.zeros_like(far), eye, act=act, pre=far,
                                   need_dw=False)[2]
            assert torch.equal(slope, torch.tensor([0., 0, 0, 1, 1, 1, 1, 0], device="cuda")), (act, slope)


def test_residual_in_place_and_same_bits(cuda):
    x, w = rand(200, 96, dtype=torch.bfloat16, seed=1), rand(96, 256, dtype=torch.bfloat16, seed=2)
    for dt in (torch.float32, torch.bfloat16):
        r = rand(200, 256, dtype=dt, seed=3)
        apart = dg.linear(x, w, act="gelu", residual=r, out_dtype=dt)
        for split in (1, 2):
            dg.gemm_linear_force_config(-1, split)
            try:
                whole = dg.linear(x, w, act="gelu", residual=r, out_dtype=dt)
                y = r.clone()
                dg.linear(x, w, act="gelu", residual=y, out=y)
                assert torch.equal(y, whole)
                assert torch.equal(whole, dg.linear(x, w, act="gelu", residual=r, out_dtype=dt))
            finally:
                dg.gemm_linear_force_config()
        assert apart.dtype == dt


def test_offsets_beyond_32_bits(cuda):
    """Weights of more than 2^32 bytes and 2^31 elements: the last group's."""
    g, k, n = 5, 32768, 16384
    w = torch.zeros(g, k, n, dtype=torch.bfloat16, device="cuda")
    assert w.numel() > 1 << 31
    w[4] = rand(k, n, dtype=torch.bfloat16, seed=1, scale=k ** -0.5)
    x = rand(5, k, dtype=torch.bfloat16, seed=2)
    off = torch.tensor([0, 1, 1, 1, 2, 5], dtype=torch.int32, device="cuda")
    y = dg.grouped_linear(x, w, off)
    cols = torch.arange(0, n, 97, device="cuda")
    _, want, _, bound = ref.forward(x[2:], w[4][:, cols], None, "none", None, 1.0, False, torch.float32)
    check("last group", y[2:][:, cols], want, bound)
    assert not y[:2].any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_expert_layers_together(cuda, dtype):
    """A routed feed-forward layer as a model runs it -- two grouped layers
    with a dense one behind them and a residual -- forward and backward against
    the same network differentiated by torch in 64 bits on the CPU.  The bound
    follows the roundings of the stored values: with h the half step of the
    type, every one of the at most 8 stored values on the way to a gradient is
    off by h relative to its row's magnitude, so the norm is off by less than
    8 h and a part in 10^4 for the fp32 sums (f32: the latter alone)."""
    dt = DTYPES[dtype]
    rows, d, f, offsets = 150, 96, 200, [0, 40, 40, 41, 120, 150]
    g = len(offsets) - 1
    x = rand(rows, d, dtype=dt, seed=1)
    w1, b1 = rand(g, d, f, dtype=dt, seed=2, scale=d ** -0.5), rand(g, f, dtype=dt, seed=3)
    w2, b2 = rand(g, d, f, dtype=dt, seed=4, scale=f ** -0.5), rand(g, d, dtype=dt, seed=5)
    w3 = rand(d, d, dtype=dt, seed=6, scale=d ** -0.5)
    dy = rand(rows, d, dtype=dt, seed=7)
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    z1 = torch.empty(rows, f, dtype=dt, device="cuda")
    z3 = torch.empty(rows, d, dtype=dt, device="cuda")
    h1 = dg.grouped_linear(x, w1, off, bias=b1, act="silu", pre=z1, out_dtype=dt)
    h2 = dg.grouped_linear(h1, w2, off, bias=b2, transb=True, residual=x, out_dtype=dt)
    y = dg.linear(h2, w3, act="gelu_tanh", pre=z3, out_dtype=dt)
    dh2, dw3, _ = dg.linear_grad(dy, h2, w3, act="gelu_tanh", pre=z3, out_dtype=dt)
    dh1, dw2, db2 = dg.grouped_linear_grad(dh2, h1, w2, off, transb=True, out_dtype=dt)
    dx, dw1, db1 = dg.grouped_linear_grad(dh1, x, w1, off, act="silu", pre=z1, out_dtype=dt)
    dx = dx.double() + dh2.double()
    torch.cuda.synchronize()
    leaves = [t.cpu().double().requires_grad_() for t in (x, w1, b1, w2, b2, w3)]
    X, W1, B1, W2, B2, W3 = leaves
    parts = []
    for i, (lo, hi) in enumerate(zip(offsets[:-1], offsets[1:])):
        h = torch.nn.functional.silu(X[lo:hi] @ W1[i] + B1[i])
        parts.append(h @ W2[i].T + B2[i] + X[lo:hi])
    out = torch.nn.functional.gelu(torch.cat(parts) @ W3, approximate="tanh")
    out.backward(dy.cpu().double())
    limit = 1e-4 if dtype == "f32" else 8 * ref.half_step(dt) + 1e-4
    for name, got, want in [("y", y, out.detach())] + [
            (n, got, leaf.grad) for n, got, leaf in zip("dx dw1 db1 dw2 db2 dw3".split(),
                                                        (dx, dw1, db1, dw2, db2, dw3), leaves)]:
        rel = float((got.cpu().double() - want).norm() / want.norm())
        log("  %s: %.2e" % (name, rel))
        assert rel <= limit, (name, rel)


def test_graph_replays_with_new_rows_and_offsets(cuda):
    """Forward and backward captured once, no workspace shared with another
    capture, replayed with other inputs and another division into groups."""
    dt = torch.bfloat16
    rows, d, f, g = 128, 256, 512, 8
    x, dy = rand(rows, d, dtype=dt, seed=1), rand(rows, f, dtype=dt, seed=2)
    w = rand(g, d, f, dtype=dt, seed=3, scale=d ** -0.5)
    bias = rand(g, f, dtype=dt, seed=4)
    off = torch.tensor([0, 16, 32, 48, 64, 80, 96, 112, 128], dtype=torch.int32, device="cuda")
    wd = rand(d, f, dtype=dt, seed=5, scale=d ** -0.5)

    def step():
        z = torch.empty(rows, f, dtype=dt, device="cuda")
        y = dg.grouped_linear(x, w, off, bias=bias, act="silu", pre=z, out_dtype=dt)
        grads = dg.grouped_linear_grad(dy, x, w, off, act="silu", pre=z, out_dtype=dt)
        one = dg.linear(x[:4], wd, act="gelu", out_dtype=dt)
        return (y, one, *grads, *dg.linear_grad(dy, x, wd, out_dtype=dt))

    step()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            graphs.append((graph, step()))
    cuts = [[0, 0, 1, 2, 60, 60, 61, 120, 128], [0, 128, 128, 128, 128, 128, 128, 128, 128],
            [0, 16, 32, 48, 64, 80, 96, 112, 128]]
    for rep, cut in enumerate(cuts):
        x.copy_(rand(rows, d, dtype=dt, seed=10 + rep))
        dy.copy_(rand(rows, f, dtype=dt, seed=20 + rep))
        off.copy_(torch.tensor(cut, dtype=torch.int32))
        torch.cuda.synchronize()
        # both graphs at once, on streams of their own
        streams = [torch.cuda.Stream() for _ in graphs]
        for (graph, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        eager = step()
        torch.cuda.synchronize()
        for _, outs in graphs:
            for i, (a, b) in enumerate(zip(outs, eager)):
                assert torch.equal(a, b), (rep, i)


def test_streams(cuda):
    """On a stream that is not torch's current one, given by handle: the
    temporaries live until that stream is done with them."""
    x, w = rand(48, 4096, dtype=torch.bfloat16, seed=1), rand(1024, 4096, dtype=torch.bfloat16, seed=2)
    dy, z = rand(48, 1024, dtype=torch.bfloat16, seed=3), rand(48, 1024, dtype=torch.bfloat16, seed=4)
    want = (dg.linear(x, w, transb=True, act="silu"), *dg.linear_grad(dy, x, w, act="silu", pre=z, transb=True))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        got = (dg.linear(x, w, transb=True, act="silu", stream=s.cuda_stream),
               *dg.linear_grad(dy, x, w, act="silu", pre=z, transb=True, stream=s.cuda_stream))
        junk = [torch.full((1 << 20,), float("nan"), device="cuda") for _ in range(8)]
        s.synchronize()
        torch.cuda.synchronize()
        del junk
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_refusals(cuda):
    x, w = rand(6, 8, dtype=torch.float32, seed=1), rand(8, 16, dtype=torch.float32, seed=2)
    off = torch.tensor([0, 2, 6], dtype=torch.int32, device="cuda")
    w3 = torch.stack([w, w])
    for bad in [lambda: dg.linear(x, w.t()), lambda: dg.linear(x, w, bias=torch.zeros(8, device="cuda")),
                lambda: dg.linear(x, w, act="tanh"), lambda: dg.linear(x, w, residual=x),
                lambda: dg.linear(x, w.t().contiguous().t()), lambda: dg.linear(x, w, pre=torch.zeros(6, 15, device="cuda")),
                lambda: dg.linear(x, w3), lambda: dg.grouped_linear(x, w, off),
                lambda: dg.grouped_linear(x, w3, off[:2]), lambda: dg.grouped_linear(x, w3, off.long()),
                lambda: dg.grouped_linear(x, w3, off.cpu()), lambda: dg.linear(x.cpu(), w),
                lambda: dg.linear(x, w.cpu()), lambda: dg.linear_grad(x, x, w),
                lambda: dg.linear_grad(torch.zeros(6, 16, device="cuda"), x, w, act="silu"),
                lambda: dg.linear_grad(torch.zeros(6, 16, device="cuda"), x, w, accumulate=True)]:
        with pytest.raises(ValueError):
            bad()
    for bad in [lambda: dg.linear(x, w.bfloat16()), lambda: dg.linear(x.double(), w.double()),
                lambda: dg.linear(x, w, out_dtype=torch.float16),
                lambda: dg.linear(x, w, residual=torch.zeros(6, 16, device="cuda"), out_dtype=torch.bfloat16),
                lambda: dg.linear(x, w, bias=torch.zeros(16, device="cuda", dtype=torch.float16))]:
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(dg.GemmError):      # rows that overlap
        dg.linear(torch.zeros(1, 8, device="cuda").expand(6, 8), w)
