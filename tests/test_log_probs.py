"""Log probabilities with entropy and alternatives, and their gradient, against
their definition in 64 bits (serving_ref, where the bounds are derived): sizes at
the edges of vectors, chunks and parts, alignments, forbidden places, empty rows,
the type's lowest value, NaN and infinity, ties, padding tokens, streams, graphs;
and, without a GPU, what the calls refuse."""
from __future__ import annotations

import math

import pytest
import torch

import dense_gemm_03_amd as dg
from tests import serving_ref as ref

BAD = dg.GEMM_ERR_INVALID_ARG
P = 1 << 20     # stands in for a 16-byte aligned device address: refused calls read nothing
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
INF = math.inf


def params(**kw):
    p = dict(dtype=1, top=5, scale=1.0, reserved=0, rows=10, vocab=1000, ld=1000)
    p.update(kw)
    return dg.LogProbsParams(**p)


# ------------------------------------------------------------ without a GPU --

BAD_PARAMS = [dict(dtype=2), dict(dtype=-1), dict(top=-1), dict(top=65), dict(top=20, vocab=19), dict(scale=0.0),
              dict(scale=-1.0), dict(scale=INF), dict(scale=math.nan), dict(scale=2.0 ** 65), dict(rows=-1), dict(rows=(1 << 30) + 1),
              dict(vocab=0, top=0), dict(vocab=(1 << 30) + 1, ld=1 << 31), dict(ld=999), dict(ld=(1 << 40) + 1)]


def forward(p, z=P, tok=P, lp=P, ent=P, st=P, ids=P, tl=P, ws=P, n=1 << 40):
    return dg.gemm_log_probs(p, z, tok, lp, ent, st, ids, tl, ws, n)


def grad(p, z=P, tok=P, st=P, ent=P, g=P, h=P, dz=P + (1 << 30), ldd=1000):
    return dg.gemm_log_probs_grad(p, z, tok, st, ent, g, h, dz, ldd)


@pytest.mark.parametrize("kw", BAD_PARAMS, ids=str)
def test_bad_parameters(kw):
    p = params(**kw)
    assert forward(p) == BAD and grad(p, ldd=1 << 31) == BAD
    assert dg.gemm_log_probs_workspace_size(p) == BAD


def test_bad_arguments():
    for kw in (dict(z=None), dict(tok=None), dict(lp=None), dict(ids=None), dict(z=P + 1), dict(tok=P + 2),
               dict(lp=P + 1), dict(ent=P + 2), dict(st=P + 3), dict(ids=P + 1), dict(tl=P + 2)):
        assert forward(params(), **kw) == BAD, kw
    assert forward(params(dtype=0), z=P + 2) == BAD
    parted = params(rows=1, vocab=131072, ld=131072)
    need = dg.gemm_log_probs_workspace_size(parted)
    assert need > 0
    for kw in (dict(ws=None), dict(ws=P + 8), dict(n=need - 1)):
        assert forward(parted, **kw) == BAD, kw
    for kw in (dict(z=None), dict(st=None), dict(dz=None), dict(tok=None), dict(ent=None), dict(z=P + 1),
               dict(dz=P + 1), dict(tok=P + 1), dict(st=P + 2), dict(ent=P + 2), dict(g=P + 2), dict(h=P + 1),
               dict(ldd=999), dict(dz=P, ldd=1001)):
        assert grad(params(), **kw) == BAD, kw
    assert dg.gemm_log_probs_workspace_size(None) == BAD
    assert dg.gemm_log_probs(None, P, P, P, P, P, P, P, P, 0) == BAD
    assert dg.gemm_log_probs_grad(None, P, P, P, P, P, P, P, 1000) == BAD


def test_no_rows():
    assert forward(params(rows=0), None, None, None, None, None, None, None, None, 0) == dg.GEMM_OK
    assert grad(params(rows=0), None, None, None, None, None, None, None) == dg.GEMM_OK


def test_helpers_refuse():
    with pytest.raises(ValueError):
        dg.log_probs(torch.zeros(4, 8))
    with pytest.raises(ValueError):
        dg.log_probs_grad(torch.zeros(4, 8), None, torch.zeros(4, 2))


def test_reference_against_torch():
    gen = torch.Generator().manual_seed(1)
    z = torch.randn(6, 50, generator=gen, dtype=torch.float64) * 3
    tokens = torch.randint(0, 50, (6,), generator=gen)
    want = torch.log_softmax(0.7 * z, dim=1)
    got = ref.log_probs(z, tokens, 50, 0.7)
    assert torch.allclose(got["logprob"][0][:, 0], want[torch.arange(6), tokens], atol=1e-13)
    assert torch.allclose(got["entropy"][0][:, 0], -(want.exp() * want).sum(1), atol=1e-13)
    assert torch.equal(got["top_ids"], z.argsort(dim=1, descending=True))


def test_reference_gradient_against_differences():
    """A central difference with step h is off by at most h^2 / 6 times the third
    derivative (below 10 here) and 1e-15 / h of rounding."""
    gen = torch.Generator().manual_seed(2)
    z = torch.randn(3, 9, generator=gen, dtype=torch.float64)
    tokens = torch.tensor([2, -1, 8])
    g, h = torch.randn(3, generator=gen, dtype=torch.float64), torch.randn(3, generator=gen, dtype=torch.float64)

    def value(x):
        f = ref.log_probs(x, tokens, 0, 1.3)
        return (g[:, None] * f["logprob"][0] + h[:, None] * f["entropy"][0]).sum()

    f = ref.log_probs(z, tokens, 0, 1.3)
    got, _ = ref.log_probs_grad(z, tokens, torch.cat([f["m"][0], f["L"][0]], 1), f["entropy"][0][:, 0], g, h, 1.3)
    step = 1e-4
    for i in range(3):
        for j in range(9):
            e = torch.zeros_like(z)
            e[i, j] = step
            assert abs(float((value(z + e) - value(z - e)) / (2 * step) - got[i, j])) < 1e-6


# -------------------------------------------------------------- on the GPU --

def rand(rows, vocab, dtype, seed, pad=0, shift=0):
    """Logits, as a view with `pad` values behind each row and `shift` before the first."""
    gen = torch.Generator().manual_seed(seed)
    z = (torch.randn(rows, vocab, generator=gen) * 2.5).to(DTYPES[dtype])
    wide = torch.full((rows * (vocab + pad) + shift,), math.nan, dtype=DTYPES[dtype], device="cuda")
    view = wide[shift:].view(rows, vocab + pad)[:, :vocab]
    view.copy_(z)
    return view


def check(z, tokens, top, scale=1.0, **kw):
    got = dg.log_probs(z, tokens, top, scale=scale, **kw)
    torch.cuda.synchronize()
    want = ref.log_probs(z, tokens, top, scale)
    compare = lambda what, g, w: _compare(what, g, *w)  # noqa: E731
    compare("m", got.stats[:, :1], want["m"])
    compare("L", got.stats[:, 1:], want["L"])
    compare("entropy", got.entropy[:, None], want["entropy"])
    if tokens is not None:
        compare("logprob", got.logprob[:, None], want["logprob"])
    else:
        assert got.logprob is None
    if top:
        assert torch.equal(got.top_ids.cpu().long(), want["top_ids"])
        compare("top_logprobs", got.top_logprobs, want["top_logprobs"])
    return got


def _compare(what, got, want, bound):
    g = got.cpu().double()
    # NaN, and infinities: a value beyond the type's range (scale times the lowest value) rounds to one
    same = (g == want.to(got.dtype).double()) | (torch.isnan(g) & torch.isnan(want))
    r = torch.where(same, torch.zeros_like(g), (g - want).abs() / bound)
    r = float(torch.nan_to_num(r, nan=INF).max()) if r.numel() else 0.0
    assert r <= 1.0, "%s: error %.3g of its bound" % (what, r)


def check_grad(z, tokens, scale=1.0, entropy=True, logprob=True, seed=3, out=None):
    gen = torch.Generator().manual_seed(seed)
    rows = z.shape[0]
    g = torch.randn(rows, generator=gen).cuda() if logprob else None
    h = torch.randn(rows, generator=gen).cuda() if entropy else None
    f = dg.log_probs(z, tokens, scale=scale)
    want, bound = ref.log_probs_grad(z, tokens, f.stats, f.entropy, g, h, scale)
    got = dg.log_probs_grad(z, tokens, f.stats, f.entropy, g, h, scale=scale, out=out)
    torch.cuda.synchronize()
    assert got.dtype == z.dtype
    _compare("dlogits", got, want, bound)
    return got


def token_row(rows, vocab, seed=5):
    gen = torch.Generator().manual_seed(seed)
    t = torch.randint(0, vocab, (rows,), generator=gen, dtype=torch.int32)
    if rows > 2:
        t[1], t[2] = -1, vocab
    return t.cuda()


SIZES = [(1, 1, 1), (2, 2, 2), (1, 7, 7), (3, 64, 5), (5, 63, 63), (4, 100, 64), (2, 2048, 20), (2, 2049, 1),
         (3, 4099, 33), (1, 8192, 64), (7, 9001, 20), (1, 131072, 20), (2, 100003, 64), (40, 20011, 5),
         (300, 3001, 8), (4200, 74, 3), (4100, 5003, 6), (1, 524293, 17)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_sizes(cuda, dtype, size):
    rows, vocab, top = size
    z, t = rand(rows, vocab, dtype, rows + vocab), token_row(rows, vocab)
    check(z, t, top, scale=0.8)
    if rows * vocab <= 1 << 21:
        check_grad(z, t, scale=0.8)


@pytest.mark.gpu
@pytest.mark.parametrize("shift", [0, 1, 3, 8])
@pytest.mark.parametrize("pad", [0, 1, 2, 13])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_alignments(cuda, dtype, pad, shift):
    """Rows at every kind of address; what lies before, between and behind them
    (NaN) is neither used nor written."""
    for rows, vocab in ((9, 333), (3, 6007)):
        z, t = rand(rows, vocab, dtype, 11, pad, shift), token_row(rows, vocab)
        check(z, t, 9)
        for extra in (0, 1, 4):
            wide = torch.full((rows, vocab + extra + 3), 7.0, dtype=z.dtype, device="cuda")
            check_grad(z, t, out=wide[:, extra:extra + vocab])
            assert bool((wide[:, :extra] == 7.0).all()) and bool((wide[:, extra + vocab:] == 7.0).all())


@pytest.mark.gpu
def test_without_tokens_or_top(cuda):
    z = rand(6, 3000, "f32", 1)
    check(z, None, 4)
    check(z, None, 0)
    check(z, token_row(6, 3000), 0)
    check_grad(z, None, logprob=False)
    check_grad(z, token_row(6, 3000), entropy=False)
    f = dg.log_probs(z)
    assert bool((dg.log_probs_grad(z, None, f.stats) == 0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("vocab", [50, 5000, 70001])
def test_masks(cuda, dtype, vocab):
    """Forbidden places, rows of nothing else, of one place, of the lowest value,
    of huge and far apart logits."""
    z = rand(10, vocab, dtype, 4)
    low = torch.finfo(z.dtype).min
    z[0] = -INF
    z[1] = -INF
    z[1, vocab - 1] = 2.0
    z[2] = low
    z[3] = low
    z[3, 5] = 1.0
    z[4, ::2] = -INF
    z[5] = -INF
    z[5, 3:40] = low
    z[6] = z[6] * 1000
    z[7] = 0.0
    z[8, :] = torch.finfo(z.dtype).max
    z[9, : vocab // 2] = low
    t = torch.tensor([3, vocab - 1, 7, 5, 1, 10, 0, vocab - 1, 2, vocab - 2], dtype=torch.int32, device="cuda")
    for scale in (1.0, 0.25, 3.0):
        check(z, t, 12, scale=scale)
        check_grad(z, t, scale=scale)
    forbidden = torch.tensor([0, 0, 0, 0, 2, 1, 0, 0, 0, 0], dtype=torch.int32, device="cuda")
    got = check(z, forbidden, 0)
    assert got.logprob[0] == -INF and got.logprob[1] == -INF and got.logprob[4] == -INF and got.entropy[0] == 0.0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("vocab", [60, 20000])
def test_nan_and_infinity(cuda, dtype, vocab):
    z = rand(6, vocab, dtype, 4)
    z[0, 17] = math.nan
    z[1, 33] = INF
    z[2] = math.nan
    z[3, 7], z[3, 9] = -INF, math.nan
    z[4, 2], z[4, 50] = INF, INF
    t = torch.tensor([1, 2, 3, 7, 5, 6], dtype=torch.int32, device="cuda")
    got = check(z, t, 6)
    assert torch.isnan(got.logprob[:5]).all() and torch.isfinite(got.logprob[5])
    # a padded row's gradient is zero whatever the row holds
    pad = torch.full((6,), -1, dtype=torch.int32, device="cuda")
    g = torch.ones(6, device="cuda")
    assert bool((dg.log_probs_grad(z, pad, got.stats, dlogprob=g) == 0).all())
    assert torch.isnan(dg.log_probs_grad(z, t, got.stats, dlogprob=g)[:5]).any(dim=1).all()


@pytest.mark.gpu
@pytest.mark.parametrize("vocab", [70, 3000, 20000])
def test_nan_among_the_alternatives(cuda, vocab):
    """NaN ranks with -infinity, by place, wherever the list has to take either."""
    gen = torch.Generator().manual_seed(7)
    kind = torch.randint(0, 2, (8, vocab), generator=gen)
    z = torch.where(kind == 0, torch.tensor(-INF), torch.tensor(math.nan))
    z[1:4, ::vocab // 9] = 1.0
    z[4, -5:] = 2.0
    for dtype in DTYPES.values():
        for top in (3, 20, 64):
            got = dg.log_probs(z.to(dtype).cuda(), None, top)
            assert torch.equal(got.top_ids.cpu().long(), ref.ranks(z.double(), top))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows", [1, 4100])
def test_ties_and_orders(cuda, dtype, rows):
    """Equal logits by place, rows that rise (every value enters the list) and fall."""
    vocab = 9001
    for top in (1, 20, 64):
        base = torch.arange(vocab, device="cuda", dtype=torch.float32)
        for z in (torch.zeros(1, vocab), base.cpu()[None] / 16, -base.cpu()[None] / 16, (base.cpu() % 7)[None],
                  torch.where(base.cpu() % 2 == 0, 0.0, -0.0)[None]):
            z = z.to(DTYPES[dtype]).cuda().repeat(rows, 1)
            got = dg.log_probs(z, None, top)
            want = ref.ranks(z[:1].cpu().double(), top)
            assert torch.equal(got.top_ids.cpu().long(), want.expand(rows, top))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gradient_in_place(cuda, dtype):
    z, t = rand(33, 5001, dtype, 8), token_row(33, 5001)
    f = dg.log_probs(z, t)
    g, h = torch.randn(33, device="cuda"), torch.randn(33, device="cuda")
    want = dg.log_probs_grad(z, t, f.stats, f.entropy, g, h)
    got = dg.log_probs_grad(z, t, f.stats, f.entropy, g, h, out=z)
    assert got is z and torch.equal(got, want)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("base", [1e4, 1e6, 1e7, 1.2e7, 3e7, 1e9, 1e13, 1e20, 1e30, 1e37, -1e7, -1e20])
def test_large_logits_close_together(cuda, dtype, base):
    """Logits of any size whose scaled distances are ordinary, or large: rows of one sign,
    and rows that climb from small values to large ones."""
    gen = torch.Generator().manual_seed(5)
    step = abs(base) * torch.finfo(dtype).eps
    z = base + step * torch.randint(-40, 41, (6, 3001), generator=gen).double()
    z[4, :2000] = torch.linspace(0, 1, 2000).double() * base
    z[5] = base * torch.linspace(0.5, 1, 3001).double()
    z = z.to(dtype).cuda()
    t = torch.tensor([0, 5, 2999, -1, 2500, 3000], dtype=torch.int32, device="cuda")
    for rows in (6, 1):
        for scale in (0.3, 3.0, 7.0, 30.0, 300.0, 1e6, 1e15):
            if scale / step <= 2.0 ** 64:
                check(z[-rows:], t[-rows:], 5, scale=scale / step)
        check_grad(z[-rows:], t[-rows:], scale=0.3 / step)


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [2.0 ** 64, 2.0 ** 40, 2.0 ** -60, 2.0 ** -140])
def test_extreme_scales(cuda, scale):
    z = torch.randn(5, 2500, generator=torch.Generator().manual_seed(2)).cuda()
    t = torch.tensor([0, 7, 100, 2499, 3], dtype=torch.int32, device="cuda")
    t[1] = z[1].argmax()
    check(z, t, 3, scale=scale)


@pytest.mark.gpu
def test_gradient_against_differences(cuda):
    """The kernels' own values at z +- step: fp32 log probabilities are off by some
    2^-23, their difference over 2 step = 1/16 by 2^-18, and the difference quotient by
    step^2 / 6 of a third derivative below 2."""
    z = rand(1, 40, "f32", 6)
    t = torch.tensor([11], dtype=torch.int32, device="cuda")
    f = dg.log_probs(z, t)
    one = torch.ones(1, device="cuda")
    dz = dg.log_probs_grad(z, t, f.stats, f.entropy, one, 0.5 * one)
    step = 1 / 32
    both = torch.cat([z + step * torch.eye(40, device="cuda"), z - step * torch.eye(40, device="cuda")])
    v = dg.log_probs(both, t.repeat(80))
    v = (v.logprob + 0.5 * v.entropy).double()
    diff = (v[:40] - v[40:]) / (2 * step)
    assert float((diff - dz[0].double()).abs().max()) < step ** 2 / 3 + 2.0 ** -16


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_far_apart(cuda, dtype):
    """Offsets beyond 32 bits."""
    ld, vocab = (1 << 31) + 24, 4100
    wide = torch.empty(2 * ld + vocab, dtype=DTYPES[dtype], device="cuda")
    z = wide.as_strided((3, vocab), (ld, 1))
    z.copy_(rand(3, vocab, dtype, 2))
    t = token_row(3, vocab)
    check(z, t, 5)
    same = z.contiguous()
    f = dg.log_probs(same, t)
    one = torch.ones(3, device="cuda")
    want = dg.log_probs_grad(same, t, f.stats, f.entropy, one, one)
    assert torch.equal(dg.log_probs_grad(z, t, f.stats, f.entropy, one, one, out=z), want)


@pytest.mark.gpu
def test_streams_and_graphs(cuda):
    """Another stream, a captured graph replayed with eager calls between, two graphs."""
    z, t = rand(3, 100003, "bf16", 9), token_row(3, 100003)
    g = torch.ones(3, device="cuda")
    want = dg.log_probs(z, t, 20)
    wantg = dg.log_probs_grad(z, t, want.stats, dlogprob=g)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = dg.log_probs(z, t, 20, stream=s.cuda_stream)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs, outs, ins = [], [], []
    for i in range(2):
        zi = z.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            f = dg.log_probs(zi, t, 20)
            d = dg.log_probs_grad(zi, t, f.stats, dlogprob=g)
        graphs.append(graph), outs.append((f, d)), ins.append(zi)
    other = rand(3, 100003, "bf16", 10)
    want2 = dg.log_probs(other, t, 20)
    want2g = dg.log_probs_grad(other, t, want2.stats, dlogprob=g)
    for k in range(3):
        ins[0].copy_(z if k % 2 == 0 else other)
        ins[1].copy_(other if k % 2 == 0 else z)
        graphs[0].replay(), graphs[1].replay()
        eager = dg.log_probs(z, t, 20)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(eager, want))
        for i in range(2):
            w, wg = (want, wantg) if (k + i) % 2 == 0 else (want2, want2g)
            assert all(torch.equal(a, b) for a, b in zip(outs[i][0], w)) and torch.equal(outs[i][1], wg)


@pytest.mark.gpu
def test_two_streams_at_once(cuda):
    """Calls on two streams at a time, of rows in parts and of whole rows."""
    zs = [rand(3, 100003, "bf16", 9), rand(2100, 5003, "f32", 8)]
    ts = [token_row(3, 100003), token_row(2100, 5003)]
    want = [dg.log_probs(z, t, 20) for z, t in zip(zs, ts)]
    streams = [torch.cuda.Stream() for _ in zs]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(10):
        got = [dg.log_probs(z, t, 20, stream=s.cuda_stream) for z, t, s in zip(zs, ts, streams)]
        for s in streams:
            s.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(a, b) for a, b in zip(g, w))


@pytest.mark.gpu
def test_helper_checks(cuda):
    z, t = rand(4, 100, "f32", 1), token_row(4, 100)
    for bad in (lambda: dg.log_probs(z, t.long()), lambda: dg.log_probs(z.half(), t)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: dg.log_probs(z, t[:3]), lambda: dg.log_probs(z, t, 65), lambda: dg.log_probs(z, t, 101),
                lambda: dg.log_probs(z, t, scale=0.0), lambda: dg.log_probs(z.t(), None),
                lambda: dg.log_probs(z, t.cpu()), lambda: dg.log_probs(z[0], None),
                lambda: dg.log_probs_grad(z, None, torch.zeros(4, 2, device="cuda"), dlogprob=torch.ones(4, device="cuda")),
                lambda: dg.log_probs_grad(z, t, torch.zeros(4, 2, device="cuda"), dentropy=torch.ones(4, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    none = dg.log_probs(z[:0], t[:0], 3)
    assert none.logprob.shape == (0,) and none.top_ids.shape == (0, 3)
    assert dg.log_probs_grad(z[:0], t[:0], none.stats).shape == (0, 100)
