"""Linear layers with a low-rank adapter per row against their definition in 64 bits
(serving_ref, where the bounds are derived): rows of one and of many adapters through
every kernel of the table, ranks and widths at the edges of steps and strips, pitches
and alignments, rows without adapters, streams, graphs; a decoding step of this and the
operators next to it; and, without a GPU, what the calls refuse."""
from __future__ import annotations

import math

import pytest
import torch

import dense_gemm_03_amd as dg
from tests import serving_ref as ref
from tests.gpu_util import log

BAD = dg.GEMM_ERR_INVALID_ARG
P = 1 << 20     # stands in for a 16-byte aligned device address: refused calls read nothing
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def params(**kw):
    """A valid layer: 100 rows, 64 inputs, 48 outputs, 5 adapters of rank 16, bf16."""
    p = dict(dtype=1, dtype_y=1, dtype_bias=0, transw=0, act=dg.GEMM_ACT_SILU, reserved=0, rows=100, N=48, K=64,
             adapters=5, rank=16, ldx=64, ldw=48, ldy=48, ldr=48, lda=64, ldb=16, stride_a=16 * 64, stride_b=48 * 16)
    p.update(kw)
    return dg.AdapterParams(**p)


def call(p, x=P, w=P, a=P, b=P, ids=P, scales=P, bias=P, res=P + 4096, y=P + 4096, ws=P, n=1 << 40):
    return dg.gemm_adapter_linear(p, x, w, a, b, ids, scales, bias, res, y, ws, n)


BAD_PARAMS = [dict(dtype=2), dict(dtype_y=-1), dict(dtype_bias=3), dict(transw=2), dict(act=5), dict(rows=-1), dict(N=-1),
              dict(K=-1), dict(rows=(1 << 30) + 1), dict(adapters=-1), dict(rank=-1), dict(rank=4097, ldb=4097),
              dict(ldx=63), dict(ldw=47), dict(lda=63), dict(lda=(1 << 24) + 1), dict(ldb=15), dict(stride_a=16 * 64 - 1),
              dict(stride_b=48 * 16 - 1), dict(transw=1, ldw=63)]


@pytest.mark.parametrize("kw", BAD_PARAMS, ids=str)
def test_bad_parameters(kw):
    assert call(params(**kw)) == BAD
    assert dg.gemm_adapter_linear_workspace_size(params(**kw)) == BAD


def test_bad_arguments():
    need = dg.gemm_adapter_linear_workspace_size(params())
    assert need >= 100 * 16 * 4
    for kw in (dict(x=None), dict(w=None), dict(a=None), dict(b=None), dict(ids=None), dict(y=None), dict(ws=None),
               dict(ws=P + 8), dict(n=need - 1), dict(x=P + 1), dict(w=P + 1), dict(a=P + 1), dict(b=P + 1),
               dict(ids=P + 2), dict(scales=P + 1), dict(bias=P + 2), dict(res=P + 1), dict(y=P + 1)):
        assert call(params(), **kw) == BAD, kw
    for kw in (dict(ldy=47), dict(ldr=47), dict(ldr=49)):      # the last: in place with another pitch
        assert call(params(**kw)) == BAD, kw
    assert call(None) == BAD and dg.gemm_adapter_linear_workspace_size(None) == BAD


def test_empty_calls_launch_nothing():
    assert call(params(rows=0), None, None, None, None, None, None, None, None, None, None, 0) == dg.GEMM_OK
    assert call(params(N=0, stride_b=0), None, None, None, None, None, None, None, None, None, None, 0) == dg.GEMM_OK


def test_without_adapters_it_needs_what_the_layer_needs():
    for kw in (dict(adapters=0), dict(rank=0)):
        layer = dg.LinearParams(1, 1, 0, 0, dg.GEMM_ACT_SILU, 1.0, 100, 48, 64, 0, 64, 48, 48, 48, 0, 0, 0)
        assert dg.gemm_adapter_linear_workspace_size(params(**kw)) == dg.gemm_linear_workspace_size(layer)


def test_helper_refuses_host_tensors():
    with pytest.raises(ValueError):
        dg.adapter_linear(torch.zeros(2, 8), torch.zeros(8, 6), torch.zeros(3, 4, 8), torch.zeros(3, 6, 4),
                          torch.zeros(2).int())


# -------------------------------------------------------------- on the GPU --

def rand(*shape, dtype, seed, scale=1.0):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=gen) * scale).to(DTYPES[dtype]).cuda()


def padded(t, extra):
    """t with `extra` NaN behind each row."""
    if not extra:
        return t
    wide = torch.full((*t.shape[:-1], t.shape[-1] + extra), math.nan, dtype=t.dtype, device=t.device)
    wide[..., :t.shape[-1]] = t
    return wide[..., :t.shape[-1]]


def requests(rows, count, kind, seed=3):
    """ids: "runs" of a request's rows, "each" row another, "one" for all, "mixed" in any order with
    rows that have none, "none"."""
    gen = torch.Generator().manual_seed(seed + rows)
    if kind == "none":
        ids = torch.full((rows,), -1)
    elif kind == "one":
        ids = torch.full((rows,), count - 1)
    elif kind == "each":
        ids = torch.arange(rows) % count
    elif kind == "runs":
        ids = torch.sort(torch.randint(-1, count, (rows,), generator=gen))[0].flip(0)
    else:
        ids = torch.randint(-3, count + 3, (rows,), generator=gen)
        ids[::17] = 2 ** 31 - 1
    return ids.int().cuda()


def check(dtype, rows, k, n, rank, count=5, kind="mixed", *, transb=True, act="none", bias=False, residual=False,
          scales=True, out=None, pad=0, seed=1):
    odt = DTYPES[out or dtype]
    x = padded(rand(rows, k, dtype=dtype, seed=seed), pad)
    w = padded(rand(*((n, k) if transb else (k, n)), dtype=dtype, seed=seed + 1, scale=max(k, 1) ** -0.5), pad)
    a = padded(rand(count, rank, k, dtype=dtype, seed=seed + 2, scale=max(k, 1) ** -0.5), pad)
    b = padded(rand(count, n, rank, dtype=dtype, seed=seed + 3, scale=max(rank, 1) ** -0.5), pad)
    f = (torch.rand(count, generator=torch.Generator().manual_seed(seed)) + 0.5).cuda() if scales else None
    v = rand(n, dtype=dtype, seed=seed + 4) if bias else None
    r = padded(rand(rows, n, dtype=out or dtype, seed=seed + 5), pad) if residual else None
    ids = requests(rows, count, kind)
    wide = torch.full((rows, n + pad), 7.0, dtype=odt, device="cuda")
    y = wide[:, :n]
    got = dg.adapter_linear(x, w, a, b, ids, f, v, act, r, transb=transb, out=y)
    assert got is y
    torch.cuda.synchronize()
    want, bound = ref.adapter_linear(x, w, a, b, ids, f, v, act, r, transb, odt)
    worst = ref.worst(y, want, bound)
    assert worst <= 1.0, "error %.3g of its bound" % worst
    assert bool((wide[:, n:] == 7.0).all())
    return y


@pytest.mark.gpu
@pytest.mark.parametrize("transb", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows", [1, 2, 15, 16, 17, 48, 63, 65, 130, 300, 700])
def test_rows(cuda, dtype, transb, rows):
    for kind in ("runs", "each", "mixed"):
        check(dtype, rows, 200, 264, 16, kind=kind, transb=transb, residual=True)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rank", [1, 3, 7, 8, 15, 17, 31, 33, 40, 64, 65, 128, 200])
def test_ranks(cuda, dtype, rank):
    for rows in (1, 20, 150):
        check(dtype, rows, 136, 96, rank, kind="mixed")
        check(dtype, rows, 133, 99, rank, kind="runs", transb=False)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows", [1, 17, 64, 65, 300, 1000])
def test_parts_of_the_summed_axis(cuda, dtype, rows):
    """Long rows, whose first product is cut into parts: added up by the second's blocks for
    a few rows, joined before it for more."""
    for k, n, rank, kind in ((1100, 136, 5, "mixed"), (4099, 72, 16, "each"), (4096, 264, 72, "runs"), (2048, 40, 33, "mixed")):
        check(dtype, rows, k, n, rank, kind=kind, transb=rank != 16, residual=True)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_parts_through_every_kernel(cuda, dtype):
    """The same where the entry is forced: small tiles and few rows add up parts, large tiles do not."""
    code = dg.GEMM_DTYPE_F32 if dtype == "f32" else dg.GEMM_DTYPE_BF16
    try:
        for cfg in range(dg.gemm_linear_num_configs(code)):
            forms = dg.gemm_linear_config_forms(code, cfg)
            for split in (1, 3):
                for transb in (False, True):
                    if forms >> transb & 1:
                        log(dg.gemm_linear_config_name(code, cfg), split, transb)
                        assert dg.gemm_linear_force_config(cfg, split) == 0
                        check(dtype, 50, 2048, 136, 40, kind="mixed", transb=transb)
    finally:
        dg.gemm_linear_force_config()


@pytest.mark.gpu
@pytest.mark.parametrize("transb", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("width", [(1, 1), (3, 5), (7, 40), (8, 16), (9, 33), (65, 1), (67, 130), (515, 257), (2055, 72),
                                   (4100, 40)], ids=str)
def test_widths(cuda, dtype, transb, width):
    k, n = width
    for rows in (3, 40):
        check(dtype, rows, k, n, 8, transb=transb, bias=True, act="gelu")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_every_kernel(cuda, dtype):
    """Every entry of the linear layers' table, whole and in slices, aligned rows and odd ones."""
    code = dg.GEMM_DTYPE_F32 if dtype == "f32" else dg.GEMM_DTYPE_BF16
    try:
        for cfg in range(dg.gemm_linear_num_configs(code)):
            forms = dg.gemm_linear_config_forms(code, cfg)
            for split in (1, 3):
                for n, k in [(520, 384), (263, 331)]:
                    for transb in (False, True):
                        if forms >> transb & 1:
                            log(dg.gemm_linear_config_name(code, cfg), split, n, k, transb)
                            assert dg.gemm_linear_force_config(cfg, split) == 0
                            check(dtype, 515, k, n, 24, kind="runs", transb=transb, act="silu", residual=True)
                            check(dtype, 290, k, n, 40, kind="mixed", transb=transb)
    finally:
        dg.gemm_linear_force_config()


# Tiles of 256 x 256 on 256 compute units: whole ones, halves and quarters (as in the layers' own test).
@pytest.mark.gpu
@pytest.mark.parametrize("size", [(3300, 2800, 72), (2100, 2060, 200), (700, 600, 192)], ids=str)
def test_whole_tiles_halves_and_quarters(cuda, size):
    rows, n, k = size
    try:
        assert dg.gemm_linear_force_config(0, 1) == 0
        for transb in (False, True):
            check("bf16", rows, k, n, 20, kind="runs", transb=transb, act="silu", residual=True)
    finally:
        dg.gemm_linear_force_config()


@pytest.mark.gpu
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_epilogues(cuda, dtype, act, out):
    for rows in (9, 140):
        check(dtype, rows, 96, 200, 16, act=act, bias=True, residual=True, scales=False, out=out)


@pytest.mark.gpu
@pytest.mark.parametrize("pad", [1, 2, 4, 8])
@pytest.mark.parametrize("transb", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_pitches(cuda, dtype, transb, pad):
    check(dtype, 150, 192, 256, 24, transb=transb, pad=pad, residual=True)
    check(dtype, 7, 131, 67, 9, transb=transb, pad=pad)


@pytest.mark.gpu
@pytest.mark.parametrize("count", [1, 2, 70, 300])
def test_many_adapters(cuda, count):
    for rows in (1, 64, 200):
        for kind in ("each", "mixed", "one"):
            check("bf16", rows, 128, 80, 16, count, kind)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_without_an_adapter_are_the_layers(cuda, dtype):
    """Bit for bit, whatever the adapters hold; and without adapters at all."""
    for rows in (5, 200):
        x, w = rand(rows, 256, dtype=dtype, seed=1), rand(128, 256, dtype=dtype, seed=2)
        a, b = torch.full((3, 16, 256), math.nan, dtype=x.dtype, device="cuda"), rand(3, 128, 16, dtype=dtype, seed=3)
        want = dg.linear(x, w, transb=True, act="silu")
        got = dg.adapter_linear(x, w, a, b, requests(rows, 3, "none"), act="silu", transb=True)
        assert torch.equal(got, want)
        ids = requests(rows, 3, "none")
        ids[2] = 1
        got = dg.adapter_linear(x, w, a, b, ids, act="silu", transb=True)
        keep = [i for i in range(rows) if i != 2]
        assert torch.equal(got[keep], want[keep]) and torch.isnan(got[2]).all()
        for a0, b0 in ((a[:0], b[:0]), (a[:, :0], b[:, :, :0])):
            assert torch.equal(dg.adapter_linear(x, w, a0, b0, ids, act="silu", transb=True), want)


@pytest.mark.gpu
def test_other_adapters_are_not_read(cuda):
    x, w = rand(30, 256, dtype="bf16", seed=1), rand(128, 256, dtype="bf16", seed=2)
    a, b = rand(6, 16, 256, dtype="bf16", seed=3), rand(6, 128, 16, dtype="bf16", seed=4)
    ids = torch.tensor([1, 1, 4, 4, 4, -1] * 5, dtype=torch.int32, device="cuda")
    want = dg.adapter_linear(x, w, a, b, ids, transb=True)
    for e in (0, 2, 3, 5):
        a[e], b[e] = math.nan, math.nan
    assert torch.equal(dg.adapter_linear(x, w, a, b, ids, transb=True), want)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_broken_adapters_keep_to_their_rows(cuda, dtype):
    """NaN and infinities of one request's adapter reach no row of another's, nor rows without
    one, in any kernel: those are what they are with a whole adapter, bit for bit."""
    code = dg.GEMM_DTYPE_F32 if dtype == "f32" else dg.GEMM_DTYPE_BF16
    k, n, rank = 200, 264, 24
    for rows in (14, 290):
        x, w = rand(rows, k, dtype=dtype, seed=1), rand(n, k, dtype=dtype, seed=2)
        a, b = rand(5, rank, k, dtype=dtype, seed=3), rand(5, n, rank, dtype=dtype, seed=4)
        ids = requests(rows, 5, "mixed")
        own = ids == 2
        assert own.any() and not own.all()
        broken_b, broken_a = b.clone(), a.clone()
        broken_b[2, ::3], broken_b[2, 1::3, 5] = math.nan, math.inf
        broken_a[2, 3], broken_a[2, 4] = math.nan, math.inf
        try:
            for cfg in range(-1, dg.gemm_linear_num_configs(code)):
                for split in (1, 3):
                    for transb in (False, True):
                        if cfg >= 0 and not dg.gemm_linear_config_forms(code, cfg) >> transb & 1:
                            continue
                        assert dg.gemm_linear_force_config(cfg, split if cfg >= 0 else 0) == 0
                        args = (x, w if transb else w.T.contiguous())
                        want = dg.adapter_linear(*args, a, b, ids, transb=transb)
                        got = dg.adapter_linear(*args, broken_a, broken_b, ids, transb=transb)
                        what = "%d rows, entry %d, %d slices, transb %s" % (rows, cfg, split, transb)
                        assert torch.equal(got[~own], want[~own]), what
                        assert torch.isnan(got[own]).all(), what
                        # b alone: those of its columns that are broken
                        got = dg.adapter_linear(*args, a, broken_b, ids, transb=transb)
                        assert torch.equal(got[~own], want[~own]) and torch.equal(got[own][:, 2::3], want[own][:, 2::3]), what
                        assert not (got[own][:, ::3].isfinite().any() or got[own][:, 1::3].isfinite().any()), what
        finally:
            dg.gemm_linear_force_config()


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [4, 300])
def test_in_place_of_the_residual(cuda, rows):
    x, w = rand(rows, 256, dtype="bf16", seed=1), rand(128, 256, dtype="bf16", seed=2)
    a, b = rand(4, 16, 256, dtype="bf16", seed=3), rand(4, 128, 16, dtype="bf16", seed=4)
    res, ids = rand(rows, 128, dtype="bf16", seed=5), requests(rows, 4, "mixed")
    want = dg.adapter_linear(x, w, a, b, ids, residual=res, transb=True, out_dtype=torch.bfloat16)
    got = dg.adapter_linear(x, w, a, b, ids, residual=res, transb=True, out=res)
    assert got is res and torch.equal(got, want)


@pytest.mark.gpu
def test_adapters_far_apart(cuda):
    """Offsets beyond 32 bits."""
    x, w = rand(20, 64, dtype="bf16", seed=1), rand(40, 64, dtype="bf16", seed=2)
    a, b = rand(3, 16, 64, dtype="bf16", seed=3), rand(3, 40, 16, dtype="bf16", seed=4)
    ids = requests(20, 3, "mixed")
    want = dg.adapter_linear(x, w, a, b, ids, transb=True)
    stride = (1 << 31) + 8
    far = torch.empty(2 * stride + 4096, dtype=torch.bfloat16, device="cuda")
    a2 = far.as_strided(a.shape, (stride, 64, 1))
    b2 = far.as_strided(b.shape, (stride, 16, 1), 2048)
    a2.copy_(a), b2.copy_(b)
    assert torch.equal(dg.adapter_linear(x, w, a2, b2, ids, transb=True), want)


@pytest.mark.gpu
def test_streams_and_graphs(cuda):
    x, w = rand(40, 512, dtype="bf16", seed=1), rand(256, 512, dtype="bf16", seed=2)
    a, b = rand(8, 16, 512, dtype="bf16", seed=3), rand(8, 256, 16, dtype="bf16", seed=4)
    sets = [requests(40, 8, "mixed"), requests(40, 8, "runs")]
    run = lambda i, **kw: dg.adapter_linear(x, w, a, b, sets[i], transb=True, **kw)  # noqa: E731
    want = [run(0), run(1)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = run(0, stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(got, want[0])
    ids = sets[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = dg.adapter_linear(x, w, a, b, ids, transb=True)
    for k in range(4):
        ids.copy_(sets[k % 2])
        graph.replay()
        eager = run(1)
        torch.cuda.synchronize()
        assert torch.equal(out, want[k % 2]) and torch.equal(eager, want[1])


@pytest.mark.gpu
def test_two_streams_at_once(cuda):
    """Calls on two streams at a time, of rows whose parts are joined and of few rows."""
    jobs = []
    for rows, seed in ((300, 1), (20, 7)):
        jobs.append((rand(rows, 2048, dtype="bf16", seed=seed), rand(256, 2048, dtype="bf16", seed=seed + 1),
                     rand(4, 16, 2048, dtype="bf16", seed=seed + 2), rand(4, 256, 16, dtype="bf16", seed=seed + 3),
                     requests(rows, 4, "mixed")))
    want = [dg.adapter_linear(*j, transb=True) for j in jobs]
    streams = [torch.cuda.Stream() for _ in jobs]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        got = [dg.adapter_linear(*j, transb=True, stream=s.cuda_stream) for j, s in zip(jobs, streams)]
        for s in streams:
            s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [1, 20])
def test_a_decoding_step(cuda, rows):
    """A projection with adapters, a mixture-of-experts layer behind its router, and the
    next token's log probabilities, against the same in 64 bits (each operator on the
    others' outputs), eagerly and from a graph."""
    hidden, inner, experts, top, vocab = 128, 96, 8, 2, 1000
    x, w = rand(rows, hidden, dtype="bf16", seed=1), rand(hidden, hidden, dtype="bf16", seed=2, scale=hidden ** -0.5)
    a, b = rand(3, 8, hidden, dtype="bf16", seed=3, scale=hidden ** -0.5), rand(3, hidden, 8, dtype="bf16", seed=4)
    router = rand(hidden, experts, dtype="bf16", seed=5, scale=0.3)
    up = rand(experts, 2 * inner, hidden, dtype="bf16", seed=6, scale=hidden ** -0.5)
    down = rand(experts, hidden, inner, dtype="bf16", seed=7, scale=inner ** -0.5)
    head = rand(vocab, hidden, dtype="bf16", seed=8, scale=hidden ** -0.5)
    ids = requests(rows, 3, "runs")
    tokens = torch.arange(rows, dtype=torch.int32, device="cuda") * 40

    def step():
        h = dg.adapter_linear(x, w, a, b, ids, residual=x, transb=True, out_dtype=torch.bfloat16)
        routed = dg.log_probs(dg.linear(h, router), top=top)
        shares = torch.softmax(routed.top_logprobs, dim=1)
        y = dg.moe_layer(h, up, down, routed.top_ids, shares, residual=h, transb=True, out_dtype=torch.bfloat16)
        logits = dg.linear(y, head, transb=True)
        return h, routed.top_ids, shares, y, logits, dg.log_probs(logits, tokens, 5)

    h, chosen, shares, y, logits, answer = step()
    torch.cuda.synchronize()
    assert ref.worst(h, *ref.adapter_linear(x, w, a, b, ids, None, None, "none", x, True, torch.bfloat16)) <= 1.0
    assert torch.equal(chosen, (h.double() @ router.double()).topk(top, dim=1)[1].int())
    assert ref.worst(y, *ref.moe_layer(h, up, down, chosen, shares, "silu", h, True, True, torch.bfloat16)) <= 1.0
    want = ref.log_probs(logits, tokens, 5, 1.0)
    assert ref.worst(answer.logprob[:, None], *want["logprob"]) <= 1.0
    assert torch.equal(answer.top_ids.cpu().long(), want["top_ids"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        replayed = step()
    for _ in range(3):
        graph.replay()
        again = step()
        torch.cuda.synchronize()
        for got in (replayed, again):
            assert torch.equal(got[3], y) and torch.equal(got[4], logits)
            assert all(torch.equal(p, q) for p, q in zip(got[5], answer))


@pytest.mark.gpu
def test_helper_checks(cuda):
    x, w = rand(4, 64, dtype="bf16", seed=1), rand(48, 64, dtype="bf16", seed=2)
    a, b = rand(3, 16, 64, dtype="bf16", seed=3), rand(3, 48, 16, dtype="bf16", seed=4)
    ids, ok = requests(4, 3, "mixed"), dict(transb=True)
    f = torch.ones(3, device="cuda")
    for bad in (lambda: dg.adapter_linear(x, w, a, b, ids.long(), **ok), lambda: dg.adapter_linear(x, w, a.float(), b, ids, **ok),
                lambda: dg.adapter_linear(x, w, a, b, ids, f.half(), **ok), lambda: dg.adapter_linear(x.half(), w, a, b, ids, **ok)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: dg.adapter_linear(x, w, a, b, ids[:3], **ok), lambda: dg.adapter_linear(x, w, a[:2], b, ids, **ok),
                lambda: dg.adapter_linear(x, w, a, b[:, :, :8], ids, **ok), lambda: dg.adapter_linear(x, w, a, b, ids),
                lambda: dg.adapter_linear(x, w, a, b, ids, f[:2], **ok), lambda: dg.adapter_linear(x, w, a, b, ids.cpu(), **ok),
                lambda: dg.adapter_linear(x, w, a[:, :, ::2], b, ids, **ok),
                lambda: dg.adapter_linear(x, w, a, b, ids, bias=torch.zeros(47, device="cuda"), **ok),
                lambda: dg.adapter_linear(x, w, a, b, ids, out=torch.empty(4, 47, device="cuda"), **ok)):
        with pytest.raises(ValueError):
            bad()
