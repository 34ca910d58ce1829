"""The mixture-of-experts layer for a few tokens against its definition in 64 bits
(serving_ref, where the bounds are derived): tokens on either side of the chunks and
row tiles, widths at the edges of strips and passes, both orientations and types,
experts named twice, by all tokens or by none, absent ids, pitches, in place, streams,
graphs, threads; and, without a GPU, what the calls refuse."""
from __future__ import annotations

import math

import pytest
import torch

import dense_gemm_03_amd as dg
from tests import serving_ref as ref

BAD = dg.GEMM_ERR_INVALID_ARG
P = 1 << 20     # stands in for a 16-byte aligned device address: refused calls read nothing
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def params(**kw):
    """A valid layer: 10 tokens of 64, 4 of 8 experts of inner width 48, gated, bf16."""
    p = dict(dtype=1, dtype_y=1, transw=0, act=dg.GEMM_ACT_SILU, gated=1, reserved=0, tokens=10, hidden=64, inner=48,
             experts=8, top=4, ldx=64, ldy=64, ldr=64, ldup=96, lddown=64, stride_up=64 * 96, stride_down=48 * 64)
    p.update(kw)
    return dg.MoeParams(**p)


def call(p, x=P, up=P, down=P, ids=P, weights=P, res=P + 4096, y=P + 4096, ws=P, n=1 << 40):
    return dg.gemm_moe_layer(p, x, up, down, ids, weights, res, y, ws, n)


BAD_PARAMS = [dict(dtype=2), dict(dtype_y=-1), dict(transw=2), dict(act=5), dict(act=-1), dict(gated=2), dict(tokens=-1),
              dict(tokens=513), dict(hidden=-1), dict(hidden=(1 << 22) + 1, ldx=1 << 30, ldy=1 << 30, ldr=1 << 30, lddown=1 << 23, stride_up=1 << 40, stride_down=1 << 40), dict(inner=-1),
              dict(inner=(1 << 22) + 1, ldup=1 << 24, stride_up=1 << 40, stride_down=1 << 40), dict(ldup=(1 << 24) + 1, stride_up=1 << 40), dict(experts=-1), dict(experts=1025), dict(top=-1), dict(top=33), dict(ldx=63),
              dict(ldy=63), dict(ldup=95), dict(lddown=63), dict(transw=1, ldup=63), dict(transw=1, ldup=64, lddown=47),
              dict(stride_up=64 * 96 - 1), dict(stride_down=48 * 64 - 1), dict(ldx=(1 << 40) + 1)]


@pytest.mark.parametrize("kw", BAD_PARAMS, ids=str)
def test_bad_parameters(kw):
    assert call(params(**kw)) == BAD
    assert dg.gemm_moe_layer_workspace_size(params(**kw)) == BAD


def test_bad_arguments():
    need = dg.gemm_moe_layer_workspace_size(params())
    assert need >= 2 * 10 * 4 * 48 * 2
    for kw in (dict(x=None), dict(up=None), dict(down=None), dict(ids=None), dict(weights=None), dict(y=None),
               dict(ws=None), dict(ws=P + 8), dict(n=need - 1), dict(x=P + 1), dict(up=P + 1), dict(down=P + 1),
               dict(ids=P + 2), dict(weights=P + 1), dict(res=P + 1), dict(y=P + 1)):
        assert call(params(), **kw) == BAD, kw
    assert call(params(ldr=63)) == BAD
    assert call(params(ldr=65)) == BAD      # in place with another pitch
    assert call(None) == BAD and dg.gemm_moe_layer_workspace_size(None) == BAD
    # more blocks than a launch holds
    wide = dict(inner=1 << 22, ldup=1 << 23, stride_up=1 << 31, stride_down=1 << 30, tokens=512, experts=1024, top=32)
    assert call(params(**wide)) == BAD and dg.gemm_moe_layer_workspace_size(params(**wide)) == BAD


def test_empty_calls_launch_nothing():
    assert call(params(tokens=0), None, None, None, None, None, None, None, None, 0) == dg.GEMM_OK
    assert call(params(hidden=0), None, None, None, None, None, None, None, None, 0) == dg.GEMM_OK


def test_helper_refuses_host_tensors():
    with pytest.raises(ValueError):
        dg.moe_layer(torch.zeros(2, 8), torch.zeros(3, 8, 12), torch.zeros(3, 6, 8), torch.zeros(2, 1).int(),
                     torch.zeros(2, 1))


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


def routed(tokens, experts, top, seed, absent=0.0):
    gen = torch.Generator().manual_seed(seed)
    ids = torch.rand(tokens, max(experts, top), generator=gen).topk(top, dim=1)[1] if top else torch.zeros(tokens, 0)
    if absent:
        ids = torch.where(torch.rand(tokens, top, generator=gen) < absent, torch.tensor([-1, experts + 5])[
            torch.randint(0, 2, (tokens, top), generator=gen)], ids)
    return ids.int().cuda(), torch.rand(tokens, top, generator=gen).cuda()


def layer(dtype, experts, hidden, inner, gated, transb, seed=1, pad=0):
    n = 2 * inner if gated else inner
    up = rand(experts, *((n, hidden) if transb else (hidden, n)), dtype=dtype, seed=seed, scale=max(hidden, 1) ** -0.5)
    down = rand(experts, *((hidden, inner) if transb else (inner, hidden)), dtype=dtype, seed=seed + 1,
                scale=max(inner, 1) ** -0.5)
    return padded(up, pad), padded(down, pad)


def check(dtype, tokens, hidden, inner, experts, top, *, gated=True, transb=True, act="silu", residual=False, out=None,
          pad=0, ids=None, weights=None, absent=0.0, seed=1):
    odt = DTYPES[out or dtype]
    x = padded(rand(tokens, hidden, dtype=dtype, seed=seed), pad)
    up, down = layer(dtype, experts, hidden, inner, gated, transb, seed + 1, pad)
    if ids is None:
        ids, weights = routed(tokens, experts, top, seed + 5, absent)
    res = padded(rand(tokens, hidden, dtype=out or dtype, seed=seed + 3), pad) if residual else None
    wide = torch.full((tokens, hidden + pad), 7.0, dtype=odt, device="cuda")
    y = wide[:, :hidden]
    got = dg.moe_layer(x, up, down, ids, weights, act=act, residual=res, gated=gated, transb=transb, out=y)
    assert got is y
    torch.cuda.synchronize()
    want, bound = ref.moe_layer(x, up, down, ids, weights, act, res, gated, transb, odt)
    r = ref.worst(y, want, bound)
    assert r <= 1.0, "error %.3g of its bound" % r
    assert bool((wide[:, hidden:] == 7.0).all())
    return y


TOKENS = [1, 2, 15, 16, 17, 31, 33, 48, 64, 65, 130]


@pytest.mark.gpu
@pytest.mark.parametrize("transb", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("tokens", TOKENS)
def test_tokens(cuda, dtype, transb, tokens):
    check(dtype, tokens, 192, 160, 8, 3, transb=transb, residual=True)
    # all tokens to the same two experts: full row tiles
    ids = torch.tensor([[1, 3]], dtype=torch.int32, device="cuda").repeat(tokens, 1)
    check(dtype, tokens, 100, 72, 5, 2, transb=transb, ids=ids, weights=torch.rand(tokens, 2, device="cuda"))


@pytest.mark.gpu
@pytest.mark.parametrize("transb", [False, True])
@pytest.mark.parametrize("tokens", [300, 512])
def test_most_tokens(cuda, transb, tokens):
    """Experts with more rows than a block takes at a time, and the most ids there can be."""
    check("bf16", tokens, 72, 56, 8, 3, transb=transb, residual=True, absent=0.1)
    ids = torch.tensor([[1, 3]], dtype=torch.int32, device="cuda").repeat(tokens, 1)
    ids[5] = -1
    check("f32", tokens, 40, 72, 5, 2, transb=transb, ids=ids, weights=torch.rand(tokens, 2, device="cuda"))
    check("bf16", tokens, 40, 24, 1024, 32, transb=transb)


WIDTHS = [(1, 1), (2, 3), (1, 40), (7, 5), (15, 17), (16, 16), (33, 31), (64, 130), (129, 64), (257, 255), (515, 33),
          (40, 1030), (2048, 96)]


@pytest.mark.gpu
@pytest.mark.parametrize("transb", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("width", WIDTHS, ids=str)
def test_widths(cuda, dtype, transb, width):
    hidden, inner = width
    for gated in (False, True):
        for tokens in (3, 20, 40):
            check(dtype, tokens, hidden, inner, 4, 2, transb=transb, gated=gated, act="gelu", absent=0.2)


@pytest.mark.gpu
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_activations(cuda, dtype, act, out):
    for gated in (False, True):
        check(dtype, 12, 96, 80, 6, 2, act=act, gated=gated, out=out, residual=gated)


@pytest.mark.gpu
@pytest.mark.parametrize("pad", [1, 2, 4, 8])
@pytest.mark.parametrize("transb", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_pitches(cuda, dtype, transb, pad):
    check(dtype, 18, 136, 72, 5, 3, transb=transb, pad=pad, residual=True)
    check(dtype, 5, 131, 67, 5, 3, transb=transb, pad=pad)


@pytest.mark.gpu
@pytest.mark.parametrize("experts,top", [(1, 1), (2, 2), (33, 8), (64, 8), (100, 1), (1024, 32), (40, 32)])
def test_many_experts(cuda, experts, top):
    for tokens in (1, 16, 40, 100):
        check("bf16", tokens, 48, 40, experts, top)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("tokens", [1, 9, 30, 70])
def test_ids_as_they_come(cuda, dtype, tokens):
    """The same expert twice or always, ids out of range only, for some tokens or all."""
    gen = torch.Generator().manual_seed(tokens)
    w = torch.randn(tokens, 4, generator=gen).cuda()
    for ids in (torch.full((tokens, 4), 2), torch.randint(0, 3, (tokens, 4), generator=gen),
                torch.randint(-2, 5, (tokens, 4), generator=gen), torch.full((tokens, 4), -1),
                torch.full((tokens, 4), 2 ** 31 - 1), torch.full((tokens, 4), -2 ** 31)):
        for residual in (False, True):
            check(dtype, tokens, 72, 56, 3, 4, ids=ids.int().cuda(), weights=w, residual=residual)
    # the weight of an absent id is not used
    ids = torch.randint(0, 3, (tokens, 4), generator=gen).int()
    ids[:, 1] = -1
    bad = w.clone()
    bad[:, 1] = math.nan
    good = w.clone()
    good[:, 1] = 0.0
    a = check(dtype, tokens, 72, 56, 3, 4, ids=ids.cuda(), weights=good)
    up, down = layer(dtype, 3, 72, 56, True, True, 2)
    b = dg.moe_layer(rand(tokens, 72, dtype=dtype, seed=1), up, down, ids.cuda(), bad, transb=True, out_dtype=DTYPES[dtype])
    assert torch.equal(a, b)


@pytest.mark.gpu
def test_unused_experts_are_not_read(cuda):
    """NaN in the weights of experts that no token names, and in no token's rows."""
    for transb in (False, True):
        up, down = layer("bf16", 6, 64, 48, True, transb)
        ids, w = torch.tensor([[1, 4], [4, 4], [1, -1]], dtype=torch.int32, device="cuda"), torch.rand(3, 2, device="cuda")
        x = rand(3, 64, dtype="bf16", seed=3)
        want = dg.moe_layer(x, up, down, ids, w, transb=transb)
        for e in (0, 2, 3, 5):
            up[e], down[e] = math.nan, math.nan
        assert torch.equal(dg.moe_layer(x, up, down, ids, w, transb=transb), want)


@pytest.mark.gpu
def test_nothing_to_do(cuda):
    x, res = rand(4, 64, dtype="bf16", seed=1), rand(4, 64, dtype="bf16", seed=2)
    up, down = layer("bf16", 3, 64, 48, True, True)
    none_i = torch.empty(4, 0, dtype=torch.int32, device="cuda")
    none_w = torch.empty(4, 0, device="cuda")
    kw = dict(transb=True, out_dtype=torch.bfloat16)
    assert bool((dg.moe_layer(x, up, down, none_i, none_w, **kw) == 0).all())
    assert torch.equal(dg.moe_layer(x, up, down, none_i, none_w, residual=res, **kw), res)
    ids, w = routed(4, 3, 2, 1)
    assert dg.moe_layer(x[:0], up, down, ids[:0], w[:0], **kw).shape == (0, 64)
    thin = dg.moe_layer(x, up[:, :0], down[:, :, :0], ids, w, residual=res, **kw)       # inner width 0
    assert torch.equal(thin, res)
    assert dg.moe_layer(x[:, :0], up[:, :, :0], down[:, :0], ids, w, **kw).shape == (4, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("tokens", [1, 40])
def test_in_place_of_the_residual(cuda, dtype, tokens):
    x, res = rand(tokens, 200, dtype=dtype, seed=1), rand(tokens, 200, dtype=dtype, seed=2)
    up, down = layer(dtype, 4, 200, 120, True, True)
    ids, w = routed(tokens, 4, 2, 3)
    want = dg.moe_layer(x, up, down, ids, w, residual=res, transb=True, out_dtype=DTYPES[dtype])
    got = dg.moe_layer(x, up, down, ids, w, residual=res, transb=True, out=res)
    assert got is res and torch.equal(got, want)


@pytest.mark.gpu
def test_large_values_and_nan(cuda):
    """An infinite or NaN token spoils its own rows only."""
    up, down = layer("bf16", 4, 64, 48, False, True)
    ids, w = routed(20, 4, 2, 3)
    x = rand(20, 64, dtype="bf16", seed=1)
    want = dg.moe_layer(x, up, down, ids, w, act="relu", gated=False, transb=True)
    y = x.clone()
    y[3], y[17, 5] = math.inf, math.nan
    got = dg.moe_layer(y, up, down, ids, w, act="relu", gated=False, transb=True)
    keep = [i for i in range(20) if i not in (3, 17)]
    assert torch.equal(got[keep], want[keep]) and not torch.isfinite(got[3]).all() and torch.isnan(got[17]).any()


@pytest.mark.gpu
def test_streams_graphs_and_threads(cuda):
    import threading
    x = rand(24, 256, dtype="bf16", seed=1)
    up, down = layer("bf16", 16, 256, 192, True, True)
    sets = [routed(24, 16, 4, s) for s in (1, 2)]
    run = lambda i: dg.moe_layer(x, up, down, *sets[i], transb=True, out_dtype=torch.bfloat16)  # noqa: E731
    want = [run(i) for i in range(2)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = dg.moe_layer(x, up, down, *sets[0], transb=True, out_dtype=torch.bfloat16, stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(got, want[0])
    # the experts of a captured call are those of the replay
    ids, w = sets[0][0].clone(), sets[0][1].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = dg.moe_layer(x, up, down, ids, w, transb=True, out_dtype=torch.bfloat16)
    for k in range(4):
        ids.copy_(sets[k % 2][0]), w.copy_(sets[k % 2][1])
        graph.replay()
        eager = run(0)
        torch.cuda.synchronize()
        assert torch.equal(out, want[k % 2]) and torch.equal(eager, want[0])
    wrong = []

    def work(i):
        stream = torch.cuda.Stream()
        try:
            with torch.cuda.stream(stream):
                for _ in range(30):
                    y = run(i)
                    stream.synchronize()
                    if not torch.equal(y, want[i]):
                        wrong.append(i)
        except Exception as e:   # a failed call of a thread is the test's failure
            wrong.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong


@pytest.mark.gpu
def test_weights_far_apart(cuda):
    """Offsets beyond 32 bits between experts."""
    for transb in (False, True):
        up, down = layer("bf16", 3, 64, 32, True, transb)
        stride = (1 << 31) + 8
        far = torch.empty(2 * stride + 64 * 64, dtype=torch.bfloat16, device="cuda")
        up2 = far.as_strided(up.shape, (stride, up.shape[2], 1))
        up2.copy_(up)
        ids, w = routed(10, 3, 2, 3)
        x = rand(10, 64, dtype="bf16", seed=1)
        want = dg.moe_layer(x, up, down, ids, w, transb=transb)
        assert torch.equal(dg.moe_layer(x, up2, down, ids, w, transb=transb), want)
        del far, up2


@pytest.mark.gpu
def test_router_and_layer(cuda):
    """log_probs of a router's logits, then the layer, against 64 bits."""
    tokens, hidden, inner, experts, top = 20, 128, 96, 16, 4
    x = rand(tokens, hidden, dtype="bf16", seed=1)
    router = rand(hidden, experts, dtype="bf16", seed=2, scale=0.3)
    up, down = layer("bf16", experts, hidden, inner, True, True)
    routed_to = dg.log_probs(dg.linear(x, router), top=top)
    weights = torch.softmax(routed_to.top_logprobs, dim=1)
    y = dg.moe_layer(x, up, down, routed_to.top_ids, weights, residual=x, transb=True, out_dtype=torch.bfloat16)
    logits = x.double() @ router.double()
    best, ids = logits.topk(top, dim=1)
    assert torch.equal(ids.int(), routed_to.top_ids)
    share = torch.softmax(best, dim=1)
    # weights within 2^-20 of the exact ones: logits are sums of 128 terms in fp32
    assert float((share - weights).abs().max()) < 2.0 ** -18
    want, bound = ref.moe_layer(x, up, down, ids, weights, "silu", x, True, True, torch.bfloat16)
    assert ref.worst(y, want, bound) <= 1.0


@pytest.mark.gpu
def test_helper_checks(cuda):
    x = rand(4, 64, dtype="bf16", seed=1)
    up, down = layer("bf16", 3, 64, 48, True, True)
    ids, w = routed(4, 3, 2, 1)
    ok = dict(transb=True)
    for bad in (lambda: dg.moe_layer(x, up, down, ids.long(), w, **ok), lambda: dg.moe_layer(x, up.float(), down, ids, w, **ok),
                lambda: dg.moe_layer(x, up, down, ids, w.half(), **ok), lambda: dg.moe_layer(x.half(), up, down, ids, w, **ok)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: dg.moe_layer(x, up, down, ids[:3], w, **ok), lambda: dg.moe_layer(x, up, down, ids, w[:, :1], **ok),
                lambda: dg.moe_layer(x, up, down[:2], ids, w, **ok), lambda: dg.moe_layer(x, up, down, ids, w),
                lambda: dg.moe_layer(x, up, down, ids, w, gated=False, **ok),
                lambda: dg.moe_layer(x, up, down, ids.cpu(), w, **ok), lambda: dg.moe_layer(x[:, ::2], up, down, ids, w, **ok),
                lambda: dg.moe_layer(x, up, down, ids, w, act="tanh", **ok),
                lambda: dg.moe_layer(x, up, down, ids, w, out=torch.empty(4, 63, device="cuda"), **ok)):
        with pytest.raises(ValueError):
            bad()
    many = rand(513, 64, dtype="bf16", seed=1)
    ids, w = routed(513, 3, 2, 1)
    with pytest.raises(dg.GemmError):
        dg.moe_layer(many, up, down, ids, w, **ok)
