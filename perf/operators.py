"""Timed cases of the linear-layer operators: the dense product with bias,
activation and residual (``linear``), its backward pass (``linear_grad``), and
both for products grouped by expert with ragged row counts
(``grouped_linear``, ``grouped_linear_grad``).

With ``own`` false the operators are computed in elementary torch operations in
float32; with ``own`` true by this repository's kernels.

    z = x . w + bias          y = act(z) + residual
    dz = dy * act'(z)         dx = dz . w^T    dw = x^T . dz    dbias = sum of dz over rows

For grouped operators row r of group g (offsets[g] <= r < offsets[g + 1]) uses
w[g] and bias[g], and dw[g], dbias[g] sum over that group's rows.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------- cases --

def listed():
    # op, rows (M or all groups' rows), k, n; transb: weights stored n x k
    base = {"dtype": "bf16", "transb": True, "act": "silu", "bias": True, "residual": False,
            "pre": False, "groups": 0, "skew": 0.0, "spare": 0}
    case = lambda name, op, rows, k, n, **kw: dict(base, name=name, op=op, rows=rows, k=k, n=n, **kw)  # noqa: E731
    return [
        # one token through a projection: latency, and reading the weights once
        case("linear 1 token", "linear", 1, 4096, 4096),
        # a decoding batch through the second product of a feed-forward layer, with its residual
        case("linear 48 tokens", "linear", 48, 8192, 4096, act="none", residual=True),
        # first product of a feed-forward layer in training: the pre-activation is kept
        case("linear training", "linear", 4096, 4096, 16384, act="gelu_tanh", transb=False, pre=True),
        # full precision, no size a multiple of anything
        case("linear odd f32", "linear", 1000, 1001, 2047, dtype="f32", act="gelu", residual=True),
        # backward pass of a training step's layer
        case("grad training", "linear_grad", 4096, 4096, 8192, act="gelu_tanh", transb=False),
        # full precision backward, odd sizes
        case("grad odd f32", "linear_grad", 777, 1000, 1025, dtype="f32", act="silu"),
        # one token sent to two of 16 experts
        case("grouped 2 rows", "grouped", 2, 2048, 4096, groups=16),
        # a decoding batch over 32 experts, some of them empty
        case("grouped 64 rows", "grouped", 64, 4096, 2048, groups=32, act="none", bias=False, skew=0.7),
        # prefill or training over 16 experts, uneven, with rows behind the last group
        case("grouped prefill", "grouped", 8192, 4096, 4096, groups=16, transb=False, skew=0.5, spare=100),
        # full precision, odd sizes, few experts
        case("grouped odd f32", "grouped", 1111, 515, 1030, dtype="f32", groups=7, act="gelu", transb=False),
        # backward pass of the experts in a training step
        case("grouped grad training", "grouped_grad", 8192, 2048, 4096, groups=16, act="silu", skew=0.5),
        # full precision, odd sizes
        case("grouped grad odd f32", "grouped_grad", 500, 300, 261, dtype="f32", groups=5, act="gelu_tanh",
             transb=False),
    ]


def _cost(c):
    """(flops, weights and activations) of the case: what draw() keeps within the listed ones."""
    products = 2 if c["op"].endswith("grad") else 1
    rows = c["rows"] * (1 + 2 * c["skew"])
    return (2.0 * rows * c["k"] * c["n"] * products,
            max(1, c["groups"]) * c["k"] * c["n"] + rows * (c["k"] + c["n"]))


def draw(rng):
    log = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))  # noqa: E731
    while True:
        op = rng.choice(["linear", "linear_grad", "grouped", "grouped_grad"])
        dtype = rng.choice(["bf16", "bf16", "f32"])
        grouped = op.startswith("grouped")
        k, n = log(64, 8192), log(64, 16384)
        if rng.random() < 0.7:  # most layers' widths are multiples of 64; the others stay odd
            k, n = max(64, k // 64 * 64), max(64, n // 64 * 64)
        c = {"op": op, "rows": log(1, 8192), "k": k, "n": n, "dtype": dtype,
             "transb": rng.random() < 0.5, "act": rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]),
             "bias": rng.random() < 0.7, "residual": not op.endswith("grad") and rng.random() < 0.3,
             "pre": op == "linear" and rng.random() < 0.3,
             "groups": log(2, 64) if grouped else 0,
             "skew": round(rng.uniform(0.0, 0.8), 2) if grouped else 0.0,
             "spare": rng.choice([0, 0, 1, 37]) if op == "grouped" else 0}
        flops, elems = _cost(c)
        if flops <= 5.0e11 * (0.5 if dtype == "f32" else 1.0) and elems <= 2.0e8:
            return c


def work(case):
    c = case
    rows, k, n, grad = c["rows"], c["k"], c["n"], c["op"].endswith("grad")
    es = 2 if c["dtype"] == "bf16" else 4
    g = c["groups"]
    used = g * (1 - (1 - 1 / g) ** rows) if g else 1.0  # experts that get a row (expected)
    acts = rows * (k + n) * es                          # x, y (or dy, x)
    if not grad:
        byts = acts + used * k * n * es
        byts += used * n * es if c["bias"] else 0
        byts += rows * n * es * (int(c["residual"]) + int(c["pre"]))
    else:
        byts = acts + used * k * n * es                 # dy, x, w
        byts += rows * n * es if c["act"] != "none" else 0
        byts += rows * k * es + max(1, g) * k * n * es + max(1, g) * n * 4  # dx, dw, dbias
    return {"bytes": int(byts + (4 * (g + 1) if g else 0)),
            "flops": 2 * rows * k * n * (2 if grad else 1)}


# ------------------------------------------------------------------ inputs --

class State:
    pass


def prepare(case, seed):
    c, s = case, State()
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[c["dtype"]]
    randn = lambda *shape, scale=1.0: torch.randn(shape, generator=gen, device="cuda").mul_(scale).to(dt)  # noqa: E731
    rows, k, n, g = c["rows"], c["k"], c["n"], c["groups"]
    lead = (g,) if g else ()
    s.case, s.dt = c, dt
    total = rows + c["spare"]
    s.x = randn(total, k)
    s.w = randn(*lead, *((n, k) if c["transb"] else (k, n)), scale=k ** -0.5)
    s.bias = randn(*lead, n, scale=0.5) if c["bias"] and not c["op"].endswith("grad") else None
    s.residual = randn(total, n) if c["residual"] else None
    s.offsets = s.out = s.dx = None
    s.cap = 0
    if g:
        # rows per expert as a router leaves them: uneven, some experts empty
        rng = random.Random(seed * 1000003 + 17)
        share = [math.exp(c["skew"] * rng.gauss(0.0, 1.0)) for _ in range(g)]
        count = [0] * g
        for e in rng.choices(range(g), weights=share, k=rows):
            count[e] += 1
        off = [0]
        for m in count:
            off.append(off[-1] + m)
        s.offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
        s.cap = max(count)
    if c["op"] == "grouped":
        s.out = randn(total, n)  # rows behind the last group keep these values
    s.pre = torch.empty((rows, n), dtype=dt, device="cuda") if c["pre"] else None
    if c["op"].endswith("grad"):
        s.dy = randn(total, n)
        s.z = randn(total, n) if c["act"] != "none" else None
    return s


# -------------------------------------------------------------- plain form --

def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    if act == "gelu_tanh":
        a = math.sqrt(2 / math.pi)
        t = torch.tanh(a * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * a * (1 + 3 * 0.044715 * z * z)
    s = 1 / (1 + torch.exp(-z))
    return s * (1 + z * (1 - s))


def _padded(s):
    """For the rows of each group, up to the largest group's count: row index,
    and whether the group has that row."""
    off = s.offsets.long()
    at = off[:-1, None] + torch.arange(s.cap, device="cuda")[None, :]
    live = at < off[1:, None]
    return torch.where(live, at, torch.zeros_like(at)), live


def _plain(s):
    c, dt = s.case, s.dt
    x, w = s.x.float(), s.w.float()
    if c["transb"]:
        w = w.transpose(-1, -2).contiguous()
    if c["op"] == "linear":
        z = x @ w
        if s.bias is not None:
            z = z + s.bias.float()
        y = _act(z, c["act"])
        if s.residual is not None:
            y = y + s.residual.float()
        return {"y": y.to(dt), "pre": z.to(dt)} if c["pre"] else {"y": y.to(dt)}
    if c["op"] == "linear_grad":
        dz = s.dy.float()
        if s.z is not None:
            dz = dz * _act_slope(s.z.float(), c["act"])
        return {"dx": (dz @ w.t()).to(dt), "dw": _stored(x.t() @ dz, c).to(dt), "dbias": dz.sum(0)}
    at, live = _padded(s)
    xp = torch.where(live[:, :, None], x[at], torch.zeros((), device="cuda"))
    if c["op"] == "grouped":
        z = torch.bmm(xp, w)
        if s.bias is not None:
            z = z + s.bias.float()[:, None, :]
        y = _act(z, c["act"])[live]
        if s.residual is not None:
            y = y + s.residual[at[live]].float()
        out = s.out
        out[at[live]] = y.to(dt)
        return {"y": out}
    dz = s.dy.float()
    if s.z is not None:
        dz = dz * _act_slope(s.z.float(), c["act"])
    dzp = torch.where(live[:, :, None], dz[at], torch.zeros((), device="cuda"))
    dx = torch.empty_like(s.x)
    dx[at[live]] = torch.bmm(dzp, w.transpose(1, 2).contiguous())[live].to(dt)
    dw = torch.bmm(xp.transpose(1, 2).contiguous(), dzp)
    return {"dx": dx, "dw": _stored(dw, c).to(dt), "dbias": dzp.sum(1)}


def _stored(dw, c):
    return dw.transpose(-1, -2).contiguous() if c["transb"] else dw


# --------------------------------------------------------------------- run --

def _kernels(s):
    import dense_gemm_03_amd as dg
    c = s.case
    act = c["act"]
    if c["op"] == "linear":
        y = dg.linear(s.x, s.w, bias=s.bias, act=act, residual=s.residual, transb=c["transb"],
                      pre=s.pre, out_dtype=s.dt)
        return {"y": y, "pre": s.pre} if c["pre"] else {"y": y}
    if c["op"] == "grouped":
        return {"y": dg.grouped_linear(s.x, s.w, s.offsets, bias=s.bias, act=act, residual=s.residual,
                                       transb=c["transb"], out=s.out)}
    if c["op"] == "linear_grad":
        dx, dw, dbias = dg.linear_grad(s.dy, s.x, s.w, act=act, pre=s.z, transb=c["transb"], out_dtype=s.dt)
    else:
        dx, dw, dbias = dg.grouped_linear_grad(s.dy, s.x, s.w, s.offsets, act=act, pre=s.z,
                                               transb=c["transb"], out_dtype=s.dt)
    return {"dx": dx, "dw": dw, "dbias": dbias}


def run(state):
    if own:
        return _kernels(state)
    return _plain(state)


# ------------------------------------------------------------------- exact --

def _activation64(z, act):
    """(act(z), its derivative) in float64."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return z.clamp(min=0), (z > 0).double()
    if act == "silu":
        q = torch.sigmoid(z)
        return z * q, q + z * q * (1 - q)
    if act == "gelu":
        q = 0.5 * torch.erfc(-z / math.sqrt(2))
        return z * q, q + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    r = math.sqrt(8 / math.pi)                  # gelu_tanh(z) = z sigmoid(r (z + 0.044715 z^3))
    q = torch.sigmoid(r * (z + 0.044715 * z ** 3))
    return z * q, q + z * q * (1 - q) * r * (1 + 0.134145 * z ** 2)


def exact(case, seed):
    s, c = prepare(case, seed), case
    spans = [(0, c["rows"])]
    if c["groups"]:
        off = s.offsets.tolist()
        spans = list(zip(off[:-1], off[1:]))
    weight = lambda g: (s.w[g] if c["groups"] else s.w).double()  # noqa: E731
    grad = c["op"].endswith("grad")
    found = {"y": [], "pre": [], "dx": [], "dw": [], "dbias": []}
    for g, (lo, hi) in enumerate(spans):
        w = weight(g).T if c["transb"] else weight(g)
        x = s.x[lo:hi].double()
        if not grad:
            z = x @ w
            if s.bias is not None:
                z = z + (s.bias[g] if c["groups"] else s.bias).double()
            y = _activation64(z, c["act"])[0]
            if s.residual is not None:
                y = y + s.residual[lo:hi].double()
            found["y"].append(y)
            found["pre"].append(z)
        else:
            dz = s.dy[lo:hi].double()
            if s.z is not None:
                dz = dz * _activation64(s.z[lo:hi].double(), c["act"])[1]
            found["dx"].append(dz @ w.T)
            found["dw"].append(dz.T @ x if c["transb"] else x.T @ dz)
            found["dbias"].append(dz.sum(0))
    if not grad:
        y = torch.cat(found["y"])
        if c["spare"]:
            y = torch.cat([y, s.out[c["rows"]:].double()])
        return {"y": y, "pre": torch.cat(found["pre"])} if c["pre"] else {"y": y}
    if not c["groups"]:
        return {name: found[name][0] for name in ("dx", "dw", "dbias")}
    return {"dx": torch.cat(found["dx"]), "dw": torch.stack(found["dw"]), "dbias": torch.stack(found["dbias"])}
