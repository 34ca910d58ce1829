"""Timed cases of the operators around a model's products when it answers: the
whole mixture-of-experts layer for a few tokens (``moe_layer``), the linear layer
with a low-rank adapter per row (``adapter_linear``), and the log probabilities of
given tokens with entropy and top alternatives (``log_probs``) with their gradient
(``log_probs_grad``).

With ``own`` false the operators are computed in elementary torch operations in
float32; with ``own`` true by this repository's kernels.

    moe      h[t, j] = act(x[t] . gate[e]) * (x[t] . up[e]), or act(x[t] . up[e]); e = ids[t, j]
             y[t] = sum_j weights[t, j] h[t, j] . down[e] + residual[t]; an id outside 0 .. E-1 counts for nothing
    adapter  y = act(x . w + bias + scales[i] (x . a[i]^T) . b[i]^T) + residual, i = ids[row]; an id outside
             0 .. n-1 leaves the row without an adapter
    log_probs       with d = scale (z - max z): logprob = d[token] - L, L = log sum exp d, entropy = -sum p log p,
                    p = exp(d - L), and the largest `top` logits' places and log probabilities (ties: the lowest
                    place first); a token outside 0 .. V-1 gives 0
    log_probs_grad  of sum(dlogprob * logprob + dentropy * entropy) with respect to z
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------- cases --

def listed():
    moe = {"op": "moe", "dtype": "bf16", "act": "silu", "gated": True, "transb": True, "residual": False,
           "absent": 0.0, "skew": 0.5}
    ada = {"op": "adapter", "dtype": "bf16", "act": "none", "bias": False, "transb": True, "residual": False,
           "plain_rows": 0.0}
    lp = {"scale": 1.0, "masked": 0.0, "padded": 0.0}
    return [
        # one token through a layer of 32 experts, 4 of them: latency, and reading their weights once
        dict(moe, name="moe 1 token", tokens=1, hidden=4096, inner=2048, experts=32, top=4),
        # a small decoding batch, many small experts, weights stored K x N
        dict(moe, name="moe 16 tokens", tokens=16, hidden=2048, inner=1024, experts=64, top=8, transb=False,
             residual=True),
        # a decoding batch over few large experts: every one of them is used, by several tokens
        dict(moe, name="moe 64 tokens", tokens=64, hidden=4096, inner=8192, experts=8, top=2),
        # full precision, no gate, odd sizes; a part of the experts lives elsewhere
        dict(moe, name="moe odd f32", tokens=7, hidden=1001, inner=515, experts=6, top=3, dtype="f32", act="gelu",
             gated=False, absent=0.3),
        # one token of one request
        dict(ada, name="adapter 1 row", rows=1, k=4096, n=4096, adapters=8, rank=16, runs=1),
        # a decoding batch: a request per row, most with an adapter of their own
        dict(ada, name="adapter 48 rows", rows=48, k=4096, n=8192, adapters=32, rank=32, runs=48, residual=True,
             plain_rows=0.2),
        # prompts of eight requests in one batch
        dict(ada, name="adapter prompts", rows=4096, k=4096, n=8192, adapters=8, rank=64, runs=8, act="silu",
             transb=False),
        # full precision, odd sizes
        dict(ada, name="adapter odd f32", rows=333, k=1001, n=515, adapters=5, rank=7, runs=11, dtype="f32",
             bias=True, act="gelu", plain_rows=0.3),
        # the next token of one answer, some tokens forbidden, with alternatives
        dict(lp, name="log_probs 1 row", op="log_probs", rows=1, vocab=131072, top=20, dtype="f32", masked=0.3,
             scale=1.25),
        # scoring a long batch of prompts, odd sizes
        dict(lp, name="log_probs prompts", op="log_probs", rows=4001, vocab=50021, top=5, dtype="bf16",
             padded=0.1),
        # the loss of a training batch
        dict(lp, name="log_probs_grad training", op="log_probs_grad", rows=4096, vocab=32768, dtype="bf16",
             entropy=False, padded=0.1),
        # a short batch with an entropy term, odd sizes
        dict(lp, name="log_probs_grad odd f32", op="log_probs_grad", rows=77, vocab=50021, dtype="f32",
             entropy=True, scale=0.7),
    ]


def draw(rng):
    log = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))  # noqa: E731

    def width(lo, hi):
        v = log(lo, hi)   # most layers' widths are multiples of 64; the others stay odd
        return max(64, v // 64 * 64) if rng.random() < 0.7 else v

    while True:
        op = rng.choice(["moe", "adapter", "log_probs", "log_probs_grad"])
        c = {"op": op, "dtype": rng.choice(["bf16", "bf16", "f32"])}
        half = 0.5 if c["dtype"] == "f32" else 1.0
        if op == "moe":
            e = log(2, 64)
            c.update(tokens=log(1, 128), hidden=width(64, 8192), inner=width(64, 8192), experts=e,
                     top=rng.randint(1, min(8, e)), act=rng.choice(["silu", "silu", "gelu", "gelu_tanh", "relu"]),
                     gated=rng.random() < 0.8, transb=rng.random() < 0.5, residual=rng.random() < 0.3,
                     absent=rng.choice([0.0, 0.0, 0.4]), skew=round(rng.uniform(0.0, 0.8), 2))
            elems = e * c["hidden"] * c["inner"] * (3 if c["gated"] else 2)
            if elems <= 8.0e8 * half and work(c)["flops"] <= 2.6e10 * half:
                return c
        elif op == "adapter":
            rows = log(1, 4096)
            c.update(rows=rows, k=width(64, 8192), n=width(64, 8192), adapters=log(1, 64),
                     rank=rng.choice([8, 16, 16, 32, 64, rng.randint(1, 64)]), runs=min(rows, log(1, 64)),
                     act=rng.choice(["none", "none", "silu", "gelu_tanh"]), bias=rng.random() < 0.4,
                     transb=rng.random() < 0.6, residual=rng.random() < 0.3,
                     plain_rows=rng.choice([0.0, 0.0, 0.3]))
            if work(c)["flops"] <= 2.75e11 * half:
                return c
        else:
            c.update(rows=log(1, 4096), vocab=log(32, 131072), scale=rng.choice([1.0, 1.0, 0.7, 1.25]),
                     masked=rng.choice([0.0, 0.0, 0.3]), padded=rng.choice([0.0, 0.1]))
            if op == "log_probs":
                c["top"] = min(c["vocab"] // 4, rng.choice([0, 1, 5, 20, rng.randint(1, 64)]))
            else:
                c["entropy"] = rng.random() < 0.5
            if c["rows"] * c["vocab"] <= 2.0e8 * half * (1.0 if op == "log_probs" else 0.65):
                return c


def work(case):
    c = case
    es = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "moe":
        t, h, i, e, k = c["tokens"], c["hidden"], c["inner"], c["experts"], c["top"]
        per = h * i * (3 if c["gated"] else 2)
        live = t * k * (1 - c["absent"])
        used = e * (1 - (1 - 1 / e) ** live) if t > 1 else live   # experts that get a token (expected)
        return {"bytes": int(used * per * es + t * h * es * (3 if c["residual"] else 2) + t * k * 8),
                "flops": int(2 * live * per)}
    if c["op"] == "adapter":
        rows, k, n, r = c["rows"], c["k"], c["n"], c["rank"]
        live = rows * (1 - c["plain_rows"])
        runs = c["runs"] * (1 - c["plain_rows"])
        used = c["adapters"] * (1 - (1 - 1 / c["adapters"]) ** runs)
        byts = (rows * (k + n * (2 if c["residual"] else 1)) + k * n + used * r * (k + n) +
                (n if c["bias"] else 0)) * es + 4 * rows
        return {"bytes": int(byts), "flops": int(2 * rows * k * n + 2 * live * r * (k + n))}
    cells = c["rows"] * c["vocab"]
    if c["op"] == "log_probs":
        return {"bytes": cells * es + c["rows"] * (4 + 16 + 8 * c["top"]), "flops": 6 * cells}
    return {"bytes": 2 * cells * es + c["rows"] * 20, "flops": (9 if c["entropy"] else 6) * cells}


# ------------------------------------------------------------------ inputs --

class State:
    pass


def prepare(case, seed):
    c, s = case, State()
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = random.Random(seed * 1000003 + 29)
    dt = DTYPES[c["dtype"]]
    randn = lambda *shape, scale=1.0: torch.randn(shape, generator=gen, device="cuda").mul_(scale).to(dt)  # noqa: E731
    uniform = lambda *shape: torch.rand(shape, generator=gen, device="cuda")  # noqa: E731
    s.case, s.dt = c, dt
    if c["op"] == "moe":
        t, h, i, e = c["tokens"], c["hidden"], c["inner"], c["experts"]
        n = 2 * i if c["gated"] else i   # with a gate: its columns first, then the others
        s.x = randn(t, h)
        s.up = randn(e, *((n, h) if c["transb"] else (h, n)), scale=h ** -0.5)
        s.down = randn(e, *((h, i) if c["transb"] else (i, h)), scale=i ** -0.5)
        s.residual = randn(t, h) if c["residual"] else None
        # what a router leaves: some experts more popular than others, distinct ones per token
        logits = torch.randn((t, e), generator=gen, device="cuda") + \
            c["skew"] * torch.randn((1, e), generator=gen, device="cuda")
        best, ids = logits.topk(c["top"], dim=1)
        s.weights = torch.softmax(best, dim=1)
        if c["absent"]:
            ids = torch.where(uniform(t, c["top"]) < c["absent"], torch.full_like(ids, -1), ids)
        s.ids = ids.to(torch.int32)
    elif c["op"] == "adapter":
        rows, k, n, r, m = c["rows"], c["k"], c["n"], c["rank"], c["adapters"]
        s.x = randn(rows, k)
        s.w = randn(*((n, k) if c["transb"] else (k, n)), scale=k ** -0.5)
        s.a = randn(m, r, k, scale=k ** -0.5)
        s.b = randn(m, n, r, scale=0.5 * r ** -0.5)
        s.scales = 0.5 + uniform(m)
        s.bias = randn(n, scale=0.5) if c["bias"] else None
        s.residual = randn(rows, n) if c["residual"] else None
        # requests one after another, each with one adapter or none
        cuts = sorted(rng.sample(range(1, rows), c["runs"] - 1)) if c["runs"] > 1 else []
        ids = []
        for lo, hi in zip([0] + cuts, cuts + [rows]):
            ids += [-1 if rng.random() < c["plain_rows"] else rng.randrange(m)] * (hi - lo)
        s.ids = torch.tensor(ids, dtype=torch.int32, device="cuda")
    else:
        rows, v = c["rows"], c["vocab"]
        z = torch.randn((rows, v), generator=gen, device="cuda").mul_(2.5)
        s.tokens = torch.randint(0, v, (rows,), generator=gen, device="cuda", dtype=torch.int32)
        # models are fairly sure of the tokens that they are asked about
        z.scatter_add_(1, s.tokens.long()[:, None], 8.0 * uniform(rows, 1))
        if c["masked"]:
            hide = uniform(rows, v) < c["masked"]
            hide.scatter_(1, s.tokens.long()[:, None], False)
            z.masked_fill_(hide, -math.inf)
        if c["padded"]:
            s.tokens.masked_fill_(uniform(rows) < c["padded"], -1)
        s.logits = z.to(dt)
        if c["op"] == "log_probs_grad":
            # what the forward pass left: the row's largest logit, L and the entropy
            top, total, entropy = [], [], []
            for lo in range(0, rows, 256):
                m, d, total_, _, h = _row_values(s.logits[lo:lo + 256].double(), c["scale"])
                top.append(m), total.append(total_), entropy.append(h)
            s.stats = torch.cat([torch.cat(top), torch.cat(total)], dim=1).float()
            s.entropy = torch.cat(entropy)[:, 0].float()
            s.dlogprob = torch.randn((rows,), generator=gen, device="cuda") / rows
            s.dentropy = torch.full((rows,), -0.01 / rows, device="cuda") if c["entropy"] else None
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


def _plain_moe(s):
    c = s.case
    t, e, k, inner = c["tokens"], c["experts"], c["top"], c["inner"]
    live = (s.ids >= 0) & (s.ids < e)
    ids = torch.where(live, s.ids, torch.zeros_like(s.ids)).long()
    share = torch.where(live, s.weights, torch.zeros_like(s.weights))
    x = s.x.float()

    def oriented(w):
        w = w.float()
        return w.transpose(1, 2).contiguous() if c["transb"] else w

    few = t * k <= e   # fewer places than experts: those experts' weights alone
    if few:
        at = ids.reshape(-1)
        up, down = oriented(s.up[at]), oriented(s.down[at])
        xs = x[:, None, :].expand(t, k, x.shape[1]).reshape(t * k, 1, -1)
    else:
        up, down = oriented(s.up), oriented(s.down)
        xs = x[None].expand(e, *x.shape).contiguous()
    z = torch.bmm(xs, up)
    h = _act(z[..., :inner], c["act"]) * z[..., inner:] if c["gated"] else _act(z, c["act"])
    out = torch.bmm(h, down)
    if few:
        y = (out.reshape(t, k, -1) * share[:, :, None]).sum(1)
    else:
        to = torch.zeros((t, e), device="cuda").scatter_add_(1, ids, share)
        y = (out * to.t()[:, :, None]).sum(0)
    if s.residual is not None:
        y = y + s.residual.float()
    return {"y": y.to(s.dt)}


def _plain_adapter(s):
    c = s.case
    n, r, m = c["n"], c["rank"], c["adapters"]
    x, w = s.x.float(), s.w.float()
    z = x @ (w.t() if c["transb"] else w)
    # every row through every adapter, its own kept
    mine = (s.ids[:, None] == torch.arange(m, device="cuda")[None, :]).float() * s.scales[None, :]
    t = (x @ s.a.float().reshape(m * r, -1).t()).reshape(-1, m, r) * mine[:, :, None]
    z = z + t.reshape(-1, m * r) @ s.b.float().permute(0, 2, 1).reshape(m * r, n)
    if s.bias is not None:
        z = z + s.bias.float()
    y = _act(z, c["act"])
    if s.residual is not None:
        y = y + s.residual.float()
    return {"y": y.to(s.dt)}


def _row_values(z, scale):
    """Of rows of logits: the largest, the scaled distances from it, the logarithm of the sum of their
    exponentials, the probabilities, the entropy."""
    m = z.max(dim=1, keepdim=True).values
    d = (z - m) * scale
    e = torch.exp(d)
    total = e.sum(dim=1, keepdim=True)
    p = e / total
    # a forbidden place has d = -infinity and p = 0
    h = torch.log(total) - torch.where(p > 0, p * d, torch.zeros_like(p)).sum(dim=1, keepdim=True)
    return m, d, torch.log(total), p, h


def _plain_log_probs(s):
    c = s.case
    z = s.logits.float()
    m, d, total, _, entropy = _row_values(z, c["scale"])
    held = (s.tokens >= 0) & (s.tokens < c["vocab"])
    at = torch.where(held, s.tokens, torch.zeros_like(s.tokens)).long()[:, None]
    logprob = (d.gather(1, at) - total)[:, 0]
    found = {"logprob": torch.where(held, logprob, torch.zeros_like(logprob)), "entropy": entropy[:, 0],
             "stats": torch.cat([m, total], dim=1)}
    if c["top"]:
        # stable: equal logits stay in the order of their places
        order = z.sort(dim=1, descending=True, stable=True)[1][:, :c["top"]]
        found["top_ids"] = order.to(torch.int32)
        found["top_logprobs"] = d.gather(1, order) - total
    return found


def _plain_log_probs_grad(s):
    c = s.case
    logp = (s.logits.float() - s.stats[:, :1]) * c["scale"] - s.stats[:, 1:]
    p = torch.exp(logp)
    held = (s.tokens >= 0) & (s.tokens < c["vocab"])
    g = torch.where(held, s.dlogprob, torch.zeros_like(s.dlogprob))[:, None]
    hit = torch.arange(c["vocab"], device="cuda")[None, :] == s.tokens[:, None]
    dz = torch.where(hit, g, torch.zeros_like(g)) - g * p
    if s.dentropy is not None:
        dz = dz - s.dentropy[:, None] * torch.where(p > 0, p * (logp + s.entropy[:, None]), torch.zeros_like(p))
    return {"dlogits": (dz * c["scale"]).to(s.dt)}


PLAIN = {"moe": _plain_moe, "adapter": _plain_adapter, "log_probs": _plain_log_probs,
         "log_probs_grad": _plain_log_probs_grad}


# --------------------------------------------------------------------- run --

def _kernels(s):
    import dense_gemm_03_amd as dg
    c = s.case
    if c["op"] == "moe":
        return {"y": dg.moe_layer(s.x, s.up, s.down, s.ids, s.weights, act=c["act"], residual=s.residual,
                                  gated=c["gated"], transb=c["transb"], out_dtype=s.dt)}
    if c["op"] == "adapter":
        return {"y": dg.adapter_linear(s.x, s.w, s.a, s.b, s.ids, scales=s.scales, bias=s.bias, act=c["act"],
                                       residual=s.residual, transb=c["transb"], out_dtype=s.dt)}
    if c["op"] == "log_probs":
        got = dg.log_probs(s.logits, s.tokens, top=c["top"], scale=c["scale"])
        found = {"logprob": got.logprob, "entropy": got.entropy, "stats": got.stats}
        if c["top"]:
            found["top_ids"], found["top_logprobs"] = got.top_ids, got.top_logprobs
        return found
    return {"dlogits": dg.log_probs_grad(s.logits, s.tokens, s.stats, s.entropy, dlogprob=s.dlogprob,
                                         dentropy=s.dentropy, scale=c["scale"])}


def run(state):
    if own:
        return _kernels(state)
    return PLAIN[state.case["op"]](state)


# ------------------------------------------------------------------- exact --

def _activation64(z, act):
    if act == "none":
        return z
    if act == "relu":
        return z.clamp(min=0)
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return z * 0.5 * torch.erfc(-z / math.sqrt(2))
    return z * torch.sigmoid(math.sqrt(8 / math.pi) * (z + 0.044715 * z ** 3))


def _exact_moe(s):
    c = s.case
    y = s.residual.double() if s.residual is not None else torch.zeros(s.x.shape, dtype=torch.float64, device="cuda")
    for e in range(c["experts"]):
        t, j = torch.nonzero(s.ids == e, as_tuple=True)
        if t.numel() == 0:
            continue
        up, down = s.up[e].double(), s.down[e].double()
        if c["transb"]:
            up, down = up.T, down.T
        h = s.x[t].double() @ up
        if c["gated"]:
            gate, h = h.chunk(2, dim=1)
            h = h * _activation64(gate, c["act"])
        else:
            h = _activation64(h, c["act"])
        y.index_add_(0, t, s.weights[t, j].double()[:, None] * (h @ down))
    return {"y": y}


def _exact_adapter(s):
    c = s.case
    w = s.w.double().T if c["transb"] else s.w.double()
    z = s.x.double() @ w
    if s.bias is not None:
        z += s.bias.double()
    for i in range(c["adapters"]):
        rows = torch.nonzero(s.ids == i)[:, 0]
        if rows.numel():
            low = s.x[rows].double() @ s.a[i].double().T
            z[rows] += s.scales[i].double() * (low @ s.b[i].double().T)
    y = _activation64(z, c["act"])
    return {"y": y + s.residual.double() if s.residual is not None else y}


def _exact_log_probs(s):
    c = s.case
    parts = []
    for lo in range(0, c["rows"], 512):
        z = s.logits[lo:lo + 512].double()
        tokens = s.tokens[lo:lo + 512].tolist()
        norm = torch.logsumexp(c["scale"] * z, dim=1)
        logp = c["scale"] * z - norm[:, None]
        top = z.max(dim=1).values
        picked = torch.stack([logp[i, t] if 0 <= t < c["vocab"] else torch.zeros_like(norm[0])
                              for i, t in enumerate(tokens)])
        found = {"logprob": picked, "entropy": torch.special.entr(logp.exp()).sum(dim=1),
                 "stats": torch.stack([top, norm - c["scale"] * top], dim=1)}
        if c["top"]:
            # among equal logits the lowest place: places as a second key
            places = torch.argsort(-z, dim=1, stable=True)[:, :c["top"]]
            found["top_ids"] = places.to(torch.int32)
            found["top_logprobs"] = torch.gather(logp, 1, places)
        parts.append(found)
    return {name: torch.cat([p[name] for p in parts]) for name in parts[0]}


def _exact_log_probs_grad(s):
    c = s.case
    out = []
    for lo in range(0, c["rows"], 512):
        hi = min(c["rows"], lo + 512)
        norm = c["scale"] * s.stats[lo:hi, 0].double() + s.stats[lo:hi, 1].double()
        p = torch.exp(c["scale"] * s.logits[lo:hi].double() - norm[:, None])
        dz = torch.zeros_like(p)
        held = torch.nonzero((s.tokens[lo:hi] >= 0) & (s.tokens[lo:hi] < c["vocab"]))[:, 0]
        g = s.dlogprob[lo:hi].double()[held]
        dz[held] -= g[:, None] * p[held]
        dz[held, s.tokens[lo:hi].long()[held]] += g
        if s.dentropy is not None:
            # -entr(p) is p log p, 0 where p is
            dz -= s.dentropy[lo:hi].double()[:, None] * (s.entropy[lo:hi].double()[:, None] * p - torch.special.entr(p))
        out.append(c["scale"] * dz)
    return {"dlogits": torch.cat(out)}


EXACT = {"moe": _exact_moe, "adapter": _exact_adapter, "log_probs": _exact_log_probs,
         "log_probs_grad": _exact_log_probs_grad}


def exact(case, seed):
    return EXACT[case["op"]](prepare(case, seed))
