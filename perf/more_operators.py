"""What the products and norms of any width are measured on.

Three operators: `linear` (a matrix product with bias, activation, gate and
residual in its epilogue), `expert_linear` (the same product grouped by expert,
ragged sizes) and `residual_norm` (the norms after one block and before the
next, with the gate and the residual between them).  A case is a dict of plain
values; `prepare` makes its inputs, `run` takes one pass, in the plain form
(elementary torch operations in 32 bits) or, where `own` is true, through the
framework's public calls; `exact` is the definition in 64 bits.
"""
import math
import random

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f16": 2, "f32": 4}
_ACTIVATIONS = ["none", "gelu", "gelu_tanh", "silu", "relu"]


# ------------------------------------------------------------------- cases
def _lin(name, dtype, rows, inner, outer, **kw):
    c = dict(op="linear", name=name, dtype=dtype, rows=rows, inner=inner, outer=outer, bias=False,
             activation="none", gated=False, residual=False)
    c.update(kw)
    return c


def _exp(name, dtype, experts, rows, inner, outer, **kw):
    c = dict(op="expert_linear", name=name, dtype=dtype, experts=experts, rows=rows, inner=inner,
             outer=outer, bias=False, activation="none", gated=False, scaled=False, skew=0.5, lengths=1)
    c.update(kw)
    return c


def _norm(name, dtype, rows, width, **kw):
    c = dict(op="residual_norm", name=name, dtype=dtype, rows=rows, width=width, norm="layer",
             after=False, before=True, biases=False, gate="none", sequences=1, residual_scale=1.0)
    c.update(kw)
    return c


def listed():
    return [
        # the classifier's hidden layer on eight pooled rows: latency
        _lin("linear_pooled", "bf16", 8, 768, 768, bias=True, activation="gelu"),
        # every vocabulary entry for a few masked tokens: the weights once
        _lin("linear_vocabulary", "bf16", 24, 768, 50368, bias=True),
        # the gated MLP of a wider encoder over a long packed batch
        _lin("linear_gated", "bf16", 32768, 1024, 4096, activation="gelu", gated=True),
        # the way back to the residual stream, ragged batch, with biases
        _lin("linear_residual", "f16", 5003, 1152, 768, bias=True, residual=True),
        # 16 tokens with two experts each: latency, and the weights that are met
        _exp("expert_token", "bf16", 8, 32, 768, 1152, activation="gelu", gated=True),
        # many small experts with a handful to a few hundred rows each
        _exp("expert_many", "f16", 64, 4001, 768, 1152, activation="silu", gated=True, bias=True, lengths=2),
        # a long packed batch with two experts a token: the way up
        _exp("expert_up", "bf16", 8, 65536, 768, 1152, activation="gelu", gated=True, lengths=3),
        # and the way down, each row times its router weight
        _exp("expert_down", "bf16", 8, 65536, 1152, 768, scaled=True, lengths=3),
        # one new token of each of 32 sequences: latency
        _norm("norm_token", "bf16", 32, 768),
        # the residual and the next block's norm over the benchmark's 65536 tokens
        _norm("norm_packed", "bf16", 65536, 768),
        # norms on both sides of the block, a gate for each sequence, RMS
        _norm("norm_both", "f16", 20011, 1152, norm="rms", after=True, gate="sequences", sequences=33),
        # wide rows in 32 bits, a learned scale per channel, biases
        _norm("norm_wide", "f32", 4099, 8192, after=True, biases=True, gate="channels", residual_scale=0.5),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["linear", "linear", "expert_linear", "expert_linear", "residual_norm"])
    if op == "residual_norm":
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        width = _log_int(rng, 32, 16384)
        if rng.random() < 0.7:
            width = (width + 31) // 32 * 32
        rows = _log_int(rng, 1, max(2, min(65536, 65536 * 768 * 2 // (width * _BYTES[dtype]))))
        after = rng.random() < 0.5
        return _norm("", dtype, rows, width, norm=rng.choice(["rms", "layer"]), after=after,
                     before=not after or rng.random() < 0.8, biases=rng.random() < 0.3,
                     gate=rng.choice(["none", "none", "channels", "sequences", "rows"]),
                     sequences=rng.randint(1, min(rows, 64)), residual_scale=rng.choice([1.0, 1.0, 0.5, 2.5]))
    inner = 8 * _log_int(rng, 4, 1024)
    outer = _log_int(rng, 1, 16384)
    if rng.random() < 0.6:
        outer = (outer + 31) // 32 * 32
    gated = rng.random() < 0.4
    rows = _log_int(rng, 1, 65536)
    experts = _log_int(rng, 2, 128) if op == "expert_linear" else 1
    while experts > 2 and experts * inner * outer > 32 << 20:
        experts //= 2
    common = dict(bias=rng.random() < 0.5, activation=rng.choice(_ACTIVATIONS), gated=gated)
    dtype = rng.choice(["bf16", "f16"])
    if op == "linear":
        c = _lin("", dtype, rows, inner, outer, residual=rng.random() < 0.4, **common)
        most = _MOST_LINEAR
    else:
        c = _exp("", dtype, experts, rows, inner, outer, scaled=rng.random() < 0.5,
                 skew=rng.choice([0.0, 0.5, 1.5]), lengths=rng.randint(4, 10 ** 6), **common)
        most = _MOST_EXPERT
    while _over(c, most):       # no more than the largest listed case: fewer rows, then narrower
        if c["rows"] > 256:
            c["rows"] = c["rows"] * 2 // 3
        else:
            c["outer"] = max(1, c["outer"] * 2 // 3)
    return c


def _over(case, most):
    w = work(case)
    return w["bytes"] > most["bytes"] or w["flops"] > most["flops"]


# ------------------------------------------------------------------ inputs
def _sizes(case):
    """Rows of each expert, from the case alone: shares e^(skew z), some of
    them empty where there are few rows."""
    r = random.Random(case["lengths"])
    shares = [math.exp(case["skew"] * r.gauss(0, 1)) for _ in range(case["experts"])]
    n = [0] * case["experts"]
    for e in r.choices(range(case["experts"]), shares, k=case["rows"]):
        n[e] += 1
    return n


def _offsets(lengths):
    out = [0]
    for x in lengths:
        out.append(out[-1] + x)
    return out


def _cuts(case):
    """Offsets of the sequences that share a gate, none of them empty."""
    r = random.Random(case["rows"])
    return [0] + sorted(r.sample(range(1, case["rows"]), case["sequences"] - 1)) + [case["rows"]]


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev).manual_seed(seed)
    t = _TYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32)

    st = dict(case=case)
    if own:
        from encoder_only_transformer_gb300 import binding
        st["binding"] = binding
    T = case["rows"]
    if case["op"] == "residual_norm":
        D = case["width"]
        st["x"] = normal(T, D).mul_(2.0).to(t)              # a residual stream some blocks deep
        st["branch"] = normal(T, D).to(t)
        st["weight"] = (1 + 0.1 * normal(D)).to(t) if case["before"] else None
        st["branch_weight"] = (1 + 0.1 * normal(D)).to(t) if case["after"] else None
        st["bias"] = (0.1 * normal(D)).to(t) if case["before"] and case["biases"] else None
        st["branch_bias"] = (0.1 * normal(D)).to(t) if case["after"] and case["biases"] else None
        st["gate"] = st["cu"] = None
        if case["gate"] == "channels":
            st["gate"] = (0.2 + 0.1 * normal(D)).to(t)
        elif case["gate"] == "rows":
            st["gate"] = normal(T, D).mul_(0.5).to(t)
        elif case["gate"] == "sequences":
            st["gate"] = normal(case["sequences"], D).mul_(0.5).to(t)
            st["cu"] = torch.tensor(_cuts(case), dtype=torch.int32, device=dev)
        st["eps"] = 1e-5
        return st
    K, N, E = case["inner"], case["outer"], case.get("experts", 1)
    W = 2 * N if case["gated"] else N
    st["x"] = normal(T, K).to(t)
    if case["op"] == "linear":
        st["weight"] = normal(W, K).mul_(K ** -0.5).to(t)
        st["bias"] = (0.1 * normal(W)).to(t) if case["bias"] else None
        st["residual"] = normal(T, N).to(t) if case["residual"] else None
        return st
    st["weight"] = torch.empty(E, W, K, dtype=t, device=dev)
    for e in range(E):
        st["weight"][e] = normal(W, K).mul_(K ** -0.5)
    st["bias"] = (0.1 * normal(E, W)).to(t) if case["bias"] else None
    st["row_scale"] = torch.rand(T, generator=g, device=dev) if case["scaled"] else None
    st["offsets"] = _offsets(_sizes(case))
    st["cu"] = torch.tensor(st["offsets"], dtype=torch.int32, device=dev)
    return st


# -------------------------------------------------------------- plain forms
def _plain_activate(z, name):
    if name == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if name == "silu":
        return z / (1.0 + torch.exp(-z))
    if name == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    return z


def _plain_product(x, w, b, case):
    z = x.float() @ w.float().T
    if b is not None:
        z = z + b.float()
    if case["gated"]:
        N = case["outer"]
        return _plain_activate(z[:, :N], case["activation"]) * z[:, N:]
    return _plain_activate(z, case["activation"])


def _plain_norm(z, w, b, norm, eps):
    if norm == "layer":
        z = z - z.mean(-1, keepdim=True)
    y = z / torch.sqrt((z * z).mean(-1, keepdim=True) + eps) * w.float()
    return y if b is None else y + b.float()


def _per_row(gate, cu, T):
    """A sequence's gate for each of its rows."""
    row = torch.arange(T, device=gate.device)
    return gate[torch.searchsorted(cu.long(), row, right=True) - 1]


def run(st):
    case = st["case"]
    if case["op"] == "linear":
        if own:
            return st["binding"].linear(st["x"], st["weight"], bias=st["bias"], activation=case["activation"],
                                        gated=case["gated"], residual=st["residual"])
        y = _plain_product(st["x"], st["weight"], st["bias"], case)
        if st["residual"] is not None:
            y = y + st["residual"].float()
        return y.to(st["x"].dtype)
    if case["op"] == "expert_linear":
        if own:
            return st["binding"].expert_linear(st["x"], st["weight"], st["cu"], bias=st["bias"],
                                               activation=case["activation"], gated=case["gated"],
                                               row_scale=st["row_scale"])
        out = torch.empty(case["rows"], case["outer"], dtype=st["x"].dtype, device=st["x"].device)
        o = st["offsets"]
        for e in range(case["experts"]):
            if o[e] == o[e + 1]:
                continue
            rows = slice(o[e], o[e + 1])
            y = _plain_product(st["x"][rows], st["weight"][e], None if st["bias"] is None else st["bias"][e], case)
            if st["row_scale"] is not None:
                y = y * st["row_scale"][rows, None]
            out[rows] = y.to(out.dtype)
        return out
    if own:
        h, y = st["binding"].residual_norm(
            st["x"], st["branch"], weight=st["weight"], bias=st["bias"], branch_weight=st["branch_weight"],
            branch_bias=st["branch_bias"], gate=st["gate"], cu_seqlens=st["cu"], norm=case["norm"],
            residual_scale=case["residual_scale"], eps=st["eps"])
        return (h, y) if case["before"] else (h,)
    b = st["branch"].float()
    if case["after"]:
        b = _plain_norm(b, st["branch_weight"], st["branch_bias"], case["norm"], st["eps"])
    if st["gate"] is not None:
        gate = _per_row(st["gate"], st["cu"], case["rows"]) if st["cu"] is not None else st["gate"]
        b = b * gate.float()
    h = case["residual_scale"] * st["x"].float() + b
    if not case["before"]:
        return (h.to(st["x"].dtype),)
    return h.to(st["x"].dtype), _plain_norm(h, st["weight"], st["bias"], case["norm"], st["eps"]).to(st["x"].dtype)


# --------------------------------------------------------------------- work
def work(case):
    b, T = _BYTES[case["dtype"]], case["rows"]
    if case["op"] == "residual_norm":
        D = case["width"]
        # x and the branch in, the new stream and its norm out
        n = (4 if case["before"] else 3) * T * D
        n += {"none": 0, "channels": D, "rows": T * D, "sequences": case["sequences"] * D}[case["gate"]]
        sides = int(case["before"]) + int(case["after"])
        n += sides * D * (2 if case["biases"] else 1)
        flops = T * D * (2 + 5 * sides)
        return {"bytes": n * b + (4 * (case["sequences"] + 1) if case["gate"] == "sequences" else 0),
                "flops": flops}
    K, N = case["inner"], case["outer"]
    W = 2 * N if case["gated"] else N
    if case["op"] == "linear":
        met = 1
        n = T * K + T * N * (2 if case["residual"] else 1)
        extra = 0
    else:
        met = sum(1 for x in _sizes(case) if x)      # weights of experts without rows are not read
        n = T * K + T * N
        extra = 4 * (case["experts"] + 1) + (4 * T if case["scaled"] else 0)
    n += met * (W * K + (W if case["bias"] else 0))
    return {"bytes": n * b + extra, "flops": 2 * T * K * W}


_MOST_LINEAR = work(next(c for c in listed() if c["name"] == "linear_gated"))
_MOST_EXPERT = work(next(c for c in listed() if c["name"] == "expert_up"))


# ------------------------------------------------------------ the definition
def _exact_activate(z, name):
    if name == "gelu":
        return z * 0.5 * torch.special.erfc(-z / math.sqrt(2.0))
    if name == "gelu_tanh":
        # (1 + tanh u) / 2 is the logistic function of 2 u
        return z * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3))
    if name == "silu":
        return z * torch.sigmoid(z)
    return torch.clamp(z, min=0.0) if name == "relu" else z


def _exact_product(x, w, b, case):
    N = case["outer"]

    def side(rows):
        z = torch.einsum("tk,nk->tn", x.double(), w[rows].double())
        return z if b is None else z + b[rows].double()

    if case["gated"]:
        return _exact_activate(side(slice(0, N)), case["activation"]) * side(slice(N, 2 * N))
    return _exact_activate(side(slice(0, N)), case["activation"])


def _exact_norm(z, w, b, norm, eps):
    if norm == "rms":
        r = torch.rsqrt((z ** 2).sum(-1) / z.shape[-1] + eps)
        y = torch.einsum("td,t,d->td", z, r, w.double())
    else:
        var, mean = torch.var_mean(z, -1, unbiased=False, keepdim=True)
        y = (z - mean) * torch.rsqrt(var + eps) * w.double()
    return y if b is None else y + b.double()


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "linear":
        y = _exact_product(st["x"], st["weight"], st["bias"], case)
        return y if st["residual"] is None else y + st["residual"].double()
    if case["op"] == "expert_linear":
        parts = []
        o = st["offsets"]
        for e in range(case["experts"]):
            y = _exact_product(st["x"][o[e]:o[e + 1]], st["weight"][e],
                               None if st["bias"] is None else st["bias"][e], case)
            if st["row_scale"] is not None:
                y = torch.einsum("tn,t->tn", y, st["row_scale"][o[e]:o[e + 1]].double())
            parts.append(y)
        return torch.cat(parts)
    z = st["branch"].double()
    if case["after"]:
        z = _exact_norm(z, st["branch_weight"], st["branch_bias"], case["norm"], st["eps"])
    if case["gate"] == "sequences":
        cu = st["cu"].tolist()
        for s in range(case["sequences"]):
            z[cu[s]:cu[s + 1]] = z[cu[s]:cu[s + 1]] * st["gate"][s].double()
    elif case["gate"] != "none":
        z = z * st["gate"].double()
    h = torch.add(z, st["x"].double(), alpha=case["residual_scale"])
    if not case["before"]:
        return (h,)
    return h, _exact_norm(h, st["weight"], st["bias"], case["norm"], st["eps"])
