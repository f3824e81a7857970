"""What the operators beside the attention block are measured on.

Three operators: `rotary` (rotary positions on rows of heads), `norm_rotary`
(the norm of every query and key head with the rotation in the same pass) and
`cross` (attention of packed queries over an encoder's states of another
length).  A case is a dict of plain values; `prepare` makes its inputs, `run`
takes one pass, in the plain form (elementary torch operations in 32 bits) or,
where `own` is true, through the framework's public calls; `exact` is the
definition in 64 bits.
"""
import math
import random

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f16": 2, "f32": 4}


# ------------------------------------------------------------------- cases
def _rot(op, name, dtype, tokens, heads, head_dim, **kw):
    c = dict(op=op, name=name, dtype=dtype, tokens=tokens, heads=heads, kv_heads=0,
             head_dim=head_dim, rotary_dim=head_dim, layout="half", base=10000.0, scaling="none",
             factor=1.0, original=8192, far=8192, packed=False, norm="none", fused=False)
    c.update(kw)
    return c


def _cross(name, dtype, sequences, heads, kv_heads, head_dim, q_min, q_max, k_min, k_max, **kw):
    c = dict(op="cross", name=name, dtype=dtype, sequences=sequences, heads=heads,
             kv_heads=kv_heads, head_dim=head_dim, q_min=q_min, q_max=q_max, k_min=k_min,
             k_max=k_max, lengths=1, padded=False)
    c.update(kw)
    return c


def listed():
    return [
        # one new token of each of 32 sequences, somewhere in its text: latency
        _rot("rotary", "rotary_token", "bf16", 32, 12, 64, base=160000.0),
        # the queries of a long packed batch of the encoder's shape (the
        # benchmark's 65536 tokens), positions from the packing
        _rot("rotary", "rotary_packed", "bf16", 65536, 12, 64, base=160000.0, packed=True),
        # half of each head turned in interleaved pairs, fp16, a stretched
        # context with far positions, an odd number of rows
        _rot("rotary", "rotary_part_yarn", "f16", 5003, 16, 128, rotary_dim=64,
             layout="interleaved", scaling="yarn", factor=16.0, far=131072),
        # a decode step's queries and keys out of the fused projection rows
        _rot("norm_rotary", "norm_rotary_token", "bf16", 8, 12, 64, kv_heads=12, norm="rms",
             fused=True),
        # a prompt's queries and keys out of the fused projection rows
        # (row pitch 2304, as the encoder's Wqkv writes them)
        _rot("norm_rotary", "norm_rotary_packed", "bf16", 65536, 12, 64, kv_heads=12, norm="rms",
             packed=True, fused=True, base=160000.0),
        # few shared key heads, LayerNorm, fp16, part of a wide head, odd rows
        _rot("norm_rotary", "norm_rotary_shared", "f16", 9001, 32, 128, kv_heads=4, norm="layer",
             rotary_dim=96, layout="interleaved", scaling="by_parts", factor=8.0, far=65536),
        # a decoder's token over four short texts' states: latency
        _cross("cross_token_short", "bf16", 4, 12, 12, 64, 1, 1, 60, 300),
        # a decode step of 32 sequences over long texts' states: K and V once
        _cross("cross_token_long", "bf16", 32, 12, 12, 64, 1, 1, 128, 8192),
        # the same with shared key heads, a few drafted tokens, wide heads, fp16
        _cross("cross_token_shared", "f16", 16, 32, 8, 128, 1, 4, 1000, 5000),
        # a whole text of queries over a whole text of states
        _cross("cross_prompt", "bf16", 1, 12, 12, 64, 8192, 8192, 8192, 8192),
        # a padded batch: 16 rows of 250 queries over states padded to 2011
        _cross("cross_padded", "bf16", 16, 12, 12, 64, 250, 250, 100, 2011, padded=True),
        # ragged prompts, shared key heads, wide heads, fp16
        _cross("cross_prompt_shared", "f16", 6, 16, 4, 128, 300, 2500, 500, 6000),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary", "norm_rotary", "cross", "cross"])
    if op == "cross":
        head_dim = rng.choice([64, 64, 128])
        kv = rng.choice([1, 2, 4, 8, 12])
        group = rng.choice([1, 1, 2, 4, 8])
        heads = min(kv * group, 32) // kv * kv
        dtype = rng.choice(["bf16", "f16"])
        if rng.random() < 0.5:      # single tokens (or a few) over long states
            n = _log_int(rng, 1, 64)
            q_max = rng.choice([1, 1, 1, 2, 5, 16])
            k_max = _log_int(rng, 30, 8192)
        else:                       # prompts
            n = _log_int(rng, 1, 16)
            q_max = _log_int(rng, 17, 4096)
            k_max = _log_int(rng, 30, 8192)
        while n * heads * head_dim * q_max * k_max > 12 * 64 * 8192 * 8192 or \
                n * kv * head_dim * k_max > 12 * 64 * 8192 * 16:
            n = max(1, n // 2)
            k_max = max(30, k_max * 2 // 3)
        padded = rng.random() < 0.3
        return _cross("", dtype, n, heads, kv, head_dim, q_max if padded else rng.randint(1, q_max),
                      q_max, rng.choice([0, 1, k_max // 2, k_max]), k_max,
                      lengths=rng.randint(2, 10 ** 6), padded=padded)
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    head_dim = rng.choice([64, 64, 80, 96, 128, 256])
    heads = rng.choice([1, 2, 4, 8, 12, 16, 32])
    kv = rng.choice([1, 2, 4, heads]) if op == "norm_rotary" else 0
    kv = min(kv, heads)
    most = 65536 * 12 * 64 * 2 // ((heads + kv) * head_dim * (_BYTES[dtype] // 2 or 1))
    tokens = _log_int(rng, 1, min(65536, most))
    part = rng.choice([head_dim, head_dim, head_dim // 2, head_dim // 4])
    scaling = rng.choice(["none", "linear", "ntk", "by_parts", "yarn"])
    return _rot(op, "", dtype, tokens, heads, head_dim, kv_heads=kv, rotary_dim=part // 2 * 2,
                layout=rng.choice(["half", "interleaved"]),
                base=rng.choice([10000.0, 160000.0, 500000.0]), scaling=scaling,
                factor=1.0 if scaling == "none" else rng.choice([2.0, 4.0, 16.0]),
                far=_log_int(rng, 100, 1000000), packed=rng.random() < 0.5,
                norm=rng.choice(["rms", "layer"]) if op == "norm_rotary" else "none",
                fused=rng.random() < 0.5)


# ------------------------------------------------------------------ inputs
def _scaling(case):
    if case["scaling"] == "none":
        return None
    s = {"kind": case["scaling"], "factor": case["factor"]}
    if case["scaling"] in ("by_parts", "yarn"):
        s["original"] = case["original"]
    return s


def _lengths(case):
    """Per sequence (queries, states), from the case alone."""
    r = random.Random(case["lengths"])
    n = case["sequences"]
    q = [r.randint(case["q_min"], case["q_max"]) for _ in range(n)]
    k = [r.randint(case["k_min"], case["k_max"]) for _ in range(n)]
    if case["padded"]:
        q = [case["q_max"]] * n
    return q, k


def _offsets(lengths):
    out = [0]
    for x in lengths:
        out.append(out[-1] + x)
    return out


def _packing(tokens):
    """Sequence lengths in 128..8192 that fill `tokens` rows."""
    r = random.Random(tokens)
    out, left = [], tokens
    while left > 0:
        out.append(min(left, r.randint(128, 8192)))
        left -= out[-1]
    return out


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev).manual_seed(seed)
    t = _TYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32)

    st = dict(case=case)
    D, H, K = case["head_dim"], case["heads"], case["kv_heads"]
    if case["op"] == "cross":
        ql, kl = _lengths(case)
        if case["padded"]:
            # right-padded rows, as a tokenizer pads a batch
            B, Sq, Sk = case["sequences"], case["q_max"], max(1, case["k_max"])
            st["q"] = normal(B, Sq, H, D).to(t)
            kv = normal(B, Sk, 2 * K, D).to(t)
            st["k"], st["v"] = kv[:, :, :K], kv[:, :, K:]
            st["key_mask"] = (torch.arange(Sk, device=dev)[None, :]
                              < torch.tensor(kl, device=dev)[:, None]).to(torch.int32)
        else:
            qo, ko = _offsets(ql), _offsets(kl)
            st["q"] = normal(qo[-1], H, D).to(t)
            kv = normal(ko[-1], 2 * K, D).to(t)       # one fused key/value projection
            st["k"], st["v"] = kv[:, :K], kv[:, K:]
            st["qo"], st["ko"] = qo, ko
            st["cu_q"] = torch.tensor(qo, dtype=torch.int32, device=dev)
            st["cu_k"] = torch.tensor(ko, dtype=torch.int32, device=dev)
        if own:
            from encoder_only_transformer_gb300 import binding
            st["binding"] = binding
        return st
    T = case["tokens"]
    if case["fused"]:
        rows = normal(T, H + 2 * max(K, 1), D).to(t)  # Q | K | V of a fused projection
        st["q"], st["k"] = rows[:, :H], rows[:, H:H + K]
    else:
        st["q"], st["k"] = normal(T, H, D).to(t), normal(T, max(K, 1), D).to(t)[:, :K]
    if case["packed"]:
        cu = _offsets(_packing(T))
        st["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev)
        st["positions"] = None
    else:
        st["positions"] = torch.randint(0, case["far"], (T,), generator=g, device=dev,
                                        dtype=torch.int32)
        st["cu"] = None
    if case["norm"] != "none":
        st["wq"] = (1 + 0.1 * normal(D)).to(t)
        st["wk"] = (1 + 0.1 * normal(D)).to(t)
    st["eps"] = 1e-6
    if own:
        from encoder_only_transformer_gb300 import binding
        st["binding"] = binding
        st["rope"] = binding.Rotary(case["rotary_dim"], base=case["base"], layout=case["layout"],
                                    scaling=_scaling(case))
    return st


# -------------------------------------------------------------- plain forms
def _plain_freqs(case, dev):
    """Radians per position of each pair (64 bits) and the amplitude."""
    R, base, s, kind = case["rotary_dim"], case["base"], case["factor"], case["scaling"]
    m = torch.arange(R // 2, dtype=torch.float64, device=dev)
    if kind == "ntk":
        base = base * s ** (R / (R - 2))
    f = base ** (-2.0 * m / R)
    if kind == "linear":
        f = f / s
    elif kind == "by_parts":
        # pairs that turn more than 32 times over the original context keep
        # their frequency, those that turn less than once are stretched
        keep = ((case["original"] * f / (2 * math.pi) - 1.0) / (32.0 - 1.0)).clamp(0, 1)
        f = f * keep + f / s * (1 - keep)
    elif kind == "yarn":
        # the same two borders as pair numbers, rounded outwards, and a ramp
        # over the pair numbers between them
        def pair_at(turns):
            return R * math.log(case["original"] / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo = max(math.floor(pair_at(32.0)), 0)
        hi = min(math.ceil(pair_at(1.0)), R - 1)
        keep = 1 - ((m - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        f = f * keep + f / s * (1 - keep)
    amp = 0.1 * math.log(s) + 1.0 if kind == "yarn" else 1.0
    return f, amp


def _plain_positions(st, T):
    if st["positions"] is not None:
        return st["positions"]
    cu = st["cu"].long()
    row = torch.arange(T, device=cu.device)
    return row - cu[torch.searchsorted(cu, row, right=True) - 1]


def _plain_heads(x, w, st, cos, sin):
    case = st["case"]
    y = x.float()
    if case["norm"] != "none":
        if case["norm"] == "layer":
            y = y - y.mean(-1, keepdim=True)
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + st["eps"]) * w.float()
    R = case["rotary_dim"]
    if case["layout"] == "half":
        a, b = y[..., :R // 2], y[..., R // 2:R]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = y[..., 0:R:2], y[..., 1:R:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, y[..., R:]], -1).to(x.dtype)


def _plain_attend(q, k, v, mask=None):
    """[Lq, H, D] over [Lk, K, D]; mask [Lk] of truth values."""
    g = q.shape[1] // k.shape[1]
    qf = q.float().transpose(0, 1)
    kf = k.float().transpose(0, 1).repeat_interleave(g, 0)
    vf = v.float().transpose(0, 1).repeat_interleave(g, 0)
    if k.shape[0] == 0:
        return torch.zeros_like(q)
    s = qf @ kf.transpose(1, 2) * (q.shape[2] ** -0.5)
    if mask is not None:
        s = torch.where(mask[None, None, :], s, torch.full_like(s, -math.inf))
    top = s.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    p = torch.exp(s - top)
    total = p.sum(-1, keepdim=True)
    o = (p @ vf) / torch.where(total == 0, torch.ones_like(total), total)
    return o.transpose(0, 1).to(q.dtype)


def run(st):
    case = st["case"]
    if own:
        b = st["binding"]
        if case["op"] == "rotary":
            return b.rotary(st["q"], st["rope"], positions=st["positions"], cu_seqlens=st["cu"])
        if case["op"] == "norm_rotary":
            return b.qk_norm_rotary(st["q"], st["k"], st["wq"], st["wk"], rope=st["rope"],
                                    positions=st["positions"], cu_seqlens=st["cu"],
                                    norm=case["norm"], eps=st["eps"])
        if case["padded"]:
            return b.cross_attention_padded(st["q"], st["k"], st["v"], key_mask=st["key_mask"])
        return b.cross_attention(st["q"], st["k"], st["v"], st["cu_q"], st["cu_k"],
                                 max_seqlen_q=case["q_max"])
    if case["op"] == "cross":
        q, k, v = st["q"], st["k"], st["v"]
        if case["padded"]:
            return torch.stack([_plain_attend(q[b], k[b], v[b], st["key_mask"][b] != 0)
                                for b in range(case["sequences"])])
        qo, ko = st["qo"], st["ko"]
        out = torch.empty_like(q)
        for b in range(case["sequences"]):
            out[qo[b]:qo[b + 1]] = _plain_attend(q[qo[b]:qo[b + 1]], k[ko[b]:ko[b + 1]],
                                                 v[ko[b]:ko[b + 1]])
        return out
    f, amp = _plain_freqs(case, st["q"].device)
    ang = _plain_positions(st, case["tokens"]).double()[:, None] * f
    cos, sin = (amp * torch.cos(ang)).float()[:, None], (amp * torch.sin(ang)).float()[:, None]
    if case["op"] == "rotary":
        return _plain_heads(st["q"], None, st, cos, sin)
    return (_plain_heads(st["q"], st["wq"], st, cos, sin),
            _plain_heads(st["k"], st["wk"], st, cos, sin))


# --------------------------------------------------------------------- work
def work(case):
    b, D = _BYTES[case["dtype"]], case["head_dim"]
    if case["op"] == "cross":
        ql, kl = _lengths(case)
        rows = sum(kl)
        by = 2 * sum(ql) * case["heads"] * D * b + 2 * rows * case["kv_heads"] * D * b
        if case["padded"]:
            by += 4 * case["sequences"] * max(1, case["k_max"])
        return {"bytes": by,
                "flops": 4 * D * case["heads"] * sum(x * y for x, y in zip(ql, kl))}
    n = case["tokens"] * (case["heads"] + case["kv_heads"]) * D
    by = 2 * n * b + (4 * case["tokens"] if not case["packed"] else 0)
    if case["norm"] != "none":
        by += 2 * D * b
    flops = 3 * n * case["rotary_dim"] // D + (4 * n if case["norm"] != "none" else 0)
    return {"bytes": by, "flops": flops}


# ------------------------------------------------------------ the definition
def _exact_turn(case, pos):
    """amplitude * e^{i pos f} for every (row, pair), 128-bit complex."""
    import numpy as np
    R, s = case["rotary_dim"], case["factor"]
    f = np.empty(R // 2)
    for m in range(R // 2):
        w = math.exp(-2.0 * m / R * math.log(case["base"]))
        turns = case["original"] * w / (2.0 * math.pi)
        if case["scaling"] == "linear":
            w /= s
        elif case["scaling"] == "ntk":
            w = math.exp(-2.0 * m / R * (math.log(case["base"]) + R / (R - 2) * math.log(s)))
        elif case["scaling"] == "by_parts":
            gamma = min(1.0, max(0.0, (turns - 1.0) / 31.0))
            w = (1.0 - gamma) * w / s + gamma * w
        elif case["scaling"] == "yarn":
            per_pair = 2.0 * math.log(case["base"]) / R
            first = math.floor(math.log(case["original"] / (64.0 * math.pi)) / per_pair)
            last = math.ceil(math.log(case["original"] / (2.0 * math.pi)) / per_pair)
            first, last = max(first, 0), min(last, R - 1)
            ramp = min(1.0, max(0.0, (m - first) / max(last - first, 1e-3)))
            w = ramp * w / s + (1.0 - ramp) * w
        f[m] = w
    amp = 1.0 + 0.1 * math.log(s) if case["scaling"] == "yarn" else 1.0
    ang = pos.double()[:, None] * torch.from_numpy(f).to(pos.device)[None]
    return torch.polar(torch.full_like(ang, amp), ang)


def _exact_heads(case, x, w, eps, turn):
    z = x.double()
    if case["norm"] == "rms":
        z = z * torch.rsqrt((z ** 2).sum(-1) / z.shape[-1] + eps)[..., None] * w.double()
    elif case["norm"] == "layer":
        var, mean = torch.var_mean(z, -1, unbiased=False, keepdim=True)
        z = (z - mean) * torch.rsqrt(var + eps) * w.double()
    R = case["rotary_dim"]
    out = z.clone()
    if case["layout"] == "half":
        c = torch.complex(z[..., :R // 2].contiguous(), z[..., R // 2:R].contiguous()) * turn[:, None]
        out[..., :R // 2], out[..., R // 2:R] = c.real, c.imag
    else:
        c = torch.complex(z[..., 0:R:2].contiguous(), z[..., 1:R:2].contiguous()) * turn[:, None]
        out[..., 0:R:2], out[..., 1:R:2] = c.real, c.imag
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] != "cross":
        if st["positions"] is not None:
            pos = st["positions"]
        else:
            cu = st["cu"].tolist()
            pos = torch.cat([torch.arange(b - a, device=st["cu"].device)
                             for a, b in zip(cu, cu[1:])])
        turn = _exact_turn(case, pos)
        if case["op"] == "rotary":
            return _exact_heads(case, st["q"], None, 0.0, turn)
        return (_exact_heads(case, st["q"], st["wq"], st["eps"], turn),
                _exact_heads(case, st["k"], st["wk"], st["eps"], turn))
    q, k, v = st["q"], st["k"], st["v"]
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    group = case["heads"] // case["kv_heads"]
    ql, kl = _lengths(case)
    for b in range(case["sequences"]):
        if kl[b] == 0 or ql[b] == 0:
            continue
        if case["padded"]:      # the visible keys of a row are its first ones
            qb, kb, vb, ob = q[b], k[b, :kl[b]], v[b, :kl[b]], out[b]
        else:
            i, j = st["qo"][b], st["ko"][b]
            qb, ob = q[i:i + ql[b]], out[i:i + ql[b]]
            kb, vb = k[j:j + kl[b]], v[j:j + kl[b]]
        for h in range(case["heads"]):
            s = torch.einsum("id,jd->ij", qb[:, h].double(), kb[:, h // group].double())
            p = torch.softmax(s / math.sqrt(case["head_dim"]), -1)
            ob[:, h] = torch.einsum("ij,jd->id", p, vb[:, h // group].double())
    return out
