"""Rotary positions and per-head norms (binding.rotary, binding.qk_norm_rotary)
against their formulas in 64 bits.

Tolerances, from the arithmetic.  The output is rounded once to type t: at most
u_t = eps_t / 2 relative to the value.  Before that everything is fp32 with
u = 2^-24: a turned number is x0 c - x1 s with each of c, s off by the function's
own error (fp32 rows: 2 ulp of sincospif; 16-bit rows: 2^-20.9 = 8.6 u of the
fast sine), the angle's (a fraction of turns exact to 2^-32, rounded to fp32:
at most pi u + 0.1 u rad) and the amplitude's product (1 u), then two products
and a sum (3 u): below 16.1 u (|x0| + |x1|) a absolute, 18 u taken.  A norm adds
its factor: a mean of D <= 256 squares summed in D / lanes + 5 steps (below
20 u), rsqrt (2 ulp, 4 u), two products (2 u); relative 28 u taken on x0 and x1.
LayerNorm also subtracts the mean: 24 u max|x| absolute before the
factor.
"""
import ctypes
import math

import pytest
import torch

from encoder_only_transformer_gb300 import binding

U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


@pytest.fixture(scope="module")
def built():
    import __graft_entry__
    __graft_entry__.build()


def freqs(dim, base=10000.0, kind="none", factor=1.0, original=8192.0, low=1.0, high=32.0):
    """Frequencies and amplitude from the definitions, one pair at a time."""
    out = []
    for m in range(dim // 2):
        f = base ** (-2 * m / dim)
        turns = original * f / (2 * math.pi)
        if kind == "linear":
            f /= factor
        elif kind == "ntk":
            f = (base * factor ** (dim / (dim - 2))) ** (-2 * m / dim)
        elif kind == "by_parts":
            g = min(1.0, max(0.0, (turns - low) / (high - low)))
            f = (1 - g) * f / factor + g * f
        elif kind == "yarn":
            def pair(t):
                return dim * math.log(original / (t * 2 * math.pi)) / (2 * math.log(base))
            lo, hi = max(math.floor(pair(high)), 0), min(math.ceil(pair(low)), dim - 1)
            r = min(1.0, max(0.0, (m - lo) / max(hi - lo, 1e-3)))
            f = r * f / factor + (1 - r) * f
        out.append(f)
    return out, (0.1 * math.log(factor) + 1 if kind == "yarn" else 1.0)


def reference(x, pos, f, amp, layout, norm=None, w=None, eps=0.0, inverse=False):
    """-> (value, tolerance before the last rounding), both fp64 on the CPU."""
    z = x.double().cpu()
    slack = torch.zeros_like(z)
    if norm:
        w = w.double().cpu()
        big = z.abs().amax(-1, keepdim=True)
        if norm == "layer":
            z = z - z.mean(-1, keepdim=True)
        inv = ((z * z).mean(-1, keepdim=True) + eps) ** -0.5
        if norm == "layer":
            slack = 24 * U * big * inv * w.abs()
        z = z * inv * w
        slack = slack + 28 * U * z.abs()
    R = 2 * len(f)
    if R == 0:
        return z, slack + U * z.abs()
    ang = pos.double().cpu()[:, None] * torch.tensor(f, dtype=torch.float64)
    c, s = amp * torch.cos(ang)[:, None], amp * torch.sin(ang)[:, None] * (-1 if inverse else 1)
    i0 = torch.arange(R // 2) if layout == "half" else torch.arange(0, R, 2)
    i1 = i0 + R // 2 if layout == "half" else i0 + 1
    a, b = z[..., i0], z[..., i1]
    out, tol = z.clone(), slack.clone()
    out[..., i0], out[..., i1] = a * c - b * s, b * c + a * s
    t = amp * (18 * U * (a.abs() + b.abs()) + slack[..., i0] + slack[..., i1])
    tol[..., i0] = t
    tol[..., i1] = t
    # the frequency itself is a double: pos * f is off by a few 2^-53 of itself
    far = (ang.abs() * 2.0 ** -51)[:, None] * amp * (a.abs() + b.abs())
    tol[..., i0] += far
    tol[..., i1] += far
    return out, tol


def check(got, ref, tol):
    got = got.double().cpu()
    u = torch.finfo(TYPES["f32"]).eps / 2
    assert torch.isfinite(got).all()
    err = (got - ref).abs()
    bound = tol + (ref.abs() + tol) * u
    worst = ((err - bound) / (bound + 1e-300)).max().item() if err.numel() else -1
    assert (err <= bound).all(), f"worst excess {worst:.3e}, max err {err.max().item():.3e}"


def check_typed(got, ref, tol):
    if got.dtype == torch.float32:
        return check(got, ref, tol)
    u = torch.finfo(got.dtype).eps / 2
    tiny = torch.finfo(got.dtype).smallest_normal * torch.finfo(got.dtype).eps / 2
    g = got.double().cpu()
    assert torch.isfinite(g).all()
    err, bound = (g - ref).abs(), tol + (ref.abs() + tol) * u + tiny
    assert (err <= bound).all(), f"max err {err.max().item():.3e}, excess {(err - bound).max().item():.3e}"


# ------------------------------------------------------------------- CPU
SCALINGS = [
    (None, dict()),
    ({"kind": "linear", "factor": 4.0}, dict(kind="linear", factor=4.0)),
    ({"kind": "ntk", "factor": 8.0}, dict(kind="ntk", factor=8.0)),
    ({"kind": "by_parts", "factor": 8.0, "original": 4096},
     dict(kind="by_parts", factor=8.0, original=4096)),
    ({"kind": "by_parts", "factor": 2.0, "original": 300, "low": 0.5, "high": 4.0},
     dict(kind="by_parts", factor=2.0, original=300, low=0.5, high=4.0)),
    ({"kind": "yarn", "factor": 16.0, "original": 8192},
     dict(kind="yarn", factor=16.0, original=8192)),
]


@pytest.mark.parametrize("dim", [2, 4, 20, 64, 128, 256])
@pytest.mark.parametrize("scaling,kw", SCALINGS)
def test_frequencies(built, dim, scaling, kw):
    if dim == 2 and kw.get("kind") == "ntk":
        with pytest.raises(binding.MbertAttnError):
            binding.Rotary(dim, scaling=scaling)
        return
    r = binding.Rotary(dim, base=160000.0, scaling=scaling)
    f, amp = freqs(dim, 160000.0, **kw)
    assert r.dim == dim and len(r.frequencies) == dim // 2
    assert r.amplitude == pytest.approx(amp, rel=1e-15)
    for a, b in zip(r.frequencies, f):
        assert a == pytest.approx(b, rel=1e-13)


def test_rotary_refusals_without_device(built):
    for bad in (dict(dim=3), dict(dim=-2), dict(dim=258), dict(dim=64, base=1.0),
                dict(dim=64, base=float("nan")), dict(dim=64, base=float("inf"))):
        with pytest.raises(binding.MbertAttnError):
            binding.Rotary(**bad)
    for sc in ({"kind": "linear"}, {"kind": "spline", "factor": 2}, {"factor": 2.0},
               {"kind": "yarn", "factor": 2.0}, {"kind": "linear", "factor": 2.0, "original": 1},
               {"kind": "yarn", "factor": 2.0, "original": 64, "amplitude": 0}):
        with pytest.raises(ValueError):
            binding.Rotary(64, scaling=sc)
    for sc in ({"kind": "linear", "factor": 0.0}, {"kind": "linear", "factor": float("nan")},
               {"kind": "ntk", "factor": 0.5}, {"kind": "yarn", "factor": 2.0, "original": 0},
               {"kind": "by_parts", "factor": 2.0, "original": 64, "low": 4.0, "high": 4.0}):
        with pytest.raises(binding.MbertAttnError):
            binding.Rotary(64, scaling=sc)
    with pytest.raises(ValueError):
        binding.Rotary(64, layout="quarter")
    lib = binding.load_library()
    spec = binding.RotarySpec()
    assert lib.mbert_attn_rotary_init(None, 64, 0, 1e4, None) == -1
    assert lib.mbert_attn_rotary_init(ctypes.byref(spec), 64, 2, 1e4, None) == -1
    x = binding.Heads()
    assert lib.mbert_attn_rotary(None, ctypes.byref(x), 1, 64, 0, ctypes.byref(spec), None, 0, None,
                                 0, 0, None) == -1
    assert lib.mbert_attn_qk_norm_rotary(None, None, None, 1, 64, 0, 1, 0.0, None, None, 0, None, 0,
                                         None) == -1
    with pytest.raises(ValueError):
        binding.rotary(torch.zeros(1, 1, 64), binding.Rotary(64), torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        binding.qk_norm_rotary(None, None, None, None)


# ------------------------------------------------------------------- GPU
def rnd(*shape, seed=0, dtype="bf16", scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(TYPES[dtype])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("T,H,D,R", [
    (1, 1, 64, 64), (1, 12, 64, 64), (3, 1, 128, 64), (33, 12, 64, 64), (130, 7, 80, 20),
    (17, 3, 96, 24), (9, 5, 256, 256), (257, 2, 256, 64), (5, 2, 6, 2), (31, 33, 10, 10),
    (700, 1, 64, 32), (4, 40, 128, 128)])
def test_rotary(built, T, H, D, R, layout, dtype):
    x = rnd(T, H, D, seed=T + D, dtype=dtype).cuda()
    g = torch.Generator().manual_seed(R)
    pos = torch.randint(-5000, 200000, (T,), generator=g)
    f, amp = freqs(R, 160000.0, "yarn", 4.0, 8192)
    rope = binding.Rotary(R, 160000.0, layout, {"kind": "yarn", "factor": 4.0, "original": 8192})
    ref, tol = reference(x, pos, f, amp, layout)
    p32 = pos.to(torch.int32).cuda()
    got = binding.rotary(x, rope, positions=p32)
    check_typed(got, ref, tol)
    assert torch.equal(binding.rotary(x, rope, positions=pos.cuda()), got)      # int64
    back, btol = reference(x, pos, f, amp, layout, inverse=True)
    check_typed(binding.rotary(x, rope, positions=p32, inverse=True), back, btol)
    mine = x.clone()
    assert binding.rotary(mine, rope, positions=p32, out=mine) is mine          # in place
    assert torch.equal(mine, got)


@pytest.mark.gpu
def test_rotary_inverse_is_the_gradient(built):
    """<R x, g> differentiated by x is R^T g: the inverse call, against the
    formula's differences in 64 bits."""
    x, g = rnd(5, 3, 64, seed=1, dtype="f32"), rnd(5, 3, 64, seed=2, dtype="f32")
    pos = torch.tensor([0, 1, 77, 8191, 100000])
    f, amp = freqs(32, 10000.0)
    rope = binding.Rotary(32, layout="interleaved")
    grad = binding.rotary(g.cuda(), rope, positions=pos.cuda(), inverse=True).double().cpu()
    h = 1e-3
    for t, hd, d in [(0, 0, 0), (1, 2, 1), (2, 1, 31), (3, 0, 30), (4, 2, 7), (4, 1, 50)]:
        e = torch.zeros_like(x).double()
        e[t, hd, d] = h
        up = (reference(x.double() + e, pos, f, amp, "interleaved")[0] * g.double()).sum()
        dn = (reference(x.double() - e, pos, f, amp, "interleaved")[0] * g.double()).sum()
        # the function is linear: the difference quotient is exact up to 1e-12
        assert abs((up - dn).item() / (2 * h) - grad[t, hd, d].item()) < 1e-5


@pytest.mark.gpu
@pytest.mark.parametrize("pos", [0, 1, -1, 2 ** 31 - 1, -2 ** 31, 2 ** 40 + 12345])
def test_rotary_far_positions(built, pos):
    """The turns of any position are exact modulo one: in 64 bits the product
    pos * f is off by 2^-53 of itself, so the far ones are compared with
    integer arithmetic on the same double frequencies."""
    from fractions import Fraction
    f, _ = freqs(64, 160000.0)
    two_pi = Fraction(6283185307179586476925286766559005768394338798750211641949889, 10 ** 60)
    ang = []
    for w in f:
        turns = Fraction(w) * pos / two_pi
        ang.append(float((turns - math.floor(turns)) * two_pi))
    x = rnd(1, 4, 64, seed=9, dtype="f32")
    a = torch.tensor(ang, dtype=torch.float64)
    lo, hi = x.double()[..., :32], x.double()[..., 32:]
    ref = torch.cat([lo * a.cos() - hi * a.sin(), hi * a.cos() + lo * a.sin()], -1)
    got = binding.rotary(x.cuda(), binding.Rotary(64, 160000.0),
                         positions=torch.tensor([pos], dtype=torch.int64).cuda())
    # w / 2 pi is a double: its last bits count pos times
    tol = (18 * U + abs(pos) * 2.0 ** -52 * 0.5) * (lo.abs() + hi.abs())
    check(got, ref, torch.cat([tol, tol], -1))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("norm", ["rms", "layer"])
@pytest.mark.parametrize("T,Hq,Hk,D,R,layout", [
    (1, 12, 12, 64, 64, "half"), (50, 12, 12, 64, 64, "half"), (3, 32, 4, 128, 96, "interleaved"),
    (129, 3, 1, 80, 40, "half"), (11, 2, 2, 256, 0, "half"), (1000, 1, 5, 64, 16, "interleaved"),
    (7, 4, 2, 14, 6, "half"), (2, 1, 1, 2, 2, "interleaved")])
def test_qk_norm_rotary(built, T, Hq, Hk, D, R, layout, norm, dtype):
    rows = rnd(T, Hq + 2 * Hk, D, seed=T + D, dtype=dtype, scale=1.5).cuda()
    q, k = rows[:, :Hq], rows[:, Hq:Hq + Hk]
    wq = (1 + 0.2 * rnd(D, seed=3, dtype="f32")).to(TYPES[dtype]).cuda()
    wk = (1 + 0.2 * rnd(D, seed=4, dtype="f32")).to(TYPES[dtype]).cuda()
    pos = torch.arange(T) * 37 % 9001
    f, amp = freqs(R, 10000.0)
    rope = binding.Rotary(R, layout=layout) if R else None
    kw = dict(rope=rope, positions=pos.to(torch.int32).cuda() if R else None, norm=norm, eps=1e-5)
    gq, gk = binding.qk_norm_rotary(q, k, wq, wk, **kw)
    for got, x, w in ((gq, q, wq), (gk, k, wk)):
        check_typed(got, *reference(x, pos, f, amp, layout, norm, w, 1e-5))
    # one tensor alone, and both in place among the fused rows
    only, none = binding.qk_norm_rotary(q, None, wq, None, **kw)
    assert none is None and torch.equal(only, gq)
    none, only = binding.qk_norm_rotary(None, k, None, wk, **kw)
    assert none is None and torch.equal(only, gk)
    before = rows.clone()
    oq, ok = binding.qk_norm_rotary(q, k, wq, wk, q_out=q, k_out=k, **kw)
    assert torch.equal(oq, gq) and torch.equal(ok, gk)
    assert torch.equal(rows[:, Hq + Hk:], before[:, Hq + Hk:])      # V as it was


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("T,H,D,R", [
    (65, 1, 2, 2), (192, 1, 16, 16), (200, 1, 16, 4), (193, 2, 4, 2), (300, 1, 8, 8), (5003, 2, 16, 16),
    (1000, 1, 32, 32), (97, 1, 32, 6), (30000, 1, 2, 2)])
def test_small_heads(built, T, H, D, R, dtype):
    """One or two heads of a few numbers: a block has room for more rows side by
    side than it keeps positions for."""
    x = rnd(T, H, D, seed=T + D, dtype=dtype).cuda()
    pos = torch.arange(T) * 53 % 7919
    f, amp = freqs(R, 10000.0)
    rope = binding.Rotary(R)
    p32 = pos.to(torch.int32).cuda()
    check_typed(binding.rotary(x, rope, positions=p32), *reference(x, pos, f, amp, "half"))
    w = (1 + 0.2 * rnd(D, seed=3, dtype="f32")).to(TYPES[dtype]).cuda()
    got, _ = binding.qk_norm_rotary(x, None, w, None, rope, p32, eps=1e-2)
    check_typed(got, *reference(x, pos, f, amp, "half", "rms", w, 1e-2))


@pytest.mark.gpu
@pytest.mark.parametrize("lens", [[1], [5, 0, 1, 300], [0, 0, 7], [1] * 70, [129, 64, 1000]])
@pytest.mark.parametrize("behind", [0, 13])
def test_positions_from_cu_seqlens(built, lens, behind):
    n = sum(lens)
    x = rnd(n + behind, 12, 64, seed=n).cuda()
    cu = torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32).cuda()
    pos = torch.cat([torch.arange(v) for v in lens])
    f, amp = freqs(64, 10000.0)
    out = torch.full_like(x, 7.0)
    binding.rotary(x, binding.Rotary(64), cu_seqlens=cu, out=out)
    check_typed(out[:n], *reference(x[:n], pos, f, amp, "half"))
    assert (out[n:] == 7.0).all()           # rows behind the last sequence
    h = binding._default(x.device)
    assert h.get_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("cu", [[1, 4, 10], [0, 8, 5, 10], [0, 4, 11]])
def test_bad_cu_seqlens_is_reported(built, cu):
    x = rnd(10, 2, 64).cuda()
    h = binding._default(x.device)
    binding.rotary(x, binding.Rotary(64), cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda())
    assert h.get_error() == -4 and h.get_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strides_and_alignment(built, dtype):
    """Heads before rows, odd pitches, addresses off the 16-byte grid, a
    broadcast input; every form equals the contiguous call's result."""
    T, H, D = 37, 6, 64
    base = rnd(T, H, D, seed=5, dtype=dtype).cuda()
    pos = torch.arange(T, dtype=torch.int32).cuda() * 11
    rope = binding.Rotary(32, layout="interleaved")
    want = binding.rotary(base, rope, positions=pos)
    hm = base.transpose(0, 1).contiguous().transpose(0, 1)              # [H, T, D] storage
    out = torch.empty(H, T, D, dtype=base.dtype, device="cuda").transpose(0, 1)
    assert torch.equal(binding.rotary(hm, rope, positions=pos, out=out), want)
    for pad in (1, 2, 4, 8):
        store = torch.zeros(T, H * D + pad + 1, dtype=base.dtype, device="cuda")
        view = store[:, pad:pad + H * D].unflatten(1, (H, D))
        view.copy_(base)
        assert torch.equal(binding.rotary(view, rope, positions=pos), want)
        assert torch.equal(binding.rotary(view, rope, positions=pos, out=view), want)
        assert (store[:, :pad] == 0).all() and (store[:, pad + H * D:] == 0).all()
    one = base[:, :1].expand(T, H, D)
    assert torch.equal(binding.rotary(one, rope, positions=pos),
                       want[:, :1].expand(T, H, D))
    # another column block of the same rows is a fair place for the result
    two = torch.cat([base, torch.zeros_like(base)], 1)
    binding.rotary(two[:, :H], rope, positions=pos, out=two[:, H:])
    assert torch.equal(two[:, H:], want) and torch.equal(two[:, :H], base)


@pytest.mark.gpu
def test_extreme_values(built):
    """Infinities and NaN stay in their own pair (rotation) or head (norm);
    a head of zeros stays zero; T = 0 is a no-op."""
    x = rnd(4, 2, 64, dtype="f32").cuda()
    x[1, 0, 3] = math.inf
    x[2, 1, 40] = math.nan
    pos = torch.full((4,), 5, dtype=torch.int32).cuda()
    y = binding.rotary(x, binding.Rotary(64), positions=pos)
    bad = ~torch.isfinite(y)
    want = torch.zeros_like(bad)
    want[1, 0, 3] = want[1, 0, 35] = want[2, 1, 8] = want[2, 1, 40] = True
    assert torch.equal(bad, want)
    x[3, 1] = 0
    w = torch.ones(64, device="cuda")
    q, _ = binding.qk_norm_rotary(x, None, w, None, binding.Rotary(64), pos)
    assert not torch.isfinite(q[2, 1]).any() and torch.isfinite(q[[0, 3]]).all()
    assert (q[3, 1] == 0).all()
    e = torch.empty(0, 2, 64, device="cuda")
    assert binding.rotary(e, binding.Rotary(64), positions=torch.empty(0, dtype=torch.int32, device="cuda")).shape == e.shape


@pytest.mark.gpu
def test_streams_and_graph(built):
    x = rnd(300, 12, 64, seed=8).cuda()
    w = (1 + 0.1 * rnd(64, seed=9, dtype="f32")).bfloat16().cuda()
    cu = torch.tensor([0, 100, 300], dtype=torch.int32).cuda()
    rope = binding.Rotary(64, 160000.0)
    want = binding.qk_norm_rotary(x, x, w, w, rope, cu_seqlens=cu)
    torch.cuda.synchronize()
    outs = []
    for _ in range(2):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            outs.append(binding.qk_norm_rotary(x, x, w, w, rope, cu_seqlens=cu))
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o[0], want[0]) and torch.equal(o[1], want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = binding.rotary(x, rope, cu_seqlens=cu)
    x.copy_(rnd(300, 12, 64, seed=10))
    cu.copy_(torch.tensor([0, 7, 250], dtype=torch.int32))
    y.fill_(3.0)
    g.replay()
    torch.cuda.synchronize()
    ref = torch.full_like(x, 3.0)
    binding.rotary(x, rope, cu_seqlens=cu, out=ref)
    assert torch.equal(y, ref) and (y[250:] == 3.0).all()


@pytest.mark.gpu
def test_refusals(built):
    x = rnd(6, 4, 64).cuda()
    p = torch.arange(6, dtype=torch.int32).cuda()
    r = binding.Rotary(64)
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(TypeError):
        binding.rotary(x.double(), r, positions=p)
    with pytest.raises(TypeError):
        binding.rotary(x[0], r, positions=p)
    with pytest.raises(TypeError):
        binding.rotary(x, r, positions=p[:5])
    with pytest.raises(TypeError):
        binding.rotary(x, r, positions=p.float())
    with pytest.raises(ValueError):
        binding.rotary(x, r)
    with pytest.raises(ValueError):
        binding.rotary(x, r, positions=p, cu_seqlens=p)
    with pytest.raises(ValueError):
        binding.rotary(x.transpose(1, 2), r, positions=p)
    with pytest.raises(binding.MbertAttnError):
        binding.rotary(x, binding.Rotary(128), positions=p)             # wider than the head
    with pytest.raises(binding.MbertAttnError):
        binding.rotary(x[..., :63], binding.Rotary(62), positions=p)    # odd head
    with pytest.raises(TypeError):
        binding.rotary(x, r, positions=p, out=x[:5])
    with pytest.raises(binding.MbertAttnError):                         # shifted over itself
        flat = torch.zeros(7, 4, 64, dtype=x.dtype, device="cuda")
        binding.rotary(flat[:6], r, positions=p, out=flat[1:])
    with pytest.raises(binding.MbertAttnError):                         # result with shared elements
        binding.rotary(x, r, positions=p, out=x[:, :1].expand(6, 4, 64))
    with pytest.raises(ValueError):
        binding.qk_norm_rotary(x, x, w, w, r, p, norm="max")
    with pytest.raises(TypeError):
        binding.qk_norm_rotary(x, x[:5], w, w, r, p)
    with pytest.raises(TypeError):
        binding.qk_norm_rotary(x, x, w, None, r, p)
    with pytest.raises(ValueError):
        binding.qk_norm_rotary(x, x, w, w, positions=p)
    with pytest.raises(binding.MbertAttnError):
        binding.qk_norm_rotary(x, x, w, w, r, p, eps=-1.0)
    with pytest.raises(binding.MbertAttnError):                         # both results in one place
        o = torch.empty_like(x)
        binding.qk_norm_rotary(x, x, w, w, r, p, q_out=o, k_out=o)
    with pytest.raises(binding.MbertAttnError):                         # k read while q is written there
        binding.qk_norm_rotary(x, x, w, w, r, p, q_out=x)
    assert binding._default(x.device).get_error() == 0


@pytest.mark.gpu
def test_extents_beyond_any_memory(built):
    """Strides whose extents would not fit 64 bits are refused on the host."""
    import ctypes
    lib = binding.load_library()
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    out, p = torch.empty_like(x), torch.zeros(4, dtype=torch.int32, device="cuda")
    rope = binding.Rotary(64)
    h = binding._default(x.device).handle
    for tokens, strides in ((2 ** 30, (1 << 40, 64, 128, 64)), (2 ** 30, (128, 64, 1 << 40, 64)),
                            (4, (-128, 64, 128, 64)), (4, (1 << 41, 64, 128, 64))):
        heads = binding.Heads(x.data_ptr(), out.data_ptr(), None, 2, *strides)
        assert lib.mbert_attn_rotary(h, ctypes.byref(heads), tokens, 64, 0, rope._ref, p.data_ptr(), 32, None, 0,
                                     0, None) == -1
