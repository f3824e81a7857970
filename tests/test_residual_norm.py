"""The norms around a block with the gate and the residual (binding.residual_norm)
against their formulas in 64 bits.

Tolerance per element, from the arithmetic, with u_t = eps_t / 2 of the type, u =
2^-24 and a row of D numbers whose inputs are off by dv:
  - mean: dm = max |dv| + 2 u (D + 3) mean|v|;  a difference from it d = v - mean:
      dd = dv + dm + u |d|   (RMS: dd = dv)
  - the sum of squares is off by a part 2 u (D + 3), and by dd, so that the factor
      r = 1 / sqrt(var + eps) is off by a part  dr = u (D + 3) + 4 u + rms(dd) / sqrt(var + eps)
      (rsqrt 2 u, scaling of eps 2 u; |rms(d + dd) - rms(d)| <= rms(dd))
  - y = d r w + b:  dy = |w| r dd + |d r w| (dr + 3 u) + u |y|
  - h = alpha x + g P:  dh = |g| dP + 2 u (|alpha x| + |g P|)
  - the output's rounding:  u_t |out|
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


def norm(v, dv, w, b, kind, eps):
    D = v.shape[1]
    if kind == "layer":
        mean = v.mean(1, keepdim=True)
        d = v - mean
        dd = dv + dv.amax(1, keepdim=True) + 2 * U * (D + 3) * v.abs().mean(1, keepdim=True) + U * d.abs()
    else:
        d, dd = v, dv
    s = (d * d).mean(1, keepdim=True) + eps
    r = s ** -0.5
    dr = U * (D + 3) + 4 * U + (dd * dd).mean(1, keepdim=True) ** 0.5 * r
    wd = w.double()
    y = d * r * wd
    dy = wd.abs() * r * dd + y.abs() * (dr + 3 * U)
    if b is not None:
        y = y + b.double()
    return y, dy + U * y.abs()


def reference(x, branch, w, b, aw, ab, gate, kind, scale, eps):
    """fp64: -> (h, its tolerance before rounding, y, its tolerance); gate [T, D] or [D]."""
    h, dh = x.double(), torch.zeros(x.shape, dtype=torch.float64)
    if branch is not None:
        p, dp = branch.double(), dh
        if aw is not None:
            p, dp = norm(p, dp, aw, ab, kind, eps)
        if gate is not None:
            g = gate.double()
            p, dp = p * g, dp * g.abs()
        h, dh = scale * h + p, dp + 2 * U * ((scale * h).abs() + p.abs())
    y = dy = None
    if w is not None:
        y, dy = norm(h, dh, w, b, kind, eps)
    return h, dh, y, dy


def check(got, ref, tol, what=""):
    f = torch.finfo(got.dtype)
    tol = tol + f.eps / 2 * (ref.abs() + tol) + f.smallest_normal * f.eps
    g = got.double().cpu()
    assert torch.isfinite(g).all()
    err = (g - ref).abs()
    bad = err > tol
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}, "
                           f"max err {err.max().item():.3e} against {tol.max().item():.3e}")


def rnd(*shape, seed, dtype="bf16", sc=1.0, at=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * sc + at).to(TYPES[dtype])


def make(T, D, dtype, seed=0):
    return dict(x=rnd(T, D, seed=seed, dtype=dtype, sc=2.0), branch=rnd(T, D, seed=seed + 1, dtype=dtype, at=0.3),
                w=rnd(D, seed=seed + 2, dtype=dtype, sc=0.2, at=1.0), b=rnd(D, seed=seed + 3, dtype=dtype, sc=0.2),
                aw=rnd(D, seed=seed + 4, dtype=dtype, sc=0.2, at=1.0), ab=rnd(D, seed=seed + 5, dtype=dtype, sc=0.2))


def cuda(t):
    return None if t is None else t.cuda()


def err0():
    torch.cuda.synchronize()
    assert binding._default(torch.device("cuda", torch.cuda.current_device())).get_error() == 0


def run(x, branch=None, w=None, b=None, aw=None, ab=None, gate=None, kind="layer", scale=1.0, eps=1e-5):
    h, y = binding.residual_norm(cuda(x), cuda(branch), cuda(w), cuda(b), cuda(aw), cuda(ab), cuda(gate), None, kind,
                                 scale, eps)
    err0()
    rh, dh, ry, dy = reference(x, branch, w, b, aw, ab, gate, kind, scale, eps)
    if branch is not None:
        check(h, rh, dh, "h")
    if w is not None:
        check(y, ry, dy, "y")
    else:
        assert y is None
    return h, y


# ------------------------------------------------------------------- CPU
def test_host_refusals_without_device(built):
    lib = binding.load_library()
    a = binding.ResidualNormArgs()
    assert lib.mbert_attn_residual_norm(None, ctypes.byref(a), None) == -1
    with pytest.raises(ValueError):
        binding.residual_norm(torch.zeros(2, 8), torch.zeros(2, 8), torch.ones(8))


# ------------------------------------------------------------------- GPU
WIDTHS = [1, 2, 7, 8, 9, 24, 64, 65, 100, 256, 264, 500, 768, 777, 1000, 1024, 1032, 1152, 2048, 2304, 4100, 8192,
          12000, 16383, 16384]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("D", WIDTHS)
def test_widths(built, D, kind, dtype):
    """Every number of lanes, vectors and warps, with all parts of the call."""
    eps = 1e-3 if D == 1 else 1e-5
    for T in (1, 37):
        m = make(T, D, dtype, seed=D)
        run(m["x"], m["branch"], m["w"], m["b"], m["aw"], m["ab"], rnd(T, D, seed=9, dtype=dtype), kind, 0.7, eps)
        run(m["x"], m["branch"], m["w"], kind=kind, eps=eps)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("D", [1280, 1535, 1536, 1544, 2048, 2056, 2560, 4088, 4096, 6152, 8192, 8200])
def test_wide_rows_by_fewer_warps(built, D, dtype):
    """Rows enough for every SM several times over, in crews of every size."""
    T = 650
    m = make(T, D, dtype, seed=D + 2)
    # scaled a second time (f16 holds 65504, twice 2^12 times 7 deviations are less)
    m["x"][::50] *= 2.0 ** 12 if dtype == "f16" else 2.0 ** 66
    m["branch"][7::50] = 0
    run(m["x"], m["branch"], m["w"], m["b"], m["aw"], m["ab"], rnd(T, D, seed=9, dtype=dtype), "layer", 0.7)
    run(m["x"], m["branch"], m["w"], aw=m["aw"], gate=rnd(D, seed=9, dtype=dtype), kind="rms")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("D", [64, 768, 1001, 2304])
def test_parts(built, D, dtype):
    T = 300
    m = make(T, D, dtype, seed=D + 1)
    x, branch, w, b, aw, ab = (m[k] for k in ("x", "branch", "w", "b", "aw", "ab"))
    run(x, None, w)
    run(x, None, w, b, kind="rms", eps=1e-12)
    run(x, branch)                                          # the residual alone
    run(x, branch, aw=aw, scale=-2.0)                       # no norm behind it
    run(x, branch, w, gate=rnd(D, seed=8, dtype=dtype))
    run(x, branch, w, b, aw, None, rnd(T, D, seed=9, dtype=dtype), "rms", 0.0)
    run(x, branch, w, None, aw, ab, rnd(D, seed=8, dtype=dtype), eps=0.0)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [768, 1001])
@pytest.mark.parametrize("lens", [[5], [0, 1, 0, 200, 3], [1] * 300, [0, 0, 4]])
def test_sequence_gates(built, lens, D, dtype):
    """Rows behind the last sequence keep what they held; nothing of them counts."""
    n, T, behind = len(lens), sum(lens), 3
    m = make(T + behind, D, dtype, seed=n)
    gate = rnd(n, D, seed=5, dtype=dtype)
    o = [0]
    for k in lens:
        o.append(o[-1] + k)
    rows = torch.repeat_interleave(torch.arange(n), torch.tensor(lens))
    x, branch = m["x"].cuda(), m["branch"].cuda()
    x[T:], branch[T:] = math.nan, math.inf
    h, y = torch.full_like(x, 3.0), torch.full_like(x, 4.0)
    binding.residual_norm(x, branch, m["w"].cuda(), None, m["aw"].cuda(), None, gate.cuda(),
                          torch.tensor(o, dtype=torch.int32).cuda(), h_out=h, y_out=y)
    err0()
    assert (h[T:] == 3.0).all() and (y[T:] == 4.0).all()
    rh, dh, ry, dy = reference(m["x"][:T], m["branch"][:T], m["w"], None, m["aw"], None, gate[rows], "layer", 1.0, 1e-5)
    check(h[:T], rh, dh, "h")
    check(y[:T], ry, dy, "y")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("D", [8, 100, 768, 4096, 16384])
@pytest.mark.parametrize("exponent,eps", [(59, 1e-6), (62, 0.0), (64, 1e-5), (90, 1.0), (122, 1e-6), (125, 0.0),
                                          (-59, 0.0), (-75, 1e-30), (-100, 0.0), (-120, 1e-37), (-60, 1e-6)])
def test_any_magnitude(built, exponent, eps, D, kind, dtype):
    """Numbers whose squares fp32 does not hold, at both ends, beside ordinary rows."""
    T = 6
    x = rnd(T, D, seed=D, dtype="f32").clamp(-3.5, 3.5)
    x[1:4] = (x[1:4].double() * 2.0 ** exponent).float()
    x = x.to(TYPES[dtype])
    w = rnd(D, seed=3, dtype=dtype, sc=0.2, at=1.0)
    _, y = run(x, None, w, kind=kind, eps=eps)
    # ordinary rows keep their bits beside the others
    z = x.clone()
    z[1:4] = x[0]
    _, want = binding.residual_norm(z.cuda(), None, w.cuda(), norm=kind, eps=eps)
    assert torch.equal(y[4:], want[4:]) and torch.equal(y[0], want[0])
    run(torch.zeros_like(x), x, None, aw=w, kind=kind, eps=eps)


@pytest.mark.gpu
def test_ends_of_the_range(built):
    """Differences from the mean beyond fp32's largest number, and a mean far from 0."""
    D = 64
    top = 3.0e38
    x = torch.full((2, D), top)
    x[0, ::2] = -top
    x[1, 5] = -top
    run(x, None, torch.ones(D), eps=0.0)
    x = rnd(3, 768, seed=1, dtype="f32", at=1000.0)
    run(x, None, torch.ones(768))


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 768, 2304])
def test_rows_do_not_meet(built, D):
    m = make(50, D, "bf16", seed=2)
    args = lambda x, branch: (x.cuda(), branch.cuda(), m["w"].cuda(), None, m["aw"].cuda())
    wh, wy = binding.residual_norm(*args(m["x"], m["branch"]))
    x, branch = m["x"].clone(), m["branch"].clone()
    x[7, 3], branch[20, 5], branch[21] = math.nan, math.inf, math.nan
    h, y = binding.residual_norm(*args(x, branch))
    keep = torch.ones(50, dtype=torch.bool, device="cuda")
    keep[[7, 20, 21]] = False
    assert torch.equal(h[keep], wh[keep]) and torch.equal(y[keep], wy[keep])
    assert y[7].isnan().all() and y[21].isnan().all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(TYPES))
def test_strided_in_place_graph(built, dtype):
    """Strided and unaligned rows to the last bit as near as the order of sums allows,
    in place, and captured."""
    T, D = 70, 768
    m = make(T, D, dtype, seed=3)
    x, branch, w, aw = (m[k].cuda() for k in ("x", "branch", "w", "aw"))
    gate = rnd(T, D, seed=4, dtype=dtype).cuda()
    call = lambda x, branch, gate, **kw: binding.residual_norm(x, branch, w, None, aw, None, gate, **kw)
    wh, wy = call(x, branch, gate)
    ref = reference(m["x"], m["branch"], m["w"], None, m["aw"], None, gate.cpu(), "layer", 1.0, 1e-5)

    def view(t, pitch, start):
        buf = torch.full((T * pitch + start + 8,), math.nan, dtype=t.dtype, device="cuda")
        v = buf[start:start + T * pitch].view(T, pitch)[:, :D]
        v.copy_(t)
        return v, buf

    for pitch, start in ((776, 0), (784, 8), (769, 1), (800, 3)):
        ho, hb = view(x, pitch, start)
        yo, yb = view(x, pitch, start)
        call(view(x, pitch, start)[0], view(branch, pitch, start)[0], view(gate, pitch, start)[0], h_out=ho, y_out=yo)
        err0()
        check(ho, ref[0], ref[1], "h")
        check(yo, ref[2], ref[3], "y")
        if pitch % 8 == 0 and start % 8 == 0:
            assert torch.equal(ho, wh) and torch.equal(yo, wy)
        ho.fill_(math.nan)
        yo.fill_(math.nan)
        assert hb.isnan().all() and yb.isnan().all()
    for hi, yi in ((0, 1), (1, 0), (0, None), (None, 0)):
        a, b = x.clone(), branch.clone()
        h, y = call(a, b, gate, h_out=None if hi is None else (a, b)[hi], y_out=None if yi is None else (a, b)[yi])
        assert torch.equal(h, wh) and torch.equal(y, wy)
    a, b = x.clone(), branch.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h, y = call(a, b, gate, h_out=a)
    for _ in range(2):
        a.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(h, wh) and torch.equal(y, wy) and h is a


@pytest.mark.gpu
def test_many_rows(built):
    """More rows than are in flight at once, every row the same as alone."""
    for D, T in ((8, 100001), (768, 20011), (2048, 9001)):
        x, branch = rnd(T, D, seed=1).cuda(), rnd(T, D, seed=2).cuda()
        w = rnd(D, seed=3).cuda()
        h, y = binding.residual_norm(x, branch, w, norm="rms")
        for t in (0, 1, T // 2, T - 2, T - 1):
            a, b = binding.residual_norm(x[t:t + 1], branch[t:t + 1], w, norm="rms")
            assert torch.equal(a[0], h[t]) and torch.equal(b[0], y[t])
        z = x.double() + branch.double()
        want = z * (z.square().mean(1, keepdim=True) + 1e-5).rsqrt() * w.double()
        assert ((y.double() - want).abs() <= 2.0 ** -8 * 1.01 * want.abs() + 1e-6).all()


@pytest.mark.gpu
def test_bad_sequences_and_refusals(built):
    T, D = 10, 64
    x, br, w = rnd(T, D, seed=1).cuda(), rnd(T, D, seed=2).cuda(), rnd(D, seed=3).cuda()
    gate = rnd(2, D, seed=4).cuda()
    dev = x.device
    for bad in ([1, 4, 10], [0, 4, 11], [0, 5, 4], [0, -1, 3]):
        h, y = torch.full_like(x, 3.0), torch.full_like(x, 3.0)
        binding.residual_norm(x, br, w, gate=gate, cu_seqlens=torch.tensor(bad, dtype=torch.int32).cuda(), h_out=h,
                              y_out=y)
        torch.cuda.synchronize()
        assert binding._default(dev).get_error() == -4 and (h == 3.0).all() and (y == 3.0).all()
    call = binding.residual_norm
    cu = torch.tensor([0, 4, 10], dtype=torch.int32).cuda()
    for kw in (dict(weight=w, norm="batch"), dict(), dict(branch=br, bias=w), dict(branch=br, branch_bias=w),
               dict(weight=w, gate=w), dict(weight=w, residual_scale=2.0), dict(weight=w, h_out=x.clone()),
               dict(branch=br, y_out=x.clone()), dict(branch=br, cu_seqlens=cu), dict(weight=w, branch_weight=w),
               dict(branch=br, gate=gate, cu_seqlens=cu[:1])):
        with pytest.raises(ValueError):
            call(x, **kw)
    for kw in (dict(branch=br.float()), dict(branch=br[:9]), dict(weight=w[:63]), dict(weight=w.float()),
               dict(branch=br, gate=gate), dict(branch=br, gate=w[None]), dict(branch=br, gate=gate, cu_seqlens=cu.long()),
               dict(branch=br.cpu()), dict(branch=br, h_out=x.float())):
        with pytest.raises(TypeError):
            call(x, **kw)
    with pytest.raises(ValueError):
        call(x.t().contiguous().t(), br)
    big = torch.zeros(2, 16385, dtype=x.dtype, device="cuda")
    wide = torch.zeros(T + 1, D, dtype=x.dtype, device="cuda")
    for fn in (lambda: call(x, None, w, eps=-1.0), lambda: call(x, None, w, eps=2.0), lambda: call(x, None, w, eps=math.nan),
               lambda: call(x, br, w, residual_scale=1e39), lambda: call(x, br, w, residual_scale=math.inf),
               lambda: call(big, big), lambda: call(x[:1].expand(T, D), br),
               lambda: call(wide[:T], br, w, h_out=wide[1:]), lambda: call(x, br, w, h_out=wide[:T], y_out=wide[:T]),
               lambda: call(x, br, w, gate=wide[:T], h_out=wide[:T])):
        with pytest.raises(binding.MbertAttnError):
            fn()
    assert call(x[:0], br[:0], w)[1].shape == (0, D)
    err0()
