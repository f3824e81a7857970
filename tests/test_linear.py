"""Matrix products of any width (binding.linear, binding.expert_linear) against
their formulas in 64 bits.

Tolerance per element, from the arithmetic, with u_t = eps_t / 2 of the type and
u = 2^-24:
  - z, a sum of K exact products and the bias in fp32, taken as truncating:
      dz = 2 u (K + 2) (sum |x||w| + |b|)
  - an activation has a slope of at most 1.13 (gelu 1.129, silu 1.100) and is itself
    evaluated to a part `rel` of its value:  da = 1.13 dz + rel |a|, where
      gelu: polynomial 5.3e-6, exponent up to 47 rounded four times (4 x 2^-19 ln 2
        = 5.3e-6 at most), 2^-22: 2^-16 of it; beyond |z| = 8 the polynomial stands
        still, where the result is below 1e-14 (absolute)
      silu, gelu_tanh: exponents up to 127 with 4 roundings, 127 x 4 u ln 2 = 2.1e-5, with
        ex2, 1 + and rcp 2^-22 each: 2^-15 of it
  - gated:  da |z_u| + (|a| + da) dz_u + 2 u |a z_u|
  - row weight and residual:  2 u (|y| + |residual|) more
  - the output's rounding:  u_t |out|
"""
import ctypes
import math

import pytest
import torch

from encoder_only_transformer_gb300 import binding

U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
REL = {"none": 0.0, "relu": 0.0, "gelu": 2.0 ** -16, "gelu_tanh": 2.0 ** -15, "silu": 2.0 ** -15}


@pytest.fixture(scope="module")
def built():
    import __graft_entry__
    __graft_entry__.build()


def act(z, name):
    if name == "gelu":
        return z * 0.5 * torch.special.erfc(-z / math.sqrt(2.0))
    if name == "gelu_tanh":
        return z * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3))
    if name == "silu":
        return z * torch.sigmoid(z)
    return z.clamp(min=0.0) if name == "relu" else z


def product(x, w, b, activation, gated):
    """fp64: -> (y, tolerance) of act(x w^T + b), [T, N]."""
    K = x.shape[1]
    xd, wd = x.double(), w.double()
    z, m = xd @ wd.T, xd.abs() @ wd.abs().T
    if b is not None:
        z, m = z + b.double(), m + b.double().abs()
    dz = 2 * U * (K + 2) * m
    N = w.shape[0] // 2 if gated else w.shape[0]
    a = act(z[:, :N], activation)
    da = 1.13 * dz[:, :N] + REL[activation] * a.abs() + (1e-13 if activation == "gelu" else 0.0)
    if not gated:
        return a, da
    u, du = z[:, N:], dz[:, N:]
    return a * u, da * u.abs() + (a.abs() + da) * du + 2 * U * (a * u).abs()


def finish(y, t, dtype, row_scale=None, residual=None):
    if row_scale is not None:
        s = row_scale.double()[:, None]
        y, t = y * s, t * s.abs()
    t = t + 2 * U * y.abs()
    if residual is not None:
        y = y + residual.double()
        t = t + 2 * U * (y.abs() + residual.double().abs())
    f = torch.finfo(dtype)
    return y, t + f.eps / 2 * (y.abs() + t) + f.smallest_normal * f.eps


def check(got, ref, tol):
    g = got.double().cpu()
    assert torch.isfinite(g).all()
    err = (g - ref).abs()
    bad = err > tol
    assert not bad.any(), (f"{int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}, "
                           f"max err {err.max().item():.3e} against {tol.max().item():.3e}")


def rnd(*shape, seed, dtype="bf16", sc=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * sc).to(TYPES[dtype])


def strided(t, pitch, start=0):
    """t [T, D] as a view of rows `pitch` apart, NaN around it, on the GPU."""
    buf = torch.full((t.shape[0] * pitch + start + 8,), math.nan, dtype=t.dtype).cuda()
    v = buf[start:start + t.shape[0] * pitch].view(t.shape[0], pitch)[:, :t.shape[1]]
    v.copy_(t)
    return v, buf


def err0():
    torch.cuda.synchronize()
    assert binding._default(torch.device("cuda", torch.cuda.current_device())).get_error() == 0


def run_linear(T, K, N, dtype, activation="none", bias=False, gated=False, residual=False, seed=0, sc=1.0):
    W = 2 * N if gated else N
    x, w = rnd(T, K, seed=seed, dtype=dtype, sc=sc), rnd(W, K, seed=seed + 1, dtype=dtype, sc=K ** -0.5)
    b = rnd(W, seed=seed + 2, dtype=dtype, sc=0.5) if bias else None
    r = rnd(T, N, seed=seed + 3, dtype=dtype) if residual else None
    dev = [None if t is None else t.cuda() for t in (x, w, b, r)]
    got = binding.linear(dev[0], dev[1], dev[2], activation, gated, dev[3])
    err0()
    y, t = product(x, w, b, activation, gated)
    check(got, *finish(y, t, TYPES[dtype], None, r))
    return got, dev


# ------------------------------------------------------------------- CPU
def test_host_refusals_without_device(built):
    lib = binding.load_library()
    a = binding.LinearArgs()
    assert lib.mbert_attn_linear(None, ctypes.byref(a), None) == -1
    assert lib.mbert_attn_linear(None, None, None) == -1
    x, w = torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(8, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        binding.linear(x, w)
    with pytest.raises(ValueError):
        binding.expert_linear(x, w[None], torch.zeros(2, dtype=torch.int32))


def test_argument_structure_matches_the_header(built):
    """Field for field: name order and sizes as include/mbert_attn.h lays them out."""
    assert ctypes.sizeof(binding.LinearArgs) == 5 * 8 + 6 * 8 + 6 * 4 + 2 * 8
    assert ctypes.sizeof(binding.ResidualNormArgs) == 9 * 8 + 6 * 8 + 4 * 4 + 8 + 4 + 4 + 4 + 4
    assert binding.LinearArgs.cu_experts.offset == 112 and binding.ResidualNormArgs.cu_seqlens.offset == 136


# ------------------------------------------------------------------- GPU
@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("T,K,N", [
    (1, 8, 1), (1, 64, 4), (1, 768, 768), (2, 72, 33), (7, 200, 130), (16, 768, 2304), (17, 1152, 500),
    (33, 768, 129), (64, 520, 257), (65, 768, 768), (100, 2048, 384), (128, 264, 1000),     # few rows
    (129, 64, 64), (200, 768, 768), (255, 72, 250), (256, 1000, 256), (257, 768, 513), (300, 8, 1),
    (600, 1152, 768), (1000, 136, 2304), (2500, 64, 1100)])                                 # pairs
def test_sizes(built, T, K, N, dtype):
    run_linear(T, K, N, dtype, seed=T + N)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("activation", ["none", "gelu", "gelu_tanh", "silu", "relu"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("T,K,N", [(3, 328, 70), (24, 768, 1152), (50, 96, 129), (120, 520, 200), (300, 768, 1152),
                                   (1030, 200, 330)])
def test_epilogues(built, T, K, N, gated, activation, dtype):
    """Wide spread of z (both tails of the activations), bias, residual."""
    run_linear(T, K, N, dtype, activation, bias=True, gated=gated, residual=True, seed=N, sc=4.0)


@pytest.mark.gpu
@pytest.mark.parametrize("activation", ["gelu", "gelu_tanh", "silu", "relu", "none"])
@pytest.mark.parametrize("T", [1, 4096])
def test_activations_alone(built, activation, T):
    """An identity weight: act of every finite bf16 number between -200 and 200, and
    of infinities and NaN, by both kernels."""
    bits = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    v = bits[torch.isfinite(bits.float()) & (bits.float().abs() < 200)]
    K = 8 * (-(-v.numel() // (8 * T))) if T > 1 else 40960
    assert T * K >= v.numel() or T == 1
    if T == 1:
        v = v[torch.randperm(v.numel(), generator=torch.Generator().manual_seed(1))[:K]]
    x = torch.zeros(T * K, dtype=torch.bfloat16)
    x[:v.numel()] = v
    if T > 1:
        x = x.view(T, K)
        got = binding.linear(x.cuda(), torch.eye(K, dtype=torch.bfloat16, device="cuda"), activation=activation)
    else:
        # one row times a column: every output is one number of it
        got = binding.linear(torch.ones(1, 8, dtype=torch.bfloat16, device="cuda"),
                             torch.cat([x[:, None], torch.zeros(K, 7, dtype=torch.bfloat16)], 1).cuda().contiguous(),
                             activation=activation)[0]
    err0()
    z = x.double()
    a = act(z, activation)
    # (exponentials below 2^-126 are flushed to 0)
    t = REL[activation] * a.abs() + (1e-13 if activation == "gelu" else 0.0) + 2.0 ** -118
    y, t = finish(a, t, torch.bfloat16)
    check(got, y.view(got.shape), t.view(got.shape))
    odd = torch.tensor([math.inf, -math.inf, math.nan], dtype=torch.bfloat16)
    w = torch.zeros(3, 8, dtype=torch.bfloat16)
    w[:, 0] = odd
    for rows in (1, 300):
        o = binding.linear(torch.eye(8, dtype=torch.bfloat16, device="cuda")[:1].expand(rows, 8).contiguous(), w.cuda(),
                           activation=activation)
        assert (o[:, 0] == math.inf).all() and o[:, 2].isnan().all()
        assert (o[:, 1] == (-math.inf if activation == "none" else 0.0)).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [5, 40, 700])
@pytest.mark.parametrize("gated", [False, True])
def test_strided_and_unaligned(built, T, gated):
    """Rows apart, results and residuals at odd addresses and pitches: the same bits,
    and nothing else is written."""
    K, N = 200, 150
    W = 2 * N if gated else N
    x, w, b, r = rnd(T, K, seed=1), rnd(W, K, seed=2, sc=0.1), rnd(W, seed=3), rnd(T, N, seed=4)
    want = binding.linear(x.cuda(), w.cuda(), b.cuda(), "gelu", gated, r.cuda())
    y, t = product(x, w, b, "gelu", gated)
    check(want, *finish(y, t, torch.bfloat16, None, r))
    xs, ws = strided(x, 208, 8)[0], strided(w, 264, 16)[0]
    bias = strided(b[None], W, 1)[0][0]
    for pitch, start in ((150, 0), (151, 1), (160, 8), (160, 1), (153, 0)):
        rs = strided(r, pitch, start)[0]
        os, buf = strided(torch.zeros(T, N, dtype=torch.bfloat16), pitch, start)
        got = binding.linear(xs, ws, bias, "gelu", gated, rs, out=os)
        err0()
        assert got is os and torch.equal(got, want), (pitch, start)
        os.fill_(math.nan)
        assert buf.isnan().all()
        binding.linear(xs, ws, bias, "gelu", gated, rs, out=rs)      # in place
        assert torch.equal(rs, want), (pitch, start)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [4, 30, 500])
@pytest.mark.parametrize("K", [1, 3, 60, 65, 130, 199])
def test_inner_ends_within_a_vector(built, T, K):
    """Rows padded to whole vectors: what the padding holds does not count."""
    x, w = rnd(T, K, seed=1), rnd(90, K, seed=2)
    pitch = (K + 7) // 8 * 8
    got = binding.linear(strided(x, pitch)[0], strided(w, pitch)[0])
    err0()
    y, t = product(x, w, None, "none", False)
    check(got, *finish(y, t, torch.bfloat16))


@pytest.mark.gpu
@pytest.mark.parametrize("T", [30, 500])
def test_rows_do_not_meet(built, T):
    """A row of infinities and NaN leaves the others as they were."""
    x, w = rnd(T, 136, seed=1).cuda(), rnd(77, 136, seed=2).cuda()
    want = binding.linear(x, w, activation="silu")
    y = x.clone()
    y[T // 2, 5] = math.nan
    y[3] = math.inf
    got = binding.linear(y, w, activation="silu")
    keep = torch.ones(T, dtype=torch.bool)
    keep[T // 2] = keep[3] = False
    assert torch.equal(got[keep.cuda()], want[keep.cuda()]) and got[T // 2].isnan().all()
    z = w.clone()
    z[11] = math.nan
    got = binding.linear(x, z, activation="silu")
    assert got[:, 11].isnan().all()
    got[:, 11] = want[:, 11]
    assert torch.equal(got, want)


@pytest.mark.gpu
def test_exact_integers(built):
    """Small whole numbers: every sum is exact, whatever its order."""
    g = torch.Generator().manual_seed(5)
    for T, K, N in ((9, 1024, 300), (70, 4096, 140), (777, 2048, 520)):
        x = torch.randint(-3, 4, (T, K), generator=g).to(torch.float16)
        w = torch.randint(-1, 2, (N, K), generator=g).to(torch.float16)
        got = binding.linear(x.cuda(), w.cuda())
        assert torch.equal(got.cpu(), (x.double() @ w.double().T).to(torch.float16))


@pytest.mark.gpu
def test_empty_and_wide(built):
    x, w = rnd(0, 64, seed=1).cuda(), rnd(5, 64, seed=2).cuda()
    assert binding.linear(x, w).shape == (0, 5)
    run_linear(3, 16384, 9, "bf16", seed=4)
    run_linear(2, 64, 50368, "f16", bias=True, seed=5)
    run_linear(300, 16, 20001, "bf16", bias=True, seed=6)


GROUPS = [
    [5], [0, 3, 0], [1] * 40, [16, 17, 0, 1, 31], [0, 0, 100, 7, 64, 65, 0], [300], [257, 0, 255, 256, 1],
    [40] * 33 + [0] * 40 + [5, 200], [1000, 3, 0, 500], [7] * 130,
]


def run_experts(sizes, K, N, dtype, activation="none", bias=False, gated=False, scaled=False, seed=0, behind=0,
                wpad=0):
    E, T = len(sizes), sum(sizes)
    W = 2 * N if gated else N
    x, w = rnd(T + behind, K, seed=seed, dtype=dtype), rnd(E, W, K, seed=seed + 1, dtype=dtype, sc=K ** -0.5)
    b = rnd(E, W, seed=seed + 2, dtype=dtype, sc=0.5) if bias else None
    s = torch.rand(T + behind, generator=torch.Generator().manual_seed(seed)) if scaled else None
    x[T:] = math.nan
    o = [0]
    for n in sizes:
        o.append(o[-1] + n)
    wd = w.cuda()
    if wpad:
        wide = torch.full((E, W + 3, K + wpad), math.nan, dtype=w.dtype, device="cuda")
        wide[:, :W, :K] = wd
        wd = wide[:, :W, :K]
    out = torch.full((T + behind, N), 3.0, dtype=TYPES[dtype], device="cuda")
    cu = torch.tensor(o, dtype=torch.int32).cuda()
    args = (x.cuda(), wd, cu, None if b is None else b.cuda(), activation, gated, None if s is None else s.cuda())
    got = binding.expert_linear(*args, out=out)
    err0()
    assert (got[T:] == 3.0).all()
    for e in range(E):
        rows = slice(o[e], o[e + 1])
        y, t = product(x[rows], w[e], None if b is None else b[e], activation, gated)
        check(got[rows], *finish(y, t, TYPES[dtype], None if s is None else s[rows]))
    again = binding.expert_linear(*args, out=torch.full_like(out, 3.0))
    assert torch.equal(again, got)
    return got, args


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("sizes", GROUPS, ids=lambda s: f"{len(s)}x{max(s)}")
def test_experts(built, sizes, dtype):
    run_experts(sizes, 136, 200, dtype, seed=len(sizes), behind=3)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("sizes", GROUPS[3:], ids=lambda s: f"{len(s)}x{max(s)}")
def test_experts_epilogues(built, sizes, dtype):
    run_experts(sizes, 200, 130, dtype, "gelu", bias=True, gated=True, scaled=True, seed=7, wpad=24)
    run_experts(sizes, 72, 33, dtype, "silu", bias=True, scaled=True, seed=8, behind=1)


@pytest.mark.gpu
def test_bad_offsets(built):
    """Reported, nothing written, and the next call is fine."""
    dev = torch.device("cuda", 0)
    for T, E in ((20, 4), (900, 3)):
        x, w = rnd(T, 64, seed=1).cuda(), rnd(E, 40, 64, seed=2).cuda()
        good = [T * i // E for i in range(E + 1)]
        for bad in ([1] + good[1:], good[:-1] + [T + 1], good[:1] + [good[2], good[1]] + good[3:], [0, -1] + good[2:]):
            out = torch.full((T, 40), 3.0, dtype=torch.bfloat16, device="cuda")
            binding.expert_linear(x, w, torch.tensor(bad, dtype=torch.int32).cuda(), out=out)
            torch.cuda.synchronize()
            assert binding._default(dev).get_error() == -4 and (out == 3.0).all()
        binding.expert_linear(x, w, torch.tensor(good, dtype=torch.int32).cuda())
        err0()


@pytest.mark.gpu
def test_refusals(built):
    x, w = rnd(10, 64, seed=1).cuda(), rnd(12, 64, seed=2).cuda()
    cu = torch.tensor([0, 10], dtype=torch.int32).cuda()
    f32 = x.float()
    with pytest.raises(ValueError):
        binding.linear(x, w, activation="swish")
    for a, b in ((x.cpu().cuda()[None], w), (f32, w.float()), (x, w.half()), (x, w[:, :32].contiguous()), (x, w.cpu())):
        with pytest.raises(TypeError):
            binding.linear(a, b)
    with pytest.raises(ValueError):
        binding.linear(x, w[:11], gated=True)
    with pytest.raises(ValueError):
        binding.linear(x.t()[:12].t(), x.t().contiguous().t()[:, :12])       # columns apart
    with pytest.raises(ValueError):
        binding.linear(rnd(10, 63, seed=1).cuda(), rnd(12, 63, seed=1).cuda())   # rows off 16 bytes
    with pytest.raises(binding.MbertAttnError):
        binding.linear(rnd(10 * 64 + 1, seed=1).cuda()[1:].view(10, 64), w)      # the first row off 16 bytes
    with pytest.raises(binding.MbertAttnError):
        binding.linear(x[:1].expand(10, 64), w)                                  # rows that are one
    with pytest.raises(TypeError):
        binding.linear(x, w, bias=torch.zeros(11, dtype=x.dtype, device="cuda"))
    with pytest.raises(TypeError):
        binding.linear(x, w, residual=torch.zeros(10, 11, dtype=x.dtype, device="cuda"))
    with pytest.raises(TypeError):
        binding.linear(x, w, out=torch.zeros(10, 12, device="cuda"))
    sq = rnd(64, 64, seed=3).cuda()
    with pytest.raises(binding.MbertAttnError):
        binding.linear(x, sq, out=x)                                             # out over x
    both = torch.zeros(11, 12, dtype=x.dtype, device="cuda")
    with pytest.raises(binding.MbertAttnError):
        binding.linear(x, w, residual=both[:10], out=both[1:])                   # out over other rows of the residual
    with pytest.raises(TypeError):
        binding.expert_linear(x, w, cu)
    with pytest.raises(TypeError):
        binding.expert_linear(x, w[None], cu.long())
    with pytest.raises(TypeError):
        binding.expert_linear(x, w[None], cu, row_scale=torch.ones(10, dtype=x.dtype, device="cuda"))
    with pytest.raises(ValueError):
        binding.expert_linear(x, w[None], cu[:1])
    lib, h = binding.load_library(), binding._default(x.device)._h
    out = torch.zeros(10, 12, dtype=x.dtype, device="cuda")

    def call(**kw):
        a = binding.LinearArgs(x=x.data_ptr(), weight=w.data_ptr(), out=out.data_ptr(), x_row=64, weight_row=64,
                               out_row=12, rows=10, inner=64, outer=12)
        for k, v in kw.items():
            setattr(a, k, v)
        return lib.mbert_attn_linear(h, ctypes.byref(a), torch.cuda.current_stream().cuda_stream)

    assert call() == 0
    assert call(dtype=2) == -2
    for kw in (dict(rows=-1), dict(rows=2 ** 31 - 1), dict(inner=0), dict(outer=0), dict(outer=2 ** 24 + 1),
               dict(activation=5), dict(activation=-1), dict(gated=2), dict(experts=-1), dict(x=None), dict(out=None),
               dict(weight=None), dict(x_row=56), dict(x_row=65), dict(weight_row=2 ** 61), dict(out_row=11),
               dict(x_row=2 ** 39), dict(out_row=2 ** 39),
               dict(out_row=2 ** 62), dict(out=out.data_ptr() + 1), dict(x=x.data_ptr() + 2),
               dict(cu_experts=cu.data_ptr()), dict(row_scale=out.data_ptr()), dict(experts=1),
               dict(experts=1, cu_experts=cu.data_ptr() + 1), dict(experts=1, cu_experts=cu.data_ptr(), residual=x.data_ptr()),
               dict(experts=2, cu_experts=cu.data_ptr(), weight_expert=64),
               dict(experts=2, cu_experts=cu.data_ptr(), weight_expert=2 ** 39), dict(residual=out.data_ptr(), residual_row=13)):
        assert call(**kw) == -1, kw
    assert call(rows=0, x=None) == 0
    err0()


@pytest.mark.gpu
def test_graph_streams_and_other_sizes(built):
    """A captured layer of experts and products replays on other offsets and inputs
    with the bits of eager calls; two streams at once."""
    E, K, N, T = 6, 264, 160, 400
    w, w2 = rnd(E, 2 * N, K, seed=1, sc=0.06).cuda(), rnd(E, K, N, seed=2, sc=0.08).cuda()
    wl = rnd(K, K, seed=3, sc=0.06).cuda()
    x = torch.zeros(T, K, dtype=torch.bfloat16, device="cuda")
    cu = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    s = torch.rand(T, device="cuda")
    out, mid = torch.zeros(T, K, dtype=x.dtype, device="cuda"), torch.zeros(T, N, dtype=x.dtype, device="cuda")

    def layer():
        binding.expert_linear(x, w, cu, activation="gelu", gated=True, out=mid)
        binding.expert_linear(mid, w2, cu, row_scale=s, out=out)
        return binding.linear(out, wl, residual=x), binding.linear(out[:9], wl, activation="relu")

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        layer()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a, b = layer()
    for trial, sizes in enumerate(([400, 0, 0, 0, 0, 0], [0, 30, 100, 1, 69, 200], [3, 3, 3, 3, 3, 3])):
        x.copy_(rnd(T, K, seed=trial))
        o = [0]
        for n in sizes:
            o.append(o[-1] + n)
        cu.copy_(torch.tensor(o, dtype=torch.int32))
        out.fill_(1.0)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (mid[:o[-1]], out, a, b)]
        out.fill_(1.0)
        want = layer()
        err0()
        for i, (p, q) in enumerate(zip(got, (mid[:o[-1]], out) + tuple(want))):
            assert torch.equal(p, q), (trial, i)
    xs = [rnd(n, K, seed=n).cuda() for n in (700, 12)]
    want = [binding.linear(t, wl, activation="gelu") for t in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(20):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(binding.linear(xs[i], wl, activation="gelu"))
    err0()
    for i in range(2):
        assert all(torch.equal(t, want[i]) for t in got[i])
