"""Products, norms and attention of any width together, as a layer uses them: every
step against its formula in 64 bits on the GPU's own input to it, and the steps
against calls in another order of streams and in a captured graph.  Sizes drawn over
the range, rows beyond 32 bits of elements.

Tolerances as in test_linear.py and test_residual_norm.py.
"""
import math
import random

import pytest
import torch

import test_linear as L
import test_residual_norm as N
from encoder_only_transformer_gb300 import binding
from test_linear import built, err0, rnd  # noqa: F401

pytestmark = pytest.mark.gpu


def check_linear(got, x, w, b=None, activation="none", gated=False, residual=None, row_scale=None):
    c = lambda t: None if t is None else t.cpu()
    y, t = L.product(c(x), c(w), c(b), activation, gated)
    L.check(got, *L.finish(y, t, got.dtype, c(row_scale), c(residual)))


def check_norm(h, y, x, branch, w, b=None, aw=None, ab=None, gate=None, kind="layer", scale=1.0):
    c = lambda t: None if t is None else t.cpu()
    rh, dh, ry, dy = N.reference(c(x), c(branch), c(w), c(b), c(aw), c(ab), c(gate), kind, scale, 1e-5)
    N.check(h, rh, dh, "h")
    N.check(y, ry, dy, "y")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_layer_of_another_width(built, dtype):  # noqa: F811
    """A pre-norm layer of width 640 with 10 heads of 64, biases and a gated MLP:
    the norm, Wqkv, rotary positions, attention, Wo with the residual, the norm
    with the residual of the branch, both products of the MLP."""
    lens, D, H, inner = [70, 1, 33], 640, 10, 1000
    T = sum(lens)
    cu = torch.tensor([0, 70, 71, 104], dtype=torch.int32, device="cuda")
    g = lambda *s, seed, sc=1.0: rnd(*s, seed=seed, dtype=dtype, sc=sc).cuda()
    x = g(T, D, seed=1)
    nw, mw = g(D, seed=2, sc=0.1) + 1, g(D, seed=3, sc=0.1) + 1
    wqkv, bqkv = g(3 * D, D, seed=4, sc=D ** -0.5), g(3 * D, seed=5, sc=0.1)
    wo, wi, wo2 = g(D, D, seed=6, sc=D ** -0.5), g(2 * inner, D, seed=7, sc=D ** -0.5), g(D, inner, seed=8, sc=0.03)
    bi = g(2 * inner, seed=9, sc=0.1)
    rope = binding.Rotary(64)

    def layer():
        _, y = binding.residual_norm(x, None, nw)
        qkv = binding.linear(y, wqkv, bqkv)
        heads = qkv.view(T, 3 * H, 64)
        q, k = (binding.rotary(heads[:, i * H:(i + 1) * H], rope, cu_seqlens=cu) for i in (0, 1))
        a = binding.cross_attention(q, k, heads[:, 2 * H:], cu, cu)
        branch = binding.linear(a.view(T, D), wo)
        h, y2 = binding.residual_norm(x, branch, mw)
        m = binding.linear(y2, wi, bi, "gelu", gated=True)
        return y, qkv, a, branch, h, y2, m, binding.linear(m, wo2, residual=h)

    y, qkv, a, branch, h, y2, m, out = layer()
    err0()
    N.check(y, *N.reference(x.cpu(), None, nw.cpu(), None, None, None, None, "layer", 1.0, 1e-5)[2:])
    check_linear(qkv, y, wqkv, bqkv)
    check_linear(branch, a.view(T, D), wo)
    check_norm(h, y2, x, branch, mw)
    check_linear(m, y2, wi, bi, "gelu", True)
    check_linear(out, m, wo2, residual=h)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = layer()
    x.copy_(rnd(T, D, seed=20, dtype=dtype))
    graph.replay()
    torch.cuda.synchronize()
    want = layer()
    err0()
    assert all(torch.equal(p, q) for p, q in zip(again, want)) and not torch.equal(want[-1], out)


def test_mixture_of_experts(built):  # noqa: F811
    """Routed rows sorted by expert, both products, the row weights, and the norms
    around the block with a gate."""
    T, D, inner, E, k = 200, 512, 384, 6, 2
    x = rnd(T, D, seed=1).cuda()
    router = rnd(E, D, seed=2, sc=0.1).cuda()
    wi, wo = rnd(E, 2 * inner, D, seed=3, sc=0.05).cuda(), rnd(E, D, inner, seed=4, sc=0.05).cuda()
    nw, aw, gate = rnd(D, seed=5, sc=0.1).cuda() + 1, rnd(D, seed=6, sc=0.1).cuda() + 1, rnd(D, seed=7).cuda()
    logits = binding.linear(x, router).float()
    logits[:, 3] = -1e9                                                 # an expert that nobody asks
    weight, expert = logits.softmax(-1).topk(k)
    order = expert.flatten().argsort(stable=True)
    cu = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    cu[1:] = expert.flatten().bincount(minlength=E).cumsum(0)
    xs, s = x[order // k].contiguous(), weight.flatten()[order].contiguous()
    m = binding.expert_linear(xs, wi, cu, activation="silu", gated=True)
    y = binding.expert_linear(m, wo, cu, row_scale=s)
    branch = torch.zeros(T, D, device="cuda").index_add_(0, order // k, y.float()).to(x.dtype)
    h, n = binding.residual_norm(x, branch, nw, branch_weight=aw, gate=gate, norm="rms")
    err0()
    o = cu.tolist()
    assert o[3] == o[4]
    for e in range(E):
        r = slice(o[e], o[e + 1])
        check_linear(m[r], xs[r], wi[e], activation="silu", gated=True)
        check_linear(y[r], m[r], wo[e], row_scale=s[r])
    check_norm(h, n, x, branch, nw, aw=aw, gate=gate, kind="rms")


@pytest.mark.parametrize("seed", range(40))
def test_drawn_products(built, seed):  # noqa: F811
    """Sizes over the range, odd ones among them: every kernel, tile and split, with
    the parts of the epilogue drawn too."""
    r = random.Random(seed)
    log = lambda lo, hi: int(round(math.exp(r.uniform(math.log(lo), math.log(hi)))))
    dtype, gated, act = r.choice(["bf16", "f16"]), r.random() < 0.5, r.choice(list(L.REL))
    K, n = 8 * log(1, 500), log(1, 3000)
    if seed % 2:
        sizes = [0 if r.random() < 0.2 else log(1, 400) for _ in range(log(1, 40))]
        while sum(sizes) * K * n > 4e9 or len(sizes) * K * n > 2e8:
            K, n = max(8, K // 16 * 8), max(1, n // 2)
        L.run_experts(sizes, K, n, dtype, act, r.random() < 0.5, gated, r.random() < 0.5, seed, r.choice([0, 5]),
                      r.choice([0, 8]))
    else:
        T = log(1, 5000)
        while T * K * n > 4e9:
            K, n = max(8, K // 16 * 8), max(1, n // 2)
        got, dev = L.run_linear(T, K, n, dtype, act, r.random() < 0.5, gated, r.random() < 0.5, seed)
        assert torch.equal(got, binding.linear(dev[0], dev[1], dev[2], act, gated, dev[3]))


@pytest.mark.parametrize("T,K,n", [(1, 8192, 40), (5, 16000, 700), (60, 6000, 33), (128, 4096, 512), (16, 64, 9000),
                                   (300, 5000, 20), (900, 7000, 64)])
def test_long_inner_dimensions(built, T, K, n):  # noqa: F811
    """Cut among the CTAs of a cluster, or walked by one."""
    for gated in (False, True):
        L.run_linear(T, K, n, "bf16", "gelu", bias=True, gated=gated, residual=True, seed=T)


def test_beyond_32_bits(built):  # noqa: F811
    """More than 2^31 numbers in the result, in x, in rows of a norm: sampled rows equal
    the same rows alone."""
    T, n = 270001, 8200
    x, w = rnd(T, 64, seed=1).cuda(), rnd(n, 64, seed=2, sc=0.1).cuda()
    pick = torch.tensor([0, 1, 130000, 261900, T - 130, T - 1], device="cuda")
    out = binding.linear(x, w, activation="silu")
    assert out.numel() > 2 ** 31
    check_linear(out[pick], x[pick], w, activation="silu")
    cu = torch.tensor([0, 100000, 100000, T - 3], dtype=torch.int32, device="cuda")
    we = torch.stack([w, w, -w])
    out2 = torch.zeros_like(out)
    binding.expert_linear(x, we, cu, out=out2)
    check_linear(out2[pick[:2]], x[pick[:2]], w)
    check_linear(out2[pick[2:5]], x[pick[2:5]], -w)
    assert (out2[T - 3:] == 0).all()
    h, y = binding.residual_norm(out, out2, w[:, 0].contiguous(), norm="rms", h_out=out2)
    want = binding.residual_norm(out[pick], binding.linear(x[pick], w) * torch.tensor([1, 1, -1, -1, -1, 0], device="cuda")
                                 [:, None].to(x.dtype), w[:, 0].contiguous(), norm="rms")
    assert torch.equal(h[pick], want[0]) and torch.equal(y[pick], want[1])
    back = binding.linear(out, rnd(24, n, seed=3, sc=0.01).cuda())
    check_linear(back[pick], out[pick], rnd(24, n, seed=3, sc=0.01))
    err0()


def test_calls_at_once(built):  # noqa: F811
    """Calls of all three operators on three streams, short and long ones side by side."""
    E = 5
    x, w = rnd(900, 256, seed=1).cuda(), rnd(300, 256, seed=2, sc=0.06).cuda()
    we = rnd(E, 2 * 200, 256, seed=3, sc=0.06).cuda()
    cu = torch.tensor([0, 10, 10, 300, 310, 900], dtype=torch.int32, device="cuda")
    few = torch.tensor([0, 1, 4, 4, 20, 30], dtype=torch.int32, device="cuda")
    nw = rnd(256, seed=4).cuda()
    calls = [lambda: binding.linear(x, w, activation="gelu"), lambda: binding.linear(x[:7], w),
             lambda: binding.expert_linear(x, we, cu, gated=True), lambda: binding.expert_linear(x[:30], we, few, gated=True),
             lambda: binding.residual_norm(x, x, nw)[1]]
    want = [c() for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for i in range(30):
        for s, st in enumerate(streams):
            with torch.cuda.stream(st):
                k = (i + 2 * s) % len(calls)
                got.append((k, calls[k]()))
    err0()
    assert all(torch.equal(t, want[k]) for k, t in got)


def test_threads(built):  # noqa: F811
    """Products of many sizes from four threads, each on a stream of its own."""
    import threading
    x, w = rnd(400, 512, seed=1).cuda(), rnd(900, 512, seed=2, sc=0.05).cuda()
    sizes = [(t, n) for t in (1, 9, 40, 130, 400) for n in range(20, 900, 67)]
    want = {s: binding.linear(x[:s[0]], w[:s[1]]) for s in sizes}
    torch.cuda.synchronize()
    wrong = []

    def run(seed):
        order = sizes * 3
        random.Random(seed).shuffle(order)
        with torch.cuda.stream(torch.cuda.Stream()):
            got = [(s, binding.linear(x[:s[0]], w[:s[1]])) for s in order]
            torch.cuda.current_stream().synchronize()
            wrong.extend(s for s, t in got if not torch.equal(t, want[s]))

    threads = [threading.Thread(target=run, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    err0()
    assert not wrong


@pytest.mark.parametrize("sizes", [[300, 0] * 80, [0] * 127 + [513] + [0] * 130 + [1, 700]], ids=["160", "260"])
def test_many_experts_of_many_rows(built, sizes):  # noqa: F811
    """More groups than a warp holds the offsets of at a time, whole tiles in each."""
    L.run_experts(sizes, 64, 136, "bf16", "gelu", True, False, True, 3, 5)
