"""Cross attention (binding.cross_attention, cross_attention_padded) against its
formula in 64 bits.

Tolerance per element, from the arithmetic, with W the exact weights, u_t =
eps_t / 2 of the 16-bit type, u = 2^-24:
  - the weights are rounded to the type before P V:    u_t   sum W |v|
  - a score's dot product of D terms in fp32 (taken as truncating, 2 u a term),
    its scaling and the exponent's argument, a change d of a score changes its
    weight by the factor 1 + d:  d = scale D 2 u sum |q||k| + 4 u |score|
  - ex2.approx (2^-22), the references' moves and the joining of parts:  2^-18
    in all; each of the last two counts for W |v| and, through the sum, W |out|
  - sums over the keys in fp32:  2 u L (sum W |v| + |out|)
  - fp16 weights below its normal range: 2^-25 absolute on a scale where the
    largest weight is at least 2^7: 2^-32 sum |v|
  - the output's rounding:  u_t |out|
"""
import math

import pytest
import torch

from encoder_only_transformer_gb300 import binding

U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def built():
    import __graft_entry__
    __graft_entry__.build()


def attend(q, k, v, scale, mask=None):
    """One sequence, fp64: -> (out, tolerance), [Lq, H, D]."""
    Lq, H, D = q.shape
    Lk, Hk = k.shape[0], k.shape[1]
    out, tol = torch.zeros(Lq, H, D, dtype=torch.float64), torch.zeros(Lq, H, D, dtype=torch.float64)
    vis = torch.ones(Lk, dtype=torch.bool) if mask is None else mask
    if not vis.any() or Lq == 0:
        return out, tol
    ut = torch.finfo(q.dtype).eps / 2
    for h in range(H):
        qh = q[:, h].double()
        kh, vh = k[vis, h // (H // Hk)].double(), v[vis, h // (H // Hk)].double()
        s = scale * (qh @ kh.T)
        d = scale * D * 2 * U * (qh.abs() @ kh.abs().T) + 4 * U * s.abs() + 2.0 ** -18
        w = torch.softmax(s, -1)
        o = w @ vh
        wd = (w * d) @ vh.abs() + (w * d).sum(-1, keepdim=True) * o.abs()
        wv = w @ vh.abs()
        t = ut * wv + wd + 2 * U * Lk * (wv + o.abs())
        if q.dtype == torch.float16:
            t = t + 2.0 ** -32 * vh.abs().sum(0)
        out[:, h], tol[:, h] = o, t + ut * (o.abs() + t)
    return out, tol


def check(got, ref, tol):
    g = got.double().cpu()
    assert torch.isfinite(g).all()
    err = (g - ref).abs()
    tiny = torch.finfo(got.dtype).smallest_normal * torch.finfo(got.dtype).eps
    bad = err > tol + tiny
    assert not bad.any(), (f"{int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}, "
                           f"max err {err.max().item():.3e} against {tol.max().item():.3e}")


def offsets(lens):
    out = [0]
    for x in lens:
        out.append(out[-1] + x)
    return out


def make(ql, kl, H, Hk, D, dtype, seed=0, behind=0, scale=1.0):
    """Packed inputs on the CPU; `behind` rows after the last sequence are NaN
    in k and v (nothing may see them)."""
    g = torch.Generator().manual_seed(seed)
    t = TYPES[dtype]
    q = (torch.randn(sum(ql) + behind, H, D, generator=g) * scale).to(t)
    k = (torch.randn(sum(kl) + behind, Hk, D, generator=g) * scale).to(t)
    v = torch.randn(sum(kl) + behind, Hk, D, generator=g).to(t)
    k[sum(kl):] = math.nan
    v[sum(kl):] = math.nan
    return q, k, v


def cu_of(lens):
    return torch.tensor(offsets(lens), dtype=torch.int32).cuda()


def reference(q, k, v, ql, kl, scale=None, mask=None):
    scale = q.shape[2] ** -0.5 if scale is None else scale
    out = torch.zeros(q.shape, dtype=torch.float64)
    tol = torch.zeros(q.shape, dtype=torch.float64)
    qo, ko = offsets(ql), offsets(kl)
    for s in range(len(ql)):
        i, j = slice(qo[s], qo[s + 1]), slice(ko[s], ko[s + 1])
        out[i], tol[i] = attend(q[i], k[j], v[j], scale, None if mask is None else mask[j])
    return out, tol


def run_packed(ql, kl, H, Hk, D, dtype, max_q=0, seed=0, behind=0, mask=None, scale=None, qscale=1.0):
    q, k, v = make(ql, kl, H, Hk, D, dtype, seed, behind, qscale)
    if mask is not None:
        k[:sum(kl)][~mask] = math.inf           # unseen keys may hold anything
        v[:sum(kl)][~mask] = math.nan
    m = None
    if mask is not None:
        m = torch.zeros(sum(kl) + behind, dtype=torch.int32)
        m[:sum(kl)] = mask.int() * 5            # any non-zero value is visible
        m = m.cuda()
    out = torch.full(q.shape, 3.0, dtype=q.dtype).cuda()
    got = binding.cross_attention(q.cuda(), k.cuda(), v.cuda(), cu_of(ql), cu_of(kl), max_seqlen_q=max_q,
                                  key_mask=m, scale=scale, out=out)
    torch.cuda.synchronize()
    assert binding._default(got.device).get_error() == 0
    n = sum(ql)
    assert (got[n:] == 3.0).all()               # rows behind the last sequence
    ref, tol = reference(q[:n], k[:sum(kl)], v[:sum(kl)], ql, kl, scale, mask)
    check(got[:n], ref, tol)
    return got


# ------------------------------------------------------------------- CPU
def test_host_refusals_without_device(built):
    import ctypes
    lib = binding.load_library()
    a = binding.CrossArgs()
    n = ctypes.c_int64()
    assert lib.mbert_attn_cross_workspace(None, ctypes.byref(a), ctypes.byref(n)) == -1
    assert lib.mbert_attn_cross(None, ctypes.byref(a), None, 0, None) == -1
    z = torch.zeros(1, 1, 64, dtype=torch.bfloat16)
    cu = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        binding.cross_attention(z, z, z, cu, cu)
    with pytest.raises(ValueError):
        binding.cross_attention_padded(z[None], z[None], z[None])


# ------------------------------------------------------------------- GPU
BLOCKS = [
    # query lengths, key lengths, heads, key heads
    ([128], [128], 1, 1),
    ([1, 40], [1, 40], 12, 12),
    ([127, 128, 129], [129, 128, 127], 3, 1),
    ([255, 256, 257, 0, 30], [0, 1, 300, 77, 1000], 2, 2),
    ([300], [5], 4, 2),
    ([17], [2500], 12, 12),
    ([513, 20], [900, 1300], 6, 3),
    ([20] * 40, list(range(0, 400, 10)), 2, 1),
    ([21, 1, 0, 65, 33], [300, 500, 10, 129, 0], 8, 1),         # eight heads share a block's rows
    ([5, 11], [700, 900], 32, 1),
    ([1, 3, 130], [200, 64, 90], 256, 1),                       # 128 of 256 heads share them
    ([50, 7], [130, 400], 12, 2),                               # two of six
    ([40], [333], 9, 3),                                        # none of three
    ([300, 129], [140, 700], 16, 4),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ql,kl,H,Hk", BLOCKS)
def test_blocks(built, ql, kl, H, Hk, D, dtype):
    run_packed(ql, kl, H, Hk, D, dtype, seed=len(ql) + D, behind=3)


@pytest.mark.gpu
@pytest.mark.parametrize("D,dtype", [(64, "bf16"), (128, "f16")])
@pytest.mark.parametrize("ql,kl,H", [
    ([250] * 12, [640] * 12, 12),                           # as many units as processors, near enough
    ([100, 300, 0, 256, 257, 1] * 3, [600, 520, 900, 0, 530, 700] * 3, 9),      # two rounds, halves, empty ones
    ([17] * 60, [520 + 3 * i for i in range(60)], 10),      # four rounds
    ([17] * 61, [520 + 3 * i for i in range(61)], 10),      # one unit more than four rounds
    ([200] * 9, [1400, 1300, 1200] + [600] * 6, 16),        # the longest beyond the others' share
    ([5] * 129, [515 + i % 7 for i in range(129)], 1),      # more sequences than are dealt
])
def test_whole_units(built, ql, kl, H, D, dtype):
    """Calls whose units are dealt out whole, and ones just beyond."""
    mask = torch.ones(sum(kl), dtype=torch.bool)
    mask[700:900] = False
    got = run_packed(ql, kl, H, H, D, dtype, seed=len(ql), behind=2, mask=mask)
    assert torch.equal(run_packed(ql, kl, H, H, D, dtype, seed=len(ql), behind=2, mask=mask), got)


@pytest.mark.gpu
@pytest.mark.parametrize("D,dtype", [(64, "bf16"), (64, "f16"), (128, "bf16"), (128, "f16")])
@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("ql,kl,H,Hk,max_q", [
    ([128, 17, 0, 65], [300, 1, 50, 0], 2, 2, 128),
    ([40, 100, 1], [129, 700, 640], 12, 12, 100),           # longer than what is never cut
    ([17] * 3, [4000, 10, 2000], 3, 3, 17),                 # cut
    ([16, 3, 11], [333, 1500, 64], 32, 8, 16),              # four heads share a block's rows
    ([1], [900], 256, 1, 1),                                # 128 of 256 heads do
    ([30] * 64, [520 + 2 * i for i in range(64)], 6, 6, 30),    # dealt out whole
    ([20] * 130, [100 + i for i in range(130)], 10, 10, 20),
])
def test_small_blocks(built, ql, kl, H, Hk, max_q, masked, D, dtype):
    """At most 128 rows a sequence: one query tile to a block."""
    mask = None
    if masked:
        g = torch.Generator().manual_seed(len(ql))
        mask = torch.rand(sum(kl), generator=g) < 0.7
        mask[offsets(kl)[-2]:] = False                      # nothing of the last sequence
    got = run_packed(ql, kl, H, Hk, D, dtype, max_q=max_q, seed=len(ql), behind=2, mask=mask)
    assert torch.equal(run_packed(ql, kl, H, Hk, D, dtype, max_q=max_q, seed=len(ql), behind=2, mask=mask), got)


TOKENS = [
    # query lengths, key lengths, heads, key heads, longest query sequence
    ([1], [1], 1, 1, 1),
    ([1] * 5, [0, 15, 16, 17, 300], 12, 12, 1),
    ([1, 0, 2, 1], [63, 64, 65, 129], 4, 2, 2),
    ([4] * 3, [1000, 1, 513], 8, 2, 4),
    ([16], [700], 3, 3, 16),
    ([1], [20000], 2, 1, 1),
    ([1] * 2, [6000, 30], 32, 2, 1),
    ([5, 7, 0, 16, 1], [100, 200, 300, 400, 0], 1, 1, 16),
    ([1] * 400, [(7 * i) % 90 for i in range(400)], 2, 2, 1),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ql,kl,H,Hk,max_q", TOKENS)
def test_tokens(built, ql, kl, H, Hk, max_q, D, dtype):
    run_packed(ql, kl, H, Hk, D, dtype, max_q=max_q, seed=len(ql) + D, behind=2)


@pytest.mark.gpu
@pytest.mark.parametrize("D,dtype", [(64, "bf16"), (128, "f16")])
@pytest.mark.parametrize("kind", ["token", "blocks"])
@pytest.mark.parametrize("pattern", ["holes", "first", "last", "none_in_some", "tiles", "all", "mixed"])
def test_key_masks(built, pattern, kind, D, dtype):
    """Masked keys hold infinities and NaN; whole tiles, ends and rows of the
    batch masked away."""
    kl = [300, 1, 64, 777, 129]
    ql = [1, 2, 1, 2, 1] if kind == "token" else [130, 1, 257, 40, 128]
    n, g = sum(kl), torch.Generator().manual_seed(4)
    mask = torch.ones(n, dtype=torch.bool)
    ko = offsets(kl)
    if pattern == "holes":
        mask = torch.rand(n, generator=g) < 0.5
    elif pattern == "first":
        for s in range(len(kl)):
            mask[ko[s] + 1:ko[s + 1]] = False
    elif pattern == "last":
        for s in range(len(kl)):
            mask[ko[s]:ko[s + 1] - 1] = False
    elif pattern == "none_in_some":
        for s in (0, 2, 4):
            mask[ko[s]:ko[s + 1]] = False
    elif pattern == "mixed":        # right-padded, whole and holed sequences by turns
        mask[ko[0] + 200:ko[1]] = False
        mask[ko[3] + 400] = False
        mask[ko[3] + 700:ko[4]] = False
        mask[ko[4] + 128:] = False
    elif pattern == "tiles":
        mask[ko[3]:ko[3] + 128] = False
        mask[ko[3] + 256:ko[3] + 512] = False
    run_packed(ql, kl, 4, 2, D, dtype, max_q=2 if kind == "token" else 0, seed=9, behind=1, mask=mask)


@pytest.mark.gpu
@pytest.mark.parametrize("max_q", [0, 2])
def test_cut_sequence_with_holes(built, max_q):
    """A sequence cut between CTAs whose parts have no, some and all keys
    visible."""
    mask = torch.zeros(9000, dtype=torch.bool)
    mask[4096:4100] = True
    mask[8000:8500] = True
    run_packed([2] if max_q else [40], [9000], 2, 1, 64, "bf16", max_q=max_q, mask=mask)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["token", "blocks"])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_neighbours_do_not_leak(built, kind, dtype):
    """The rows of other sequences may be infinite or NaN."""
    kl, ql = [70, 200, 61], ([1, 1, 1] if kind == "token" else [40, 130, 50])
    q, k, v = make(ql, kl, 4, 4, 64, dtype, seed=3)
    ko, qo = offsets(kl), offsets(ql)
    k[ko[1]:ko[2]] = math.nan
    v[ko[1]:ko[2]] = math.inf
    q[qo[1]:qo[2]] = math.nan
    got = binding.cross_attention(q.cuda(), k.cuda(), v.cuda(), cu_of(ql), cu_of(kl),
                                  max_seqlen_q=1 if kind == "token" else 0)
    for s in (0, 2):
        i, j = slice(qo[s], qo[s + 1]), slice(ko[s], ko[s + 1])
        check(got[i], *attend(q[i], k[j], v[j], 0.125))
    assert torch.isnan(got[qo[1]:qo[2]]).all()      # and a NaN that is seen stays one


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["token", "blocks"])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("D", [64, 128])
def test_wide_scores(built, kind, D, dtype):
    """Scores that tower and grow along the keys (references move often), and a
    long tail of small weights beside one large one."""
    ql, kl = ([3], [1500]) if kind == "token" else ([200], [1500])
    max_q = 3 if kind == "token" else 0
    q, k, v = make(ql, kl, 2, 2, D, dtype, seed=6, scale=1.5)
    k *= torch.linspace(0.2, 4, 1500)[:, None, None].to(k.dtype)
    got = binding.cross_attention(q.cuda(), k.cuda(), v.cuda(), cu_of(ql), cu_of(kl), max_seqlen_q=max_q)
    check(got, *reference(q, k, v, ql, kl))
    q[:] = 0
    q[..., 0] = 8.0
    k[:] = 0
    k[777, :, 0] = 12.0         # scores: 96 scale log2(e) once, 0 elsewhere
    v[777] = 0                  # so the tail's share is all there is
    got = binding.cross_attention(q.cuda(), k.cuda(), v.abs().cuda(), cu_of(ql), cu_of(kl),
                                  max_seqlen_q=max_q)
    ref, tol = reference(q, k, v.abs(), ql, kl)
    check(got, ref, tol)
    assert ref.max() > 0 and (got > 0).float().mean() > 0.9


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [1e-6, 0.01, 1.0, 5.0])
def test_scale(built, scale):
    run_packed([30, 2], [200, 500], 2, 2, 64, "bf16", scale=scale, qscale=0.5)
    run_packed([1, 2], [200, 500], 2, 2, 64, "f16", max_q=2, scale=scale, qscale=0.5)


@pytest.mark.gpu
@pytest.mark.parametrize("B,Sq,Sk,H,Hk,D,dtype", [
    (3, 1, 700, 12, 12, 64, "bf16"), (4, 2, 130, 16, 2, 128, "f16"), (2, 140, 333, 3, 3, 64, "bf16"),
    (5, 300, 64, 4, 1, 128, "bf16"), (1, 1, 1, 1, 1, 64, "f16"), (2, 3, 0, 2, 2, 64, "bf16")])
@pytest.mark.parametrize("masked", [False, True])
def test_padded(built, B, Sq, Sk, H, Hk, D, dtype, masked):
    g = torch.Generator().manual_seed(B * Sq)
    t = TYPES[dtype]
    q = torch.randn(B, Sq, H, D, generator=g).to(t)
    kv = torch.randn(B, Sk, 2 * Hk, D, generator=g).to(t)          # fused states
    lens = [(Sk * (b + 1)) // B if b != 1 else 0 for b in range(B)] if masked else [Sk] * B
    mask = torch.arange(Sk)[None] < torch.tensor(lens)[:, None]
    if masked:
        kv[~mask] = math.nan
    kvc = kv.cuda()
    got = binding.cross_attention_padded(q.cuda(), kvc[:, :, :Hk], kvc[:, :, Hk:],
                                         mask.int().cuda() if masked else None)
    for b in range(B):
        check(got[b], *attend(q[b], kv[b, :, :Hk], kv[b, :, Hk:], D ** -0.5, mask[b]))
    assert binding._default(got.device).get_error() == 0


@pytest.mark.gpu
def test_strided_rows(built):
    """Views of fused rows on every side give the contiguous call's result."""
    ql, kl = [140, 9], [260, 31]
    q, k, v = (x.cuda() for x in make(ql, kl, 4, 2, 64, "bf16", seed=2))
    want = binding.cross_attention(q, k, v, cu_of(ql), cu_of(kl))
    big_q = torch.full((149, 4 * 64 + 24), 9.0, dtype=q.dtype, device="cuda")
    big_o = big_q.clone()
    vq, vo = (b[:, 16:16 + 256].unflatten(1, (4, 64)) for b in (big_q, big_o))
    vq.copy_(q)
    kv = torch.cat([k, v], 1)
    got = binding.cross_attention(vq, kv[:, :2], kv[:, 2:], cu_of(ql), cu_of(kl), out=vo)
    assert torch.equal(got, want)
    assert (big_o[:, :16] == 9.0).all() and (big_o[:, 272:] == 9.0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("ql,kl,max_q", [([1] * 3, [5000, 700, 9000], 1), ([700, 300], [2000, 5000], 0)])
def test_repeatable_and_independent_of_company(built, ql, kl, max_q):
    """Bit-equal from run to run, however the CTAs race; two streams at once."""
    q, k, v = (x.cuda() for x in make(ql, kl, 12, 12, 64, "bf16", seed=5))
    cq, ck = cu_of(ql), cu_of(kl)
    want = binding.cross_attention(q, k, v, cq, ck, max_seqlen_q=max_q)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for i in range(12):
        with torch.cuda.stream(streams[i % 2]):
            outs.append(binding.cross_attention(q, k, v, cq, ck, max_seqlen_q=max_q))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


@pytest.mark.gpu
@pytest.mark.parametrize("max_q", [0, 1])
def test_captured_with_changing_lengths(built, max_q):
    """One captured call replayed after the offsets and the data changed; two
    captured calls in one graph."""
    ql, kl = [1, 1, 1], [3000, 20, 400]
    q, k, v = (x.cuda() for x in make(ql, kl, 4, 4, 64, "bf16", seed=7))
    cq, ck = cu_of(ql), cu_of(kl)
    binding.cross_attention(q, k, v, cq, ck, max_seqlen_q=max_q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a = binding.cross_attention(q, k, v, cq, ck, max_seqlen_q=max_q)
        b = binding.cross_attention(a, k, v, cq, ck, max_seqlen_q=max_q)
    for kl2 in ([3000, 20, 400], [10, 3000, 0], [0, 0, 3420]):
        ck.copy_(torch.tensor(offsets(kl2), dtype=torch.int32))
        q.mul_(0.9)
        graph.replay()
        torch.cuda.synchronize()
        qc, kc, vc = q.cpu(), k.cpu(), v.cpu()
        n = sum(kl2)
        check(a, *reference(qc, kc[:n], vc[:n], ql, kl2))
        check(b, *reference(a.cpu(), kc[:n], vc[:n], ql, kl2))


@pytest.mark.gpu
def test_with_rotary_it_is_a_global_layer(built):
    """Norm-free rotation of the encoder's own queries and keys, then attention
    with cu_q = cu_k: the framework's global layer, at its own bounds.  Then the
    whole run as a decoder would use it."""
    from encoder_only_transformer_gb300 import workloads as W
    wl = W.custom([300, 1, 130, 770], seed=12)
    qkv, cu = wl.qkv.cuda(), wl.cu_seqlens.cuda()
    heads = qkv.unflatten(1, (36, 64))
    rope = binding.Rotary(64, base=160000.0)
    q = binding.rotary(heads[:, :12], rope, cu_seqlens=cu)
    k = binding.rotary(heads[:, 12:24], rope, cu_seqlens=cu)
    got = binding.cross_attention(q, k, heads[:, 24:], cu, cu).flatten(1)
    want = binding.attention(qkv, cu, "global")
    err = (got.float() - want.float()).abs()
    # both are within 2e-2 (mean 2e-3) of the oracle
    assert err.max() <= 4e-2 and err.mean() <= 4e-3

    # a decoder's step over these states: norms and rotation of its own queries
    # and keys, self attention on the token's past, cross attention to the
    # encoder's outputs, through the framework's projection
    g = torch.Generator().manual_seed(1)
    w = (1 + 0.1 * torch.randn(64, generator=g)).bfloat16().cuda()
    dec = torch.randn(4, 36, 64, generator=g).bfloat16().cuda()
    pos = torch.tensor([5, 0, 17, 3], dtype=torch.int32).cuda()
    dq, dk = binding.qk_norm_rotary(dec[:, :12], dec[:, 12:24], w, w, rope, positions=pos)
    one = torch.arange(5, dtype=torch.int32).cuda()
    self_out = binding.cross_attention(dq, dk, dec[:, 24:], one, one, max_seqlen_q=1)
    # a single key: its value, whatever the score
    assert torch.equal(self_out, dec[:, 24:])
    states = want.unflatten(1, (12, 64))
    cross = binding.cross_attention(dq, states, states, one, cu, max_seqlen_q=1)
    check(cross, *reference(dq.cpu(), states.cpu(), states.cpu(), [1] * 4, [300, 1, 130, 770]))
    wo = (torch.randn(768, 768, generator=g) * 768 ** -0.5).bfloat16().cuda()
    y = binding.out_proj(cross.flatten(1), wo, self_out.flatten(1))
    ref = self_out.flatten(1).double() + cross.flatten(1).double() @ wo.double().T
    assert ((y.double() - ref).abs() / ref.abs().clamp(min=1)).max() <= 2e-2
    assert binding._default(q.device).get_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("max_q", [0, 2])
@pytest.mark.parametrize("cq,ck,want", [
    ([0, 2, 1], [0, 5, 10], -4), ([1, 2, 3], [0, 5, 10], -4), ([0, 1, 4], [0, 5, 10], -4),
    ([0, 1, 2], [0, 11, 10], -4), ([0, 1, 2], [0, 5, 11], -4), ([0, 1, 2], [2, 5, 10], -4),
    ([0, 3, 3], [0, 5, 10], -3), ([0, 1, 2], [-5, 5, 10], -4)])
def test_bad_offsets_write_nothing(built, cq, ck, want, max_q):
    if want == -3 and not max_q:
        return                      # without a bound every length is allowed
    q, k, v = (x.cuda() for x in make([3], [10], 2, 2, 64, "bf16"))
    out = torch.full_like(q, 3.0)
    h = binding._default(q.device)
    for mask in (None, torch.ones(10, dtype=torch.int32, device="cuda")):
        binding.cross_attention(q, k, v, torch.tensor(cq, dtype=torch.int32).cuda(),
                                torch.tensor(ck, dtype=torch.int32).cuda(), max_seqlen_q=max_q,
                                key_mask=mask, out=out)
        assert h.get_error() == want
        assert (out == 3.0).all() and h.get_error() == 0


@pytest.mark.gpu
def test_no_keys_and_no_queries(built):
    q, k, v = (x.cuda() for x in make([3], [10], 2, 2, 64, "bf16"))
    none = torch.zeros(2, dtype=torch.int32).cuda()
    some = torch.tensor([0, 3], dtype=torch.int32).cuda()
    for max_q in (0, 3):
        out = binding.cross_attention(q, k[:0], v[:0], some, none, max_seqlen_q=max_q)
        assert (out == 0).all()
        out = torch.full_like(q, 3.0)
        binding.cross_attention(q, k, v, none, torch.tensor([0, 10], dtype=torch.int32).cuda(), out=out,
                                max_seqlen_q=max_q)
        assert (out == 3.0).all()               # every row lies behind the last sequence
    assert binding.cross_attention(q[:0], k, v, none, none).shape == (0, 2, 64)
    empty = torch.zeros(1, dtype=torch.int32).cuda()
    assert binding.cross_attention(q[:0], k[:0], v[:0], empty, empty).shape == (0, 2, 64)
    assert binding._default(q.device).get_error() == 0


@pytest.mark.gpu
def test_refusals(built):
    q, k, v = (x.cuda() for x in make([3], [10], 4, 2, 64, "bf16"))
    cq, ck = cu_of([3]), cu_of([10])
    ok = dict(cu_seqlens_q=cq, cu_seqlens_k=ck)
    for bad in ((q.float(), k, v), (q, k.half(), v), (q, k, v[:9]), (q[..., :32], k[..., :32], v[..., :32]),
                (q[:, 0], k, v)):
        with pytest.raises(TypeError):
            binding.cross_attention(*bad, **ok)
    with pytest.raises(ValueError):
        binding.cross_attention(q.transpose(0, 1), k, v, **ok)
    with pytest.raises(ValueError):
        binding.cross_attention(q, k, v, cq, torch.tensor([0, 5, 10], dtype=torch.int32).cuda())
    with pytest.raises(TypeError):
        binding.cross_attention(q, k, v, cq.long(), ck)
    for scale in (0.0, -1.0, math.inf, math.nan):
        with pytest.raises(ValueError):
            binding.cross_attention(q, k, v, scale=scale, **ok)
    with pytest.raises(TypeError):
        binding.cross_attention(q, k, v, key_mask=torch.ones(10, dtype=torch.bool, device="cuda"), **ok)
    with pytest.raises(TypeError):
        binding.cross_attention(q, k, v, out=q[:2], **ok)
    with pytest.raises(binding.MbertAttnError):
        binding.cross_attention(q[:, :3], k, v, **ok)               # 3 heads over 2 (pitch kept)
    with pytest.raises(binding.MbertAttnError):
        binding.cross_attention(q, k, v, out=q, **ok)               # over its own queries
    with pytest.raises(binding.MbertAttnError):
        binding.cross_attention(q[:1].expand(3, 4, 64), k, v, **ok)  # rows over each other
    odd = torch.zeros(3, 4 * 64 + 4, dtype=q.dtype, device="cuda")[:, 4:].unflatten(1, (4, 64))
    with pytest.raises(binding.MbertAttnError):
        binding.cross_attention(odd, k, v, **ok)                    # off the 16-byte grid
    with pytest.raises(binding.MbertAttnError):
        binding.cross_attention(q, k, v, max_seqlen_q=-1, **ok)
    with pytest.raises(ValueError):
        binding.cross_attention_padded(q[None].expand(2, 3, 4, 64), k[None].repeat(2, 1, 1, 1),
                                       v[None].repeat(2, 1, 1, 1))
    with pytest.raises(TypeError):
        binding.cross_attention_padded(q[None], k[None], v[None], key_mask=torch.ones(1, 9, dtype=torch.int32).cuda())
    # the workspace is checked too
    import ctypes
    lib, h = binding.load_library(), binding._default(q.device)
    q, k, v = (x.cuda() for x in make([3], [2000], 4, 2, 64, "bf16"))
    ck = cu_of([2000])
    a = binding.CrossArgs(q.data_ptr(), k.data_ptr(), v.data_ptr(), torch.empty_like(q).data_ptr(), 256, 128, 128,
                          256, 3, 2000, 4, 2, 64, 0, 0.0, 1, cq.data_ptr(), ck.data_ptr(), 0, None)
    n = ctypes.c_int64()
    assert lib.mbert_attn_cross_workspace(h.handle, ctypes.byref(a), ctypes.byref(n)) == 0 and n.value > 0
    ws = torch.empty(n.value, dtype=torch.uint8, device="cuda")
    assert lib.mbert_attn_cross(h.handle, ctypes.byref(a), ws.data_ptr(), n.value - 1, None) == -1
    assert lib.mbert_attn_cross(h.handle, ctypes.byref(a), None, n.value, None) == -1
    a.rows_k = 500              # too short to be cut: no workspace
    assert lib.mbert_attn_cross_workspace(h.handle, ctypes.byref(a), ctypes.byref(n)) == 0 and n.value == 0
    assert h.get_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("H,Hk,D,dtype,kl", [
    (4, 4, 64, "bf16", [50000, 17, 0, 20000]), (12, 12, 64, "f16", [9000, 15000, 1]),
    (16, 4, 128, "bf16", [33000]), (6, 2, 64, "bf16", [70000, 70000]), (10, 10, 128, "f16", [14000, 300])])
@pytest.mark.parametrize("masked", [False, True])
def test_tokens_over_long_caches(built, H, Hk, D, dtype, kl, masked):
    """Every CTA with whole and cut units of several heads and sequences."""
    mask = None
    if masked:
        mask = torch.rand(sum(kl), generator=torch.Generator().manual_seed(1)) < 0.7
        mask[:4000] = False
    run_packed([1, 2, 1, 2][:len(kl)], kl, H, Hk, D, dtype, max_q=2, seed=3, behind=5, mask=mask)


@pytest.mark.gpu
def test_limits(built):
    """Sizes whose places or extents would not fit are refused on the host; a
    scale that fp32 takes for zero is no default; a bound given as a tensor
    counts by its value."""
    import ctypes
    lib, h = binding.load_library(), binding._default(torch.device("cuda", 0)).handle
    need = ctypes.c_int64()
    there = ctypes.addressof(need)      # never read: no call gets as far as a launch

    def status(rows_q=4, rows_k=4, pitch=64, scale=1.0):
        a = binding.CrossArgs(None, None, None, None, pitch, pitch, pitch, pitch, rows_q, rows_k, 1, 1, 64, 0,
                              scale, 1, there, there, 0, None)
        return lib.mbert_attn_cross_workspace(h, ctypes.byref(a), ctypes.byref(need))

    assert status() == 0
    assert status(rows_k=2 ** 31 - 2000) == 0
    assert status(rows_k=2 ** 31 - 1000) == -1 and status(rows_k=2 ** 31 - 1) == -1
    assert status(rows_q=2 ** 31 - 1) == -1
    assert status(scale=3e38) == -1
    q, k, v = (x.cuda() for x in make([3], [10], 1, 1, 64, "bf16"))
    a = binding.CrossArgs(q.data_ptr(), k.data_ptr(), v.data_ptr(), torch.empty_like(q).data_ptr(),
                          64, 1 << 37, 64, 64, 3, 2 ** 30, 1, 1, 64, 0, 1.0, 1,
                          cu_of([3]).data_ptr(), cu_of([10]).data_ptr(), 3, None)
    ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    assert lib.mbert_attn_cross(h, ctypes.byref(a), ws.data_ptr(), ws.numel(), None) == -1

    cu = dict(cu_seqlens_q=cu_of([3]), cu_seqlens_k=cu_of([10]))
    with pytest.raises(ValueError):
        binding.cross_attention(q, k, v, scale=1e-50, **cu)
    with pytest.raises(ValueError):
        binding.cross_attention_padded(q[None], k[None], v[None], scale=1e-50)
    bound = torch.tensor(3)
    want = binding.cross_attention(q, k, v, max_seqlen_q=3, **cu)
    assert torch.equal(binding.cross_attention(q, k, v, max_seqlen_q=bound, **cu), want)
    bound.fill_(-1)
    with pytest.raises(binding.MbertAttnError):
        binding.cross_attention(q, k, v, max_seqlen_q=bound, **cu)
    assert binding._default(q.device).get_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("D,dtype", [(64, "bf16"), (128, "f16")])
@pytest.mark.parametrize("Sq", [60, 250])
def test_captured_from_whole_to_cut_units(built, Sq, D, dtype):
    """A captured padded call replayed with masks that leave its units whole,
    cut, or without keys; two graphs at once on two streams, beside a global
    layer of the encoder."""
    from encoder_only_transformer_gb300 import workloads as W
    B, Sk, H = 6, 1500, 3
    g = torch.Generator().manual_seed(Sq + D)
    q = torch.randn(B, Sq, H, D, generator=g).to(TYPES[dtype])
    kv = torch.randn(B, Sk, 2 * H, D, generator=g).to(TYPES[dtype])
    lens = ([700] * B, [1500, 3, 0, 90, 640, 1], [0] * B, [1100] * B)
    dq, dkv = q.cuda(), kv.cuda()
    masks = [torch.zeros(B, Sk, dtype=torch.int32, device="cuda") for _ in range(2)]
    outs, graphs = [], []
    binding.cross_attention_padded(dq, dkv[:, :, :H], dkv[:, :, H:], key_mask=masks[0])
    for m in masks:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(binding.cross_attention_padded(dq, dkv[:, :, :H], dkv[:, :, H:], key_mask=m))
        graphs.append(graph)
    wl = W.custom([400, 9, 700], seed=3)
    qkv, cu = wl.qkv.cuda(), wl.cu_seqlens.cuda()
    layer = binding.attention(qkv, cu, "global")
    streams = [torch.cuda.Stream() for _ in range(3)]
    for i in range(len(lens)):
        pair = (lens[i], lens[i - 1])
        for m, kl in zip(masks, pair):
            m.copy_((torch.arange(Sk)[None, :] < torch.tensor(kl)[:, None]).int())
        torch.cuda.synchronize()
        for _ in range(4):
            for s, graph in zip(streams, graphs):
                with torch.cuda.stream(s):
                    graph.replay()
            with torch.cuda.stream(streams[2]):
                beside = binding.attention(qkv, cu, "global")
        torch.cuda.synchronize()
        assert torch.equal(beside, layer)
        for out, kl in zip(outs, pair):
            for b in range(B):
                n = kl[b]
                check(out[b], *reference(q[b], kv[b, :n, :H], kv[b, :n, H:], [Sq], [n]))
    assert binding._default(qkv.device).get_error() == 0
