"""Per-head norms over the whole range of the types (binding.qk_norm_rotary):
numbers whose squares fp32 does not hold, at both ends, alone and beside others.

Tolerances as in test_rotary.py: a head is scaled by a power of two, which is
exact, and eps by its square, two roundings on eps (one u on the factor, within
the 28 u taken there).
"""
import math

import pytest
import torch

from encoder_only_transformer_gb300 import binding
from test_rotary import TYPES, built, check_typed, freqs, reference, rnd  # noqa: F401

pytestmark = pytest.mark.gpu


def norm(x, w, kind, eps, rope=None, pos=None):
    return binding.qk_norm_rotary(x, None, w, None, rope, pos, norm=kind, eps=eps)[0]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("H,D,R", [(3, 64, 64), (2, 256, 64), (5, 80, 40), (1, 6, 2), (4, 130, 0)])
@pytest.mark.parametrize("exponent,eps", [
    (59, 1e-6), (61, 1e-6), (62, 0.0), (63, 1e-6), (64, 1e-12), (90, 1.0), (122, 1e-6), (125, 0.0),
    (-59, 0.0), (-70, 0.0), (-75, 1e-30), (-80, 1e-20), (-100, 0.0), (-120, 0.0), (-120, 1e-37), (-60, 1e-6)])
def test_any_magnitude(built, exponent, eps, H, D, R, kind, dtype):  # noqa: F811
    T = 5
    x = rnd(T, H, D, seed=D + exponent % 7, dtype="f32").clamp(-3.5, 3.5).to(TYPES[dtype])
    x = (x.double() * 2.0 ** exponent).to(TYPES[dtype])         # a power of two: exact
    w = (1 + 0.2 * rnd(D, seed=3, dtype="f32")).to(TYPES[dtype])
    pos = torch.arange(T) * 411
    f, amp = freqs(R, 10000.0)
    rope = binding.Rotary(R) if R else None
    got = norm(x.cuda(), w.cuda(), kind, eps, rope, pos.to(torch.int32).cuda() if R else None)
    check_typed(got, *reference(x, pos, f, amp, "half", kind, w, eps))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("exponent", [66, 124, -90])
def test_one_head_among_others(built, exponent, kind, dtype):  # noqa: F811
    """Heads beside one that is scaled keep their bits; one large number among
    small ones; in place."""
    T, H, D = 9, 7, 64
    x = rnd(T, H, D, seed=4, dtype=dtype)
    w = (1 + 0.2 * rnd(D, seed=3, dtype="f32")).to(TYPES[dtype]).cuda()
    eps = 0.0 if exponent < 0 else 1e-6
    want = norm(x.cuda(), w, kind, eps)
    y = x.clone()
    y[4, 2] = (x[4, 2].double() * 2.0 ** exponent).to(x.dtype)
    y[7, 0, 5] = 2.0 ** exponent
    got = norm(y.cuda(), w, kind, eps)
    same = torch.ones(T, H, dtype=torch.bool)
    same[4, 2] = same[7, 0] = False
    assert torch.equal(got.cpu()[same], want.cpu()[same])
    check_typed(got, *reference(y, None, [], 1.0, "half", kind, w, eps))
    mine = y.cuda()
    binding.qk_norm_rotary(mine, None, w, None, norm=kind, eps=eps, q_out=mine)
    assert torch.equal(mine, got)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("T,H", [(1, 1), (64, 24), (300, 5), (70, 1)])
def test_in_place_with_tiny_results(built, T, H, kind, dtype):  # noqa: F811
    """In place with weights so small that the results' own squares vanish: no
    head is normed twice; queries and keys at once, scaled heads in both."""
    x = rnd(T, 2 * H, 64, seed=T, dtype=dtype)
    x[::3, ::2] = (x[::3, ::2].double() * 2.0 ** 100).to(x.dtype)
    x[1::5] = (x[1::5].double() * 2.0 ** -120).to(x.dtype)
    w = (1 + 0.2 * rnd(64, seed=3, dtype="f32")).mul(2.0 ** -100).to(TYPES[dtype])
    pos = torch.arange(T, dtype=torch.int32).cuda()
    rope = binding.Rotary(32)
    mine = x.cuda()
    binding.qk_norm_rotary(mine[:, :H], mine[:, H:], w.cuda(), w.cuda(), rope, pos, norm=kind, eps=0.0,
                           q_out=mine[:, :H], k_out=mine[:, H:])
    f, amp = freqs(32, 10000.0)
    fine = (x != 0).any(-1) if kind == "rms" else (x != x[..., :1]).any(-1)     # (0/0 else)
    ref, tol = reference(x, pos, f, amp, "half", kind, w, 0.0)
    check_typed(mine.cpu()[fine], ref[fine], tol[fine])
    q, k = binding.qk_norm_rotary(x[:, :H].cuda(), x[:, H:].cuda(), w.cuda(), w.cuda(), rope, pos, norm=kind, eps=0.0)
    assert torch.equal(torch.cat([q, k], 1).cpu()[fine], mine.cpu()[fine])


@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_half_precision_ends(built, kind):  # noqa: F811
    """fp16's largest and smallest numbers: no square leaves fp32."""
    x = rnd(4, 2, 256, seed=8, dtype="f32").sign()
    w = torch.ones(256, dtype=torch.float16)
    for v in (65504.0, 2.0 ** -24):
        y = (x * v).half()
        check_typed(norm(y.cuda(), w.cuda(), kind, 0.0), *reference(y, None, [], 1.0, "half", kind, w, 0.0))


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_what_is_not_finite_stays_in_its_head(built, kind, dtype):  # noqa: F811
    x = rnd(3, 4, 64, seed=2, dtype=dtype)
    x[0, 1, 7], x[1, 2, 3], x[2, 0] = math.inf, math.nan, 0.0
    w = torch.ones(64, dtype=TYPES[dtype]).cuda()
    got = norm(x.cuda(), w, kind, 0.0).cpu()
    assert torch.isnan(got[0, 1, 7]) and torch.isnan(got[1, 2]).all() and torch.isnan(got[2, 0]).all()
    fine = torch.ones(3, 4, dtype=torch.bool)
    fine[0, 1] = fine[1, 2] = fine[2, 0] = False
    assert torch.isfinite(got[fine]).all()
    assert (norm(x.cuda(), w, kind, 1e-6).cpu()[2, 0] == 0).all()
