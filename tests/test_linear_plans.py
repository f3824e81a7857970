"""Every form of the products' kernels by calls that take it: sizes over a grid are asked
for their plan (binding.Attention.linear_plan), and the cheapest call of each form is
checked with all parts of its epilogue, rows off 16 bytes, in place, ragged groups and
bad offsets against the formula in 64 bits.

Tolerances as in test_linear.py.
"""
import math
import random

import pytest
import torch

import test_linear as L
from encoder_only_transformer_gb300 import binding
from test_linear import TYPES, built, err0, rnd  # noqa: F401

ROWS = (1, 9, 17, 40, 70, 120, 130, 200, 300, 520, 900, 1500, 2100, 3000, 5000, 9000)
INNER = (8, 72, 200, 520, 1000, 2048, 4096)
OUTER = (1, 33, 130, 200, 500, 1100, 2300, 5000, 9000)
EXPERTS = (3, 8, 20, 50)
BEHIND = 3              # rows behind the last expert's

# (kernel, columns of a unit or rows of a tile, CTAs that share the inner dimension)
FORMS = [("many", 128, 0), ("many", 256, 0)] + [("few", t, s) for t in (16, 32, 64) for s in (1, 2, 4, 8)] + \
    [("few", 128, 1)]


def test_plan_refusals_without_device(built):  # noqa: F811
    a = binding.LinearArgs(rows=1, inner=8, outer=8)
    assert binding.load_library().mbert_attn_linear_plan(None, a, (L.ctypes.c_int32 * 4)()) == -1


@pytest.fixture(scope="module")
def calls(built):  # noqa: F811
    """{(kernel, size, split, gated): {pieces: the cheapest (rows, inner, outer, experts)}} of
    plain products and of grouped ones; of the kernel for many rows also the cheapest of
    several steps ("long")."""
    h = binding._default(torch.device("cuda", 0))
    found = [{}, {}]
    for T in ROWS:
        for K in INNER:
            for N in OUTER:
                for E in (0,) + EXPERTS:
                    for gated in (False, True):
                        p = h.linear_plan(T, K, N, "gelu", gated, E)
                        sides = 2 if gated else 1
                        cost = T * K * N * sides + 50 * T * N + max(E, 1) * K * N * sides
                        if p[0] == "many":
                            keys = [((*p, 0, gated), 0)] + ([((*p, 0, gated), "long")] if K >= 200 else [])
                        else:
                            keys = [((p[0], p[1], p[3], gated), p[2])]
                        for key, pieces in keys:
                            forms = found[E > 0].setdefault(key, {})
                            if pieces not in forms or cost < forms[pieces][0]:
                                forms[pieces] = (cost, (T, K, N, E))
    return [{k: {p: c for p, (_, c) in v.items()} for k, v in kind.items()} for kind in found]


@pytest.mark.gpu
def test_every_form_is_met(calls):
    for form in FORMS:
        for gated in (False, True):
            assert (*form, gated) in calls[0] or (*form, gated) in calls[1], (form, gated)
    pieces = set()
    for kind in calls:
        for key, forms in kind.items():
            assert key[:3] in FORMS, key
            pieces |= set(forms) if key[0] == "few" else set()
    assert pieces == {1, 2, 3, 4}


def chosen(calls, form, gated, dtype):
    """The form's calls with every size of pieces for fp16, the first of them for bf16."""
    forms = calls.get((*form, gated), {})
    keys = sorted(forms, key=str)
    return [forms[k] for k in (keys if dtype == "f16" or form[0] == "many" else keys[:1])]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("form", FORMS, ids=lambda f: "-".join(map(str, f)))
def test_plain_products(calls, form, gated, dtype):
    for T, K, N, _ in chosen(calls[0], form, gated, dtype):
        W = 2 * N if gated else N
        x, w = rnd(T, K, seed=T, dtype=dtype).cuda(), rnd(W, K, seed=K, dtype=dtype, sc=K ** -0.5).cuda()
        b, r = rnd(W, seed=N, dtype=dtype, sc=0.5).cuda(), rnd(T, N, seed=3, dtype=dtype).cuda()
        want = binding.linear(x, w, b, "gelu", gated, r)
        err0()
        y, t = L.product(x, w, b, "gelu", gated)
        y, t = L.finish(y, t, TYPES[dtype], None, r)
        L.check(want, y.cpu(), t.cpu())
        # results and residuals off 16 bytes and in place: the same bits, nothing beside them
        for pitch, start in ((N + 1, 1), (N + 7 - (N + 7) % 8 + 8, 0)):
            res = L.strided(r.cpu(), pitch, start)[0]
            out, buf = L.strided(torch.zeros(T, N, dtype=TYPES[dtype]), pitch, start)
            binding.linear(x, w, b, "gelu", gated, res, out=out)
            assert torch.equal(out, want), (pitch, start)
            out.fill_(math.nan)
            assert buf.isnan().all()
            binding.linear(x, w, b, "gelu", gated, res, out=res)
            assert torch.equal(res, want), (pitch, start)
        # a row of NaN and infinities leaves the others as they were
        x[T // 2] = math.nan
        x[T // 2, 0] = math.inf
        other = binding.linear(x, w, b, "gelu", gated, r)
        assert other[T // 2].isnan().all()
        other[T // 2] = want[T // 2]
        assert torch.equal(other, want)
        err0()


def ragged(T, E, seed):
    """E groups of T rows: some empty, some of one row, some large."""
    r = random.Random(seed)
    share = [r.choice((0.0, 0.02, 1.0, 1.0, 3.0)) for _ in range(E - 1)] + [1.0]
    n = [int(T * s / sum(share)) for s in share]
    n[r.randrange(E)] += T - sum(n)
    return n


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("form", FORMS, ids=lambda f: "-".join(map(str, f)))
def test_ragged_groups(calls, form, gated, dtype):
    for T, K, N, E in chosen(calls[1], form, gated, dtype):
        behind = min(BEHIND, T - 1)
        got, args = L.run_experts(ragged(T - behind, E, T + K), K, N, dtype, "gelu", True, gated, True, T, behind)
        # offsets out of order or beyond the rows: reported, nothing written
        out, good = torch.full_like(got, 3.0), args[2].cpu()
        for bad in (torch.cat([good[:1] + 1, good[1:]]), torch.cat([good[:-1], good[-1:] + T]),
                    torch.cat([good[:1], good[1:2] - T - 1, good[2:]])):
            binding.expert_linear(*args[:2], bad.to(torch.int32).cuda(), *args[3:], out=out)
            torch.cuda.synchronize()
            assert binding._default(out.device).get_error() == -4 and (out == 3.0).all()
        again = binding.expert_linear(*args, out=out)
        err0()
        assert torch.equal(again, got)
