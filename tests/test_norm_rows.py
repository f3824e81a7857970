"""A row of the norms around a block has the same bits whatever rows are beside it and
however many: crews of every size sum in one order."""
import ctypes

import pytest
import torch

from encoder_only_transformer_gb300 import binding
from test_residual_norm import TYPES, built, err0, rnd  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("D", [768, 1024, 1536, 1544, 2048, 2056, 2304, 3000, 4096, 6152, 8192, 8200, 16384])
def test_bits_of_a_row_do_not_go_by_the_rows_beside_it(built, D, kind, dtype):  # noqa: F811
    T, part = 1600, 200
    x, branch, gate = (rnd(T, D, seed=i, dtype=dtype).cuda() for i in (1, 2, 3))
    w, b, aw = (rnd(D, seed=i, dtype=dtype, sc=0.2, at=at).cuda() for i, at in ((4, 1.0), (5, 0.0), (6, 1.0)))
    x[::40] *= 2.0 ** 10 if dtype == "f16" else 2.0 ** 66        # scaled a second time (f16: an outlier)
    call = lambda r: binding.residual_norm(x[r], branch[r], w, b, aw, None, gate[r], norm=kind)
    h, y = call(slice(0, T))
    for at in range(0, T, part):
        r = slice(at, at + part)
        hp, yp = call(r)
        assert torch.equal(h[r], hp) and torch.equal(y[r], yp), at
    one = slice(777, 778)
    hp, yp = call(one)
    assert torch.equal(h[one], hp) and torch.equal(y[one], yp)
    err0()


def test_number_of_sequences_is_bounded(built):  # noqa: F811
    """As many sequences as rows may be there at most; more (indexes beyond 32 bits on the
    device) are refused on the host."""
    x, gate = rnd(4, 64, seed=1).cuda(), rnd(4, 64, seed=2).cuda()
    cu, out = torch.tensor([0, 1, 2, 3, 4], dtype=torch.int32).cuda(), torch.zeros_like(x)
    lib, h = binding.load_library(), binding._default(x.device).handle
    a = binding.ResidualNormArgs(x=x.data_ptr(), branch=x.data_ptr(), gate=gate.data_ptr(), h=out.data_ptr(), x_row=64,
                                 branch_row=64, gate_row=64, h_row=64, rows=4, width=64, norm=1, gate_kind=3,
                                 cu_seqlens=cu.data_ptr(), n_seqs=4, residual_scale=1.0, eps=1e-5)
    stream = torch.cuda.current_stream().cuda_stream
    assert lib.mbert_attn_residual_norm(h, ctypes.byref(a), stream) == 0
    for n in (2 ** 31 - 1, 2 ** 31 - 1024, 0, -1):
        a.n_seqs = n
        assert lib.mbert_attn_residual_norm(h, ctypes.byref(a), stream) == -1, n
    err0()
