"""One handle used by several threads at once, as include/mbert_attn.h allows for the
products and norms of any width."""
import ctypes
import threading

import pytest
import torch

from encoder_only_transformer_gb300 import binding
from test_linear import built, rnd  # noqa: F401

pytestmark = pytest.mark.gpu


def test_launches_of_threads_are_counted(built):  # noqa: F811
    """Every call's launch is in the handle's count, whatever the other threads do, and the
    results are those of one thread."""
    h = binding.Attention(torch.device("cuda", 0))
    lib, calls, threads = binding.load_library(), 3000, 4
    x, w = rnd(4, 64, seed=1).cuda(), rnd(32, 64, seed=2).cuda()
    nw = rnd(64, seed=3).cuda()
    want, (_, norm) = h.linear(x, w), h.residual_norm(x, None, nw)
    torch.cuda.synchronize()
    h.profile_read()
    wrong = []

    def run():
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            out, y = torch.zeros_like(want), torch.zeros_like(norm)
            a = binding.LinearArgs(x=x.data_ptr(), weight=w.data_ptr(), out=out.data_ptr(), x_row=64, weight_row=64,
                                   out_row=32, rows=4, inner=64, outer=32)
            b = binding.ResidualNormArgs(x=x.data_ptr(), weight=nw.data_ptr(), y=y.data_ptr(), x_row=64, y_row=64, rows=4,
                                         width=64, norm=2, residual_scale=1.0, eps=1e-5)
            stream.synchronize()
            for _ in range(calls):
                if (lib.mbert_attn_linear(h.handle, ctypes.byref(a), stream.cuda_stream) != 0
                        or lib.mbert_attn_residual_norm(h.handle, ctypes.byref(b), stream.cuda_stream) != 0):
                    wrong.append("status")
            stream.synchronize()
            if not torch.equal(out, want) or not torch.equal(y, norm):
                wrong.append("result")

    ts = [threading.Thread(target=run) for _ in range(threads)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert not wrong and h.get_error() == 0
    assert h.profile_read()[2] == 2 * calls * threads
    assert h.profile_read()[2] == 0
    h.close()
