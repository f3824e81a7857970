"""Rows off 16 bytes in the norms around a block: what of memory is read for them
(csrc/pieces.h, on the CPU) and their results at a tensor's ends (GPU).

Tolerances as in test_residual_norm.py.
"""
import math
import os
import subprocess

import pytest
import torch

import test_residual_norm as N
from encoder_only_transformer_gb300 import binding
from test_residual_norm import TYPES, built, err0, rnd  # noqa: F401

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "encoder_only_transformer_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <vector>
#include "pieces.h"
using namespace mbert;

// a tensor of `rows` rows, `pitch` numbers apart, its first number `start` numbers behind a
// 16-byte boundary: every number of each row arrives once, and no byte is read that lies
// before the first number or behind the last
int main()
{
    long long seen = 0;
    for (int size : {2, 4})
        for (int width = 1; width <= 70; ++width)
            for (int pitch = width; pitch <= width + 9; ++pitch)
                for (int start = 0; start < 16 / size; ++start)
                    for (int rows = 1; rows <= 4; ++rows)
                        for (int row = 0; row < rows; ++row) {
                            const int lo = start * size, hi = lo + ((rows - 1) * pitch + width) * size;
                            const int at = lo + row * pitch * size, off = at % 16;
                            const Pieces p = pieces_of(off, width, size, at - lo, hi - at - width * size);
                            std::vector<int> byte(width * size, 0);
                            auto read = [&](int from, int n) {
                                if (from < lo || from + n > hi)
                                    return false;
                                for (int i = from; i < from + n; ++i)
                                    if (i >= at && i < at + width * size)
                                        ++byte[i - at];
                                return true;
                            };
                            bool ok = p.first >= 0 && p.head >= 0 && p.tail >= p.head && p.tail <= width &&
                                      p.head + width - p.tail <= 32;
                            for (int i = p.first; i < p.end; ++i)
                                ok = ok && read(at - off + 16 * i, 16);
                            for (int e = 0; e < width; ++e)
                                if (e < p.head || e >= p.tail)
                                    ok = ok && read(at + e * size, size);
                            for (int n : byte)
                                ok = ok && n == 1;
                            if (!ok)
                                return std::printf("size %d width %d pitch %d start %d row %d of %d\n", size, width, pitch,
                                                   start, row, rows), 1;
                            ++seen;
                        }
    std::printf("%lld rows\n", seen);
    return seen == 84000 ? 0 : 1;
}
"""


def test_nothing_outside_a_tensor_is_read(tmp_path):
    src, exe = tmp_path / "pieces.cpp", tmp_path / "pieces"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout + r.stderr


def placed(t, pitch, start):
    """t [T, D] on the GPU, rows `pitch` apart, NaN before, between and behind them."""
    buf = torch.full((t.shape[0] * pitch + start + 16,), math.nan, dtype=t.dtype, device="cuda")
    v = buf[start:start + t.shape[0] * pitch].view(t.shape[0], pitch)[:, :t.shape[1]]
    v.copy_(t)
    return v


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("T", [1, 2, 5])
def test_rows_at_a_tensors_ends(built, T, dtype):  # noqa: F811
    """Few rows, so that each is a tensor's first or last one or beside one, at every
    offset; a gate for each row, or for each of two sequences."""
    for D in (1, 2, 3, 5, 7, 8, 9, 15, 17, 31, 1001, 4099):
        x, branch = rnd(T, D, seed=1, dtype=dtype), rnd(T, D, seed=2, dtype=dtype)
        w, aw = rnd(D, seed=3, dtype=dtype, sc=0.2, at=1.0), rnd(D, seed=4, dtype=dtype, sc=0.2, at=1.0)
        rows, pair = rnd(T, D, seed=5, dtype=dtype), rnd(2, D, seed=6, dtype=dtype)
        cu = torch.tensor([0, T // 2, T], dtype=torch.int32)
        of = (torch.arange(T) >= T // 2).long()
        for start in (0, 1, 2, 3, 5, 7):
            pitch = D + start % 3
            a, b = placed(x, pitch, start), placed(branch, pitch + 1, (3 * start) % 8)
            for gate, seqs, full in ((rows, None, rows), (pair, cu.cuda(), pair[of])):
                h, y = binding.residual_norm(a, b, w.cuda(), None, aw.cuda(), None, placed(gate, D + 1, start), seqs,
                                             norm="rms", eps=1e-3)
                err0()
                rh, dh, ry, dy = N.reference(x, branch, w, None, aw, None, full, "rms", 1.0, 1e-3)
                N.check(h, rh, dh, f"h {D} {start}")
                N.check(y, ry, dy, f"y {D} {start}")
