"""The handle's count of launches under several threads (csrc/handle.h), on the CPU."""
import os
import subprocess

from encoder_only_transformer_gb300 import build

PROGRAM = r"""
#include <cstdio>
#include <thread>
#include <vector>
#include "handle.h"

int main()
{
    static mbert_attn h;
    std::vector<std::thread> threads;
    for (int t = 0; t < 4; ++t)
        threads.emplace_back([] {
            for (int i = 0; i < 500000; ++i)
                h.launches += 1;
        });
    for (auto &t : threads)
        t.join();
    const long long n = h.launches;
    std::printf("%lld\n", n);
    return n == 2000000 ? 0 : 1;
}
"""


def test_launches_of_threads_are_counted(tmp_path):
    src, exe = tmp_path / "counter.cpp", tmp_path / "counter"
    src.write_text(PROGRAM)
    cuda = os.path.join(os.path.dirname(os.path.dirname(build._nvcc())), "include")
    subprocess.run(["g++", "-std=c++17", "-O0", "-pthread", "-I", build.CSRC, "-I", build.INCLUDE, "-I", cuda, str(src),
                    "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout + r.stderr
