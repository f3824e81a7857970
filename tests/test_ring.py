"""What a CTA still has in flight when a wait has given up (csrc/ring.h), on the
CPU: a producer and readers of a ring that stop anywhere, then the drain's waits
against barriers that hold a phase bit, as the hardware's do.

A parity wait passes when the barrier's current phase is not the one waited for:
it says "arrived" for the phase before the current one, and it would also for an
older phase of the same parity, so the drain must ask for the last of each slot.
"""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "encoder_only_transformer_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <random>
#include <vector>
#include "ring.h"
using namespace mbert;

int main()
{
    std::mt19937 rng(5);
    long long runs = 0, flying = 0;
    for (uint32_t stages = 1; stages <= 4; ++stages)
        for (uint32_t limit = 0; limit <= 40; ++limit)
            for (int rep = 0; rep < 50; ++rep) {
                std::vector<uint32_t> done(stages, 0);      // completed phases of a slot's barrier
                std::vector<bool> landed;                   // by entry
                std::vector<uint32_t> in_flight;
                uint32_t issued = 0, seen = 0;
                auto passes = [&](uint32_t t) {             // what a parity wait sees now
                    return (done[ring_slot(t, stages)] & 1u) != ring_parity(t, stages);
                };
                auto land = [&](size_t i) {
                    const uint32_t t = in_flight[i];
                    in_flight.erase(in_flight.begin() + i);
                    landed[t] = true;
                    ++done[ring_slot(t, stages)];
                };
                // the loop of the kernels: an entry is issued once its slot's last one
                // has been read, which is after it has arrived; stop at a random point
                for (uint32_t step = 0; step < 200 && issued < limit; ++step) {
                    const uint32_t what = rng() % 3;
                    if (what == 0 && issued < seen + stages) {
                        landed.push_back(false);
                        in_flight.push_back(issued++);
                    } else if (what == 1 && !in_flight.empty()) {
                        land(rng() % in_flight.size());
                    } else if (what == 2 && seen < issued && passes(seen)) {
                        if (!landed[seen])
                            return std::printf("entry %u seen before it landed\n", seen), 1;
                        ++seen;
                    }
                }
                flying += in_flight.size();
                // the drain: each wait ends, as what is in flight lands at some time
                for (uint32_t t = ring_pending(issued, stages); t < issued; ++t)
                    while (!passes(t)) {
                        if (in_flight.empty())
                            return std::printf("stages %u, %u issued: the wait for %u never ends\n", stages, issued, t), 1;
                        land(rng() % in_flight.size());
                    }
                if (!in_flight.empty())
                    return std::printf("stages %u, %u issued, %u seen: %zu still in flight\n", stages, issued, seen,
                                       in_flight.size()), 1;
                ++runs;
            }
    std::printf("%lld runs, %lld in flight\n", runs, flying);
    return runs > 0 && flying > 1000 ? 0 : 1;
}
"""


def test_drain_waits_for_everything_in_flight(tmp_path):
    src, exe = tmp_path / "ring.cpp", tmp_path / "ring"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout + r.stderr
