// Rings of shared-memory slots with a barrier each, as plain arithmetic (host
// and device): entry t lies in slot t % stages, and the slot's barrier completes
// its phase t / stages when the entry has arrived.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define MBERT_HD __host__ __device__
#else
#define MBERT_HD
#endif

namespace mbert {

MBERT_HD constexpr uint32_t ring_slot(uint32_t t, uint32_t stages) { return t % stages; }
MBERT_HD constexpr uint32_t ring_parity(uint32_t t, uint32_t stages) { return (t / stages) & 1u; }

// Of `issued` entries, those from this one on may still be on their way: an
// entry is only issued into a slot whose last one has arrived and been read.
MBERT_HD constexpr uint32_t ring_pending(uint32_t issued, uint32_t stages)
{
    return issued > stages ? issued - stages : 0u;
}

}  // namespace mbert
