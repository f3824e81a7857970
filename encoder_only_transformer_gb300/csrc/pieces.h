// How a row off 16 bytes is copied by aligned pieces of 16 bytes, as plain arithmetic
// (host and device).
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define MBERT_HD __host__ __device__
#else
#define MBERT_HD
#endif

namespace mbert {

// A row of `width` numbers of `size` bytes each, `off` bytes behind a 16-byte boundary: pieces
// first .. end - 1, counted from that boundary, are copied whole, numbers 0 .. head - 1 and
// tail .. width - 1 one by one.
struct Pieces {
    int first, end, head, tail;
};

// The pieces at either end hold bytes beside the row.  Those of the row's tensor, `before` the
// row's first number and `behind` its last, may be read; a piece that holds others, which may
// be nobody's, is not, and its numbers come one by one: 14 at most.
MBERT_HD constexpr Pieces pieces_of(int off, int width, int size, long long before, long long behind)
{
    const int bytes = off + width * size, end = (bytes + 15) / 16;
    Pieces p = {before < off ? 1 : 0, behind < 16 * end - bytes ? end - 1 : end, 0, width};
    if (p.first == 1)
        p.head = (16 - off) / size < width ? (16 - off) / size : width;
    if (p.end < end)
        p.tail = (16 * p.end - off) / size > p.head ? (16 * p.end - off) / size : p.head;
    return p;
}

}  // namespace mbert
