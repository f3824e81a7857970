// The norms after one block and before the next, with the gate and the residual
// between them, in one pass (sm_103a): for every row t
//     h_t = alpha x_t + g_t P(branch_t),   y_t = N(h_t)
// P and N: LayerNorm, (v - mean) / sqrt(var + eps) w + b with the population
// variance, or RMS, v / sqrt(mean(v^2) + eps) w + b; either may be absent, and so may
// the branch (y = N(x)) and the gate (of a channel, a row, or a row's sequence).
// bf16, fp16 or fp32; everything between loading and storing is fp32, y is of the
// h that has not been rounded.
//
// Bound by HBM: x and branch in, h and y out.  A crew takes a row (or, of short rows,
// as many as a warp has lanes for): a warp up to 1536 numbers (1024 in fp32), 32 or
// 48 a lane in registers, and up to 16 warps beyond, which add their sums up in shared
// memory.  Rows come by cp.async into a ring of shared-memory slots of the crew's own,
// and a slot is filled again as soon as h is in registers: the loads of the next rows run
// while a row goes through its sums, which are chains of shuffles.  Every thread copies
// the vectors that it will read, so it waits for its own copies only; the same ring with
// bulk copies and barriers took 73 us where this takes 69 (65536 x 768 bf16, 403 MB, 5.8
// TB/s), rows loaded into registers 84.  A norm's statistics are sums over the registers
// in pairs, the LayerNorm's in two passes (mean, then squares about it).  Weights come
// from L1 or L2 for each row.  Rows off 16 bytes come as the 16-byte pieces they lie in
// (see pieces.h for those at a tensor's ends) and are taken number by number.
//
// Where the squares add up to what fp32 does not hold (or, beside a small eps, to
// what it holds badly), the row is scaled by a power of two first: see norm_row.
#include <algorithm>

#include "internal.h"
#include "pieces.h"
#include "residual_norm.h"
#include "linear.cuh"

namespace mbert {
namespace {

constexpr int kMostWarps = 16;      // of a crew
constexpr int kCrewNumbers = 16;    // numbers of a row a lane holds in a crew of several warps, or, with
                                    // all 16, up to twice as many
static_assert(kResidualNormMaxWidth == 32 * kMostWarps * 2 * kCrewNumbers, "widest rows");
constexpr int kWarpCrews = 4;       // crews of one warp in a block
constexpr int kMostSlots = 8;
// Few numbers a lane leave registers for a norm's bias and a gate of channels to be on
// their way during the sums too, as the weights are (4099 x 8192 fp32 with all of them, a
// crew of 16 warps alone on its SM: 110 us against 142).
constexpr bool early(bool vectors, int numbers) { return vectors && numbers <= kCrewNumbers; }

// Registers of a kernel: the numbers that a lane holds, what is on its way to them as it
// is in memory, and the rest.  With what the compiler takes by itself (126 for 24
// numbers) too few warps share an SM.
constexpr int most_registers(bool vectors, int numbers, int bytes)
{
    return (numbers + (early(vectors, numbers) ? 3 : 1) * numbers * bytes / 4 + 51) / 8 * 8;
}
static_assert(most_registers(true, kCrewNumbers, 4) * 32 * kMostWarps <= 65536 &&
              most_registers(true, 2 * kCrewNumbers, 4) * 32 * kMostWarps <= 65536, "a crew on an SM");

// The numbers of a row that a lane holds: kVecs vectors of 16 bytes, the lanes' side
// by side and a warp's in one piece, or (of rows off 16 bytes) as many single numbers,
// again side by side.  Numbers behind the row's end are 0.
template <int kType, bool kVectors, int kVecs>
struct Row {
    static constexpr int kBytes = kType == MBERT_F32 ? 4 : 2;
    static constexpr int kN = 16 / kBytes;
    int first, width;           // the first of them, the row's end

    __device__ Row(int warp, int lane, int w)
        : first(kVectors ? (warp * 32 * kVecs + lane) * kN : warp * 32 * kVecs * kN + lane), width(w)
    {
    }
    // number e of vector j is number first + at(j, e) of the row
    static constexpr __device__ int at(int j, int e) { return kVectors ? 32 * kN * j + e : 32 * (kN * j + e); }
    __device__ bool in(int j, int e) const { return first + at(j, kVectors ? 0 : e) < width; }

    static constexpr int kPairs = kN / 2;

    __device__ static void unpack(const uint4 &x, uint64_t (&v)[kPairs])
    {
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int e = 0; e < kPairs; ++e) {
            if constexpr (kType == MBERT_F32)
                v[e] = f2(__uint_as_float(w[2 * e]), __uint_as_float(w[2 * e + 1]));
            else
                v[e] = unpack2<kType == MBERT_F16>(w[e]);
        }
    }

    // vector j from global memory, as it is
    __device__ uint4 load_raw(const void *p, int j) const
    {
        const char *q = static_cast<const char *>(p) + first * kBytes;
        return in(j, 0) ? *reinterpret_cast<const uint4 *>(q + at(j, 0) * kBytes) : make_uint4(0, 0, 0, 0);
    }

    // vector j, from global memory
    __device__ void load(const void *p, int j, uint64_t (&v)[kPairs]) const
    {
        const char *q = static_cast<const char *>(p) + first * kBytes;
        if constexpr (kVectors) {
            unpack(load_raw(p, j), v);
        } else {
            single(j, v, [&](int offset) {
                if constexpr (kType == MBERT_F32)
                    return *reinterpret_cast<const float *>(q + offset);
                else
                    return load16<kType == MBERT_F16>(q + offset, 0);
            });
        }
    }

    // from a row in shared memory
    __device__ void load_shared(uint32_t row, int j, uint64_t (&v)[kPairs]) const
    {
        const uint32_t q = row + first * kBytes;
        if constexpr (kVectors) {
            uint4 x = make_uint4(0, 0, 0, 0);
            if (in(j, 0))
                asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                             : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(q + at(j, 0) * kBytes) : "memory");
            unpack(x, v);
        } else {
            single(j, v, [&](int offset) {
                if constexpr (kType == MBERT_F32) {
                    uint32_t x;
                    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(x) : "r"(q + offset) : "memory");
                    return __uint_as_float(x);
                } else {
                    uint16_t x;
                    asm volatile("ld.shared.b16 %0, [%1];" : "=h"(x) : "r"(q + offset) : "memory");
                    float lo, hi;
                    f2_split(unpack2<kType == MBERT_F16>(x), lo, hi);
                    return lo;
                }
            });
        }
    }

    __device__ void store(char *p, int j, const uint64_t (&v)[kPairs]) const
    {
        char *q = p + first * kBytes;
        float f[kN];
#pragma unroll
        for (int e = 0; e < kPairs; ++e)
            f2_split(v[e], f[2 * e], f[2 * e + 1]);
        if constexpr (kVectors) {
            if (!in(j, 0))
                return;
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if constexpr (kType == MBERT_F32)
                    w[e] = __float_as_uint(f[e]);
                else
                    w[e] = pack2<kType == MBERT_F16>(f[2 * e], f[2 * e + 1]);
            }
            *reinterpret_cast<uint4 *>(q + at(j, 0) * kBytes) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
#pragma unroll
            for (int e = 0; e < kN; ++e) {
                if (!in(j, e))
                    continue;
                if constexpr (kType == MBERT_F32)
                    *reinterpret_cast<float *>(q + at(j, e) * kBytes) = f[e];
                else
                    *reinterpret_cast<uint16_t *>(q + at(j, e) * kBytes) =
                        static_cast<uint16_t>(pack2<kType == MBERT_F16>(f[e], 0.f));
            }
        }
    }

    // does every lane hold numbers of the row only?
    __device__ bool full(int warps) const { return width == warps * 32 * kVecs * kN; }

    // 0 behind the row's end
    __device__ void clear_behind(int j, uint64_t (&v)[kPairs]) const
    {
        if constexpr (kVectors) {
            if (!in(j, 0))
#pragma unroll
                for (int e = 0; e < kPairs; ++e)
                    v[e] = 0;
        } else {
#pragma unroll
            for (int e = 0; e < kPairs; ++e) {
                float lo, hi;
                f2_split(v[e], lo, hi);
                v[e] = f2(in(j, 2 * e) ? lo : 0.f, in(j, 2 * e + 1) ? hi : 0.f);
            }
        }
    }

private:
    template <typename F>
    __device__ void single(int j, uint64_t (&v)[kPairs], F &&number) const
    {
#pragma unroll
        for (int e = 0; e < kPairs; ++e) {
            float lo = 0.f, hi = 0.f;
            if (in(j, 2 * e))
                lo = number(at(j, 2 * e) * kBytes);
            if (in(j, 2 * e + 1))
                hi = number(at(j, 2 * e + 1) * kBytes);
            v[e] = f2(lo, hi);
        }
    }
};

// The lanes of a row: `lanes` of a warp, or `warps` whole warps of a block.
struct Team {
    int lanes, warps;
    float *scratch;     // [2][32]
    int turn;

    template <typename Op>
    __device__ float all(float v, Op op)
    {
        if (lanes == 32) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
        } else {
            for (int o = lanes >> 1; o > 0; o >>= 1)
                v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
        }
        return warps > 1 ? join(v, 32, op) : v;
    }
    static __device__ float add(uint64_t v)
    {
        float lo, hi;
        f2_split(v, lo, hi);
        return lo + hi;
    }
    __device__ float sum(uint64_t v)
    {
        return all(add(v), [](float x, float y) { return x + y; });
    }
    // sums u of each warp's first half of numbers, v of the second, added up like those of
    // twice as many warps
    __device__ float sum(uint64_t u, uint64_t v)
    {
        const bool upper = threadIdx.x & 16;
        const float a = add(u), b = add(v);
        // lanes 0 - 15 go on with u, the others with v
        float x = (upper ? b : a) + __shfl_xor_sync(0xffffffffu, upper ? a : b, 16);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1)
            x += __shfl_xor_sync(0xffffffffu, x, o);
        return join(x, 16, [](float y, float z) { return y + z; });
    }
    __device__ float most(float v) { return all(v, [](float x, float y) { return fmaxf(x, y); }); }

private:
    // v of every group of `width` lanes of the crew
    template <typename Op>
    __device__ float join(float v, int width, Op op)
    {
        // two places in turn, so that one barrier a sum will do
        float *s = scratch + (turn ^= 1) * 32;
        const int lane = threadIdx.x & 31;
        if (lane % width == 0)
            s[threadIdx.x / width] = v;
        __syncthreads();
        v = lane < 32 / width * warps ? s[lane] : 0.f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
        return v;
    }
};

// v[] of a row -> its norm times w plus b.  Called by all lanes of a warp.
//
// LayerNorm works on half of each number, so that no difference from the mean
// overflows (the sum of numbers times sum_scale, at most 1 / width, does not either),
// and with eps / 4.  Squares that add up to more than 2^126, or, beside an eps below
// 2^-40, to less than 2^-90 (those that round to nothing are then off by 2^-45 of the
// sum at most), are taken again of the row times a power of two that brings its
// largest number to 1 .. 2, or as near as keeps eps times its square at 2^100.
template <int kType, bool kVectors, int kVecs, bool kLayer, bool kHalves>
__device__ __forceinline__ void norm_row(const ResidualNormArgs &a, const Row<kType, kVectors, kVecs> &at,
                                         uint64_t (&v)[kVecs][Row<kType, kVectors, kVecs>::kPairs], const void *w,
                                         const void *b, Team &team)
{
    constexpr int kPairs = Row<kType, kVectors, kVecs>::kPairs;
    auto each = [&](auto &&f) {
#pragma unroll
        for (int j = 0; j < kVecs; ++j)
#pragma unroll
            for (int e = 0; e < kPairs; ++e)
                f(v[j][e]);
    };
    // two chains of sums, or two for each half of a lane's vectors (see launch)
    auto total = [&](auto &&f) {
        uint64_t s[2][2] = {};
#pragma unroll
        for (int j = 0; j < kVecs; ++j)
#pragma unroll
            for (int e = 0; e < kPairs; ++e) {
                uint64_t &x = s[kHalves && j >= kVecs / 2][e & 1];
                x = f(v[j][e], x);
            }
        const uint64_t u = fadd2p(s[0][0], s[0][1]);
        if constexpr (kHalves)
            return team.sum(u, fadd2p(s[1][0], s[1][1]));
        else
            return team.sum(u);
    };
    auto half_mean = [&] {
        const uint64_t scale = bc2(a.sum_scale);
        return total([&](uint64_t x, uint64_t s) { return ffma2(x, scale, s); }) * a.half_mean_scale;
    };
    auto centre = [&](float half, float mean) {
        each([&](uint64_t &x) { x = ffma2(x, bc2(half), bc2(-mean)); });
        if (!at.full(team.warps))
#pragma unroll
            for (int j = 0; j < kVecs; ++j)
                at.clear_behind(j, v[j]);
    };
    auto squares = [&] { return total([](uint64_t x, uint64_t s) { return ffma2(x, x, s); }); };
    // the weights are on their way during the sums
    constexpr bool kEarly = early(kVectors, kVecs * 2 * kPairs);
    uint4 wr[kVectors ? kVecs : 1], br[kEarly ? kVecs : 1];
    if constexpr (kVectors) {
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
            wr[j] = at.load_raw(w, j);
            if constexpr (kEarly)
                br[j] = b ? at.load_raw(b, j) : make_uint4(0, 0, 0, 0);
        }
    }
    float eps = a.eps;
    if constexpr (kLayer) {
        centre(0.5f, half_mean());
        eps *= 0.25f;
    }
    float q = squares();
    bool again = !(q >= a.least_squares && q <= 0x1p126f);      // (NaN too, which stay)
    if (__any_sync(0xffffffffu, again)) {
        float m = 0.f;
        each([&](uint64_t &x) {
            float lo, hi;
            f2_split(x, lo, hi);
            m = fmaxf(m, fmaxf(fabsf(lo), fabsf(hi)));
        });
        m = team.most(m);
        again = again && m > 0.f && m < INFINITY;
        const int k = min(127 - (__float_as_int(m) >> 23), a.most_scale);
        const float up = again ? __int_as_float((max(k, -126) + 127) << 23) : 1.f;
        eps = eps * up * up;
        each([&](uint64_t &x) { x = fmul2(x, bc2(up)); });
        if constexpr (kLayer) {
            const float mean = half_mean();
            centre(again ? 0.5f : 1.f, again ? mean : 0.f);
            eps *= again ? 0.25f : 1.f;
        }
        const float sum = squares();
        q = again ? sum : q;
    }
    const uint64_t r = bc2(rsqrtf(fmaf(q, a.inv_width, eps)));
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
        uint64_t wv[kPairs], bv[kPairs];
        if constexpr (kVectors)
            at.unpack(wr[j], wv);
        else
            at.load(w, j, wv);
        if (b) {
            if constexpr (kEarly)
                at.unpack(br[j], bv);
            else
                at.load(b, j, bv);
#pragma unroll
            for (int e = 0; e < kPairs; ++e)
                v[j][e] = ffma2(fmul2(v[j][e], r), wv[e], bv[e]);
        } else {
#pragma unroll
            for (int e = 0; e < kPairs; ++e)
                v[j][e] = fmul2(fmul2(v[j][e], r), wv[e]);
        }
    }
}

// 16 bytes to shared memory, in the calling thread's current group of copies
__device__ __forceinline__ void copy_async(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;"
                 :: "r"(dst), "l"(reinterpret_cast<uint64_t>(src)) : "memory");
}

// a number of 2 or 4 bytes to shared memory
template <int kBytes>
__device__ __forceinline__ void copy_number(uint32_t dst, const char *src)
{
    if constexpr (kBytes == 4)
        asm volatile("st.shared.b32 [%0], %1;" :: "r"(dst), "r"(*reinterpret_cast<const uint32_t *>(src)) : "memory");
    else
        asm volatile("st.shared.b16 [%0], %1;" :: "r"(dst), "h"(*reinterpret_cast<const uint16_t *>(src)) : "memory");
}

__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// all but the `n` newest groups have landed
__device__ __forceinline__ void copy_wait(int n)
{
    switch (n) {
    case 0: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
    case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
    case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
    case 3: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
    case 4: asm volatile("cp.async.wait_group 4;" ::: "memory"); break;
    case 5: asm volatile("cp.async.wait_group 5;" ::: "memory"); break;
    case 6: asm volatile("cp.async.wait_group 6;" ::: "memory"); break;
    default: asm volatile("cp.async.wait_group 7;" ::: "memory"); break;
    }
}

// The sequence of row t: the last that begins there or before.  `seq` is the one of
// an earlier row.
__device__ __forceinline__ int sequence_of(const int32_t *cu, int n, long long t, int seq)
{
    if (seq + 1 >= n || cu[seq + 1] > t)
        return seq;
    int hi = n;
    while (hi - seq > 1) {
        const int mid = seq + ((hi - seq) >> 1);
        (cu[mid] <= t ? seq : hi) = mid;
    }
    return seq;
}

// kVecs 16-byte vectors a lane.
template <int kType, bool kVectors, int kVecs, bool kLayer, bool kHalves>
__global__ void __maxnreg__(most_registers(kVectors, kVecs * (kType == MBERT_F32 ? 4 : 8), kType == MBERT_F32 ? 4 : 2))
residual_norm_kernel(const ResidualNormArgs a)
{
    using At = Row<kType, kVectors, kVecs>;
    constexpr int kPairs = At::kPairs, kBytes = At::kBytes;
    constexpr bool kEarly = early(kVectors, kVecs * 2 * kPairs);
    extern __shared__ __align__(16) uint8_t smem_raw[];
    __shared__ float scratch[64];
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool one_warp = a.warps == 1;
    Team team{a.lanes, a.warps, scratch, 0};
    // the crew: its rows side by side, this thread's row among them and place in the row
    const int beside = 32 / a.lanes;
    const At at(one_warp ? 0 : warp, lane & (a.lanes - 1), a.width);
    const int mine = lane / a.lanes;

    bool bad = false;
    if (a.cu) {
        for (int g = threadIdx.x; g <= a.n_seqs; g += blockDim.x) {
            const int x = a.cu[g];
            bad |= g == 0 ? x != 0 : x < a.cu[g - 1];
            bad |= g == a.n_seqs && x > a.rows;
        }
        bad = __syncthreads_or(bad) != 0;
        if (bad && blockIdx.x == 0 && threadIdx.x == 0)
            atomicOr(a.err, kErrBadCu);
    }
    const unsigned all_rows = static_cast<unsigned>(a.rows);
    const unsigned rows = static_cast<unsigned>(bad ? 0 : a.cu ? a.cu[a.n_seqs] : a.rows);
    // this thread's first row and the rows from round to round (a row and a stride stay
    // below 2^32: there are at most 2^31 - 1024 rows, and a row for every lane)
    const unsigned row0 = (one_warp ? blockIdx.x * kWarpCrews + warp : blockIdx.x) * beside;
    const unsigned stride = (one_warp ? gridDim.x * kWarpCrews : gridDim.x) * beside;

    // The ring: a slot holds the crew's rows of x, of the branch and of the gate.
    const bool gate_rows = a.gate && !a.gate_channels;
    const uint32_t tensor_bytes = beside * a.row_bytes, slot_bytes = a.tensors * tensor_bytes;
    const uint32_t slot0 = smem_u32(smem_raw) + (one_warp ? warp * a.slots * slot_bytes : 0) + mine * a.row_bytes;
    const uint32_t end = slot0 + a.slots * slot_bytes;
    int seq = 0;
    auto row_of = [&](const void *p, long long pitch, unsigned row) {
        return static_cast<const char *>(p) + row * pitch * kBytes;
    };
    // the row of `gate` that row `row` takes; s is the sequence of an earlier row
    auto gate_row = [&](unsigned row, int &s) {
        return a.cu ? static_cast<unsigned>(s = sequence_of(a.cu, a.n_seqs, static_cast<int>(row), s)) : row;
    };
    // Whole vectors: every thread copies the ones that it will read, so nothing but its
    // own copies has to be waited for.  Single numbers: the crew copies the 16-byte pieces
    // of memory that the row lies in (its neighbours' numbers at either end are not looked
    // at), and waits for each other.  `row` of `count`: nothing is read before a tensor's
    // first number or behind its last (9456 x 92 bf16, gates of 12 sequences, 10.7 us
    // against 9.6 with whole pieces everywhere; 707 x 9647 fp16 32.3 / 31.3).
    auto copy = [&](uint32_t dst, const void *tensor, long long pitch, unsigned row, unsigned count) {
        const char *p = row_of(tensor, pitch, row);
        if constexpr (kVectors) {
#pragma unroll
            for (int j = 0; j < kVecs; ++j)
                if (at.in(j, 0))
                    copy_async(dst + (at.first + At::at(j, 0)) * kBytes, p + (at.first + At::at(j, 0)) * kBytes);
        } else {
            const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p) & 15);
            const Pieces s = pieces_of(off, a.width, kBytes, row * pitch * kBytes, (count - 1 - row) * pitch * kBytes);
            const int t = one_warp ? lane : threadIdx.x;
            for (int i = s.first + t; i < s.end; i += 32 * a.warps)
                copy_async(dst + 16 * i, p - off + 16 * i);
            const int e = t < s.head ? t : s.tail + t - s.head;
            if (e < a.width)
                copy_number<kBytes>(dst + off + e * kBytes, p + e * kBytes);
        }
    };
    unsigned fill_row = row0 + mine;
    uint32_t fill = slot0;
    auto refill = [&] {
        if (fill_row < rows) {
            copy(fill, a.x, a.x_row, fill_row, all_rows);
            if (a.branch)
                copy(fill + tensor_bytes, a.branch, a.branch_row, fill_row, all_rows);
            if (gate_rows)
                copy(fill + 2 * tensor_bytes, a.gate, a.gate_row, gate_row(fill_row, seq), a.cu ? a.n_seqs : all_rows);
        }
        copy_commit();      // one group a slot, if an empty one
        fill_row += stride;
        fill = fill + slot_bytes == end ? slot0 : fill + slot_bytes;
    };
    for (int s = 0; s < a.slots; ++s)
        refill();

    uint32_t from = slot0;
    int read_seq = 0;
    for (unsigned base = row0; base < rows; base += stride) {
        const unsigned row = base + mine;
        const bool on = row < rows;
        copy_wait(a.slots - 1);
        if constexpr (!kVectors)
            one_warp ? __syncwarp() : __syncthreads();
        uint64_t v[kVecs][kPairs];
        // f(j, numbers) for the row at `p`, which is in the slot as tensor i
        auto take = [&](int i, const char *p, auto &&f) {
            uint64_t w[kPairs];
            const uint32_t s = from + i * tensor_bytes + (kVectors ? 0 : static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p) & 15));
#pragma unroll
            for (int j = 0; j < kVecs; ++j) {
                at.load_shared(s, j, w);
                f(j, w);
            }
        };
        auto keep = [&](int j, const uint64_t (&w)[kPairs]) {
#pragma unroll
            for (int e = 0; e < kPairs; ++e)
                v[j][e] = w[e];
        };
        auto store = [&](void *p, long long pitch) {
            if (!on)
                return;
            char *q = static_cast<char *>(p) + row * pitch * kBytes;
#pragma unroll
            for (int j = 0; j < kVecs; ++j)
                at.store(q, j, v[j]);
        };
        uint4 gr[kEarly ? kVecs : 1];
        if constexpr (kEarly)
            if (a.gate_channels)
#pragma unroll
                for (int j = 0; j < kVecs; ++j)
                    gr[j] = at.load_raw(a.gate, j);
        if (a.branch) {
            take(1, row_of(a.branch, a.branch_row, row), keep);
            if (a.after_weight)
                norm_row<kType, kVectors, kVecs, kLayer, kHalves>(a, at, v, a.after_weight, a.after_bias, team);
            auto times = [&](int j, const uint64_t (&w)[kPairs]) {
#pragma unroll
                for (int e = 0; e < kPairs; ++e)
                    v[j][e] = fmul2(v[j][e], w[e]);
            };
            if (gate_rows) {
                take(2, kVectors ? nullptr : row_of(a.gate, a.gate_row, gate_row(on ? row : 0, read_seq)), times);
            } else if (a.gate) {
                uint64_t w[kPairs];
#pragma unroll
                for (int j = 0; j < kVecs; ++j) {
                    if constexpr (kEarly)
                        at.unpack(gr[j], w);
                    else
                        at.load(a.gate, j, w);
                    times(j, w);
                }
            }
            take(0, row_of(a.x, a.x_row, row), [&](int j, const uint64_t (&w)[kPairs]) {
#pragma unroll
                for (int e = 0; e < kPairs; ++e)
                    v[j][e] = ffma2(bc2(a.residual_scale), w[e], v[j][e]);
            });
        } else {
            take(0, row_of(a.x, a.x_row, row), keep);
        }
        // the slot has been read: filled again
        if constexpr (!kVectors)
            one_warp ? __syncwarp() : __syncthreads();
        refill();
        from = from + slot_bytes == end ? slot0 : from + slot_bytes;
        if (a.branch)
            store(a.h, a.h_row);
        if (a.weight) {
            norm_row<kType, kVectors, kVecs, kLayer, kHalves>(a, at, v, a.weight, a.bias, team);
            store(a.y, a.y_row);
        }
    }
    copy_wait(0);
    pdl_trigger();
}

// Shared memory of one SM for the rings of its blocks, each of which takes a little
// beside: one slot of the widest rows at least.
constexpr int kMostRing = 220 * 1024;
constexpr int kBlockBytes = 1024 + 256;
constexpr int ring_bytes(int blocks)
{
    return 228 * 1024 - blocks * kBlockBytes < kMostRing ? 228 * 1024 - blocks * kBlockBytes : kMostRing;
}
static_assert(3 * (kResidualNormMaxWidth * 4 + 30) <= ring_bytes(1), "a slot");

template <int kType, bool kVectors, int kVecs, bool kLayer, bool kHalves = false>
cudaError_t launch(ResidualNormArgs &a, int num_sms, cudaStream_t stream)
{
    static PerDeviceOnce once;
    constexpr int kBytes = Row<kType, kVectors, kVecs>::kBytes;
    auto *kernel = residual_norm_kernel<kType, kVectors, kVecs, kLayer, kHalves>;
    // warps on one SM, by registers: each of its four parts has 16384 of them
    int fit = 0;
    const cudaError_t e = per_device_once(once, &fit, [&](int *out) {
        cudaFuncAttributes f;
        cudaError_t r = cudaFuncGetAttributes(&f, kernel);
        if (r == cudaSuccess)
            r = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, ring_bytes(1));
        *out = 4 * (16384 / (32 * ((f.numRegs > 0 ? f.numRegs + 7 : 64) / 8 * 8)));
        return r;
    });
    if (e != cudaSuccess)
        return e;
    const int crews = a.warps > 1 ? 1 : kWarpCrews, threads = 32 * (a.warps > 1 ? a.warps : kWarpCrews);
    const int beside = 32 / a.lanes;
    // a row, from and to 16 bytes
    a.row_bytes = kVectors ? a.width * kBytes : (a.width * kBytes + 30) / 16 * 16;
    a.tensors = a.gate && !a.gate_channels ? 3 : a.branch ? 2 : 1;
    // two slots or more: the SM's blocks share the memory, fewer blocks where that does
    // not do, and one slot where it does not do for a single block (rows of more than
    // 36 KB from three tensors, 55 KB from two)
    const int slot = crews * beside * a.row_bytes * a.tensors;
    int per_sm = std::max(1, std::min(fit / (threads / 32), 2048 / threads));
    while (per_sm > 1 && ring_bytes(per_sm) < per_sm * 2 * slot)
        --per_sm;
    a.slots = std::min(kMostSlots, ring_bytes(per_sm) / (per_sm * slot));
    const long long need = (a.rows + crews * beside - 1) / (crews * beside);
    const long long most = static_cast<long long>(num_sms) * per_sm;
    return launch_chained(kernel, dim3(static_cast<unsigned>(need < most ? need : most)), dim3(threads), a.slots * slot,
                          stream, a);
}

template <int kType, bool kVectors, bool kLayer>
cudaError_t launch(ResidualNormArgs &a, int num_sms, cudaStream_t stream)
{
    constexpr int kN = Row<kType, kVectors, 1>::kN;
    const int vecs = (a.width + kN - 1) / kN;           // of a row
    // up to 32 lanes take a row (all 32 where they take single numbers), then more
    // vectors each, then more warps: those that share out 16 numbers a lane, or, with
    // many rows of 16-bit vectors, 32, so that two crews or more share an SM and one
    // sums while another loads (f16, LayerNorm with the residual, 7812 x 4096 45 us
    // against 49, 3906 x 8192 42 / 52, RMS on both sides with gates of sequences 50 / 65 and 53 / 71;
    // 304 x 4096 with all parts 5.7 / 4.5.  In fp32 slots of twice the bytes leave
    // no room for more crews: 3906 x 4096 with all parts 75 / 52)
    a.lanes = kVectors ? 1 : 32;
    while (a.lanes < 32 && a.lanes < vecs)
        a.lanes *= 2;
    const int most = kVectors ? kType == MBERT_F32 ? 8 : 6 : 32 / kN;
    const int few = (a.width + 64 * kCrewNumbers - 1) / (64 * kCrewNumbers);
    const int small = (vecs + 32 * few - 1) / (32 * few);       // vectors of a lane of such a crew
    const bool fewer = kVectors && kType != MBERT_F32 && vecs > 32 * most && few <= kMostWarps / 2 &&
                       (a.rows > 2 * num_sms || small != 4);
    a.warps = vecs <= 32 * most ? 1
              : fewer ? few
              : std::min(kMostWarps, (a.width + 32 * kCrewNumbers - 1) / (32 * kCrewNumbers));
    // A row's bits do not go by the number of rows: the halves of a lane's 4 vectors in the
    // smaller crew are the warps of the other, with 2 a lane, and are summed like these.
    // (Rows of 2056 to 2304 numbers, 3 vectors a lane, have the smaller crew always.)
    if constexpr (kVectors && kType != MBERT_F32)
        if (fewer && small == 4)
            return launch<kType, kVectors, 4, kLayer, true>(a, num_sms, stream);
    const int each = (vecs + a.lanes * a.warps - 1) / (a.lanes * a.warps);
    if constexpr (kVectors || kN == 4) {
        if constexpr (kN == 4)
            if (each > 6)
                return launch<kType, kVectors, 8, kLayer>(a, num_sms, stream);
        if (each == 6)
            return launch<kType, kVectors, 6, kLayer>(a, num_sms, stream);
        if (each == 5)
            return launch<kType, kVectors, 5, kLayer>(a, num_sms, stream);
    }
    switch (each) {
    case 1: return launch<kType, kVectors, 1, kLayer>(a, num_sms, stream);
    case 2: return launch<kType, kVectors, 2, kLayer>(a, num_sms, stream);
    case 3: return launch<kType, kVectors, 3, kLayer>(a, num_sms, stream);
    default: return launch<kType, kVectors, 4, kLayer>(a, num_sms, stream);
    }
}

template <int kType>
cudaError_t launch(ResidualNormArgs &a, bool layer, int num_sms, cudaStream_t stream)
{
    if (a.vectors)
        return layer ? launch<kType, true, true>(a, num_sms, stream) : launch<kType, true, false>(a, num_sms, stream);
    return layer ? launch<kType, false, true>(a, num_sms, stream) : launch<kType, false, false>(a, num_sms, stream);
}

}  // namespace

cudaError_t launch_residual_norm(ResidualNormArgs &a, int dtype, bool layer, int num_sms, cudaStream_t stream)
{
    switch (dtype) {
    case MBERT_F32: return launch<MBERT_F32>(a, layer, num_sms, stream);
    case MBERT_F16: return launch<MBERT_F16>(a, layer, num_sms, stream);
    default: return launch<MBERT_BF16>(a, layer, num_sms, stream);
    }
}

}  // namespace mbert
