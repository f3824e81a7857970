// Rotary positions on rows of heads, alone or after a norm of every query and
// key head, in one pass: y = R(pos) N(x).
//
//   N   nothing, RMS (x / sqrt(mean x^2 + eps) w) or LayerNorm
//       ((x - mean) / sqrt(var + eps) w, bias-free) over one head's D numbers
//   R   the pairs of the head's first R numbers, (x[m], x[m + R/2]) or
//       (x[2m], x[2m + 1]), turned by pos * f_m and scaled by an amplitude
//
// Angles.  f_m / (2 pi), the turns per position, is a 64-bit binary fraction,
// so the turns of any 64-bit position are exact modulo 1 in one integer
// multiply (positions wrap in two's complement, so negative ones work too);
// the signed fraction needs no range reduction.  The error of an angle is that
// of f_m's double (2^-53 relative), of the cut to 32 bits and of one fp32
// rounding, at any position.
//
// What bounds it: every element is read once and written once, a few flops
// each, so memory, as long as the instructions per element stay few.  So a
// thread keeps one place of a row (its tensor, its head, its slot of two
// vectors of VW numbers, the halves of VW pairs) and walks down the rows: no
// index arithmetic but an add, weights in registers.  kAhead rows are in flight
// per thread, through its own places in shared memory (cp.async: no registers
// held by loads, which is what lets enough warps be resident; with the rows in
// registers the kernel spilled or ran with half the warps, and took 1.7 to 2.2
// times as long).  The 2^k >= slots lanes of a head lie
// side by side, so a norm needs k shuffles and no shared memory.  All heads of
// a row share its cosines and sines: the block computes its rows' once into
// shared memory, laid out so that the lanes' 16-byte reads have no conflicts.
// Heads whose squares fp32 does not hold are left out by the loop and done after
// it, scaled; that they are looked for costs nothing that shows on 24 heads a row,
// on one head (262144 rows of 64, bf16) 27.6 -> 30.4 us.
//
// Measured: 65536 rows x 12 heads of 64 bf16 32.3 us, 6.2 TB/s (0.92 of the
// copy bandwidth); queries and keys with RMS norm 63.2 us, 6.4 TB/s; LayerNorm,
// interleaved pairs, 96 of 128, fp16, 9001 rows x 36 heads 38.5 us, 4.3 TB/s,
// where the chain of a row binds (two sums over a head's lanes, then the
// rotation pair by pair: 280 instructions a step, 65 % of the issue slots, and
// 64 registers leave 25 warps an SM to hide it).  fp32, 32768 rows x 12 heads of 64:
// 30.9 us with either direction or with a norm, 6.5 TB/s; the norm alone 41.7,
// probably as a lane's two vectors then lie side by side, so that a load takes half
// of each sector.
#include <cuda_fp16.h>

#include <cmath>
#include <type_traits>

#include "mbert_attn.h"
#include "common.cuh"
#include "internal.h"

namespace mbert {
namespace {

// Block shape, by sweeps over the cases above: 192 threads at 64 registers and
// two rows in flight (four: 1 to 14 % slower, fewer blocks fit; 256 threads:
// equal on long rows, 13 % slower on 5003), and at least 24 blocks an SM (16:
// 1 to 2 % slower, 10: 4 to 9 %, the last wave shows).
constexpr int kMaxThreads = 192;
constexpr int kMinBlocks = 5;
constexpr int kAhead = 2;               // rows in flight per thread
constexpr int kBlocksPerSm = 24;        // blocks that the rows are cut into, at least
constexpr int kTableBytes = 16384;      // cosines and sines of a block's rows, at most
constexpr int kMaxRows = 64;            // rows of a block

template <typename T, int N>
struct alignas(sizeof(T) * N) Vec {
    T v[N];
};

// N numbers in fp32: neighbours share a 64-bit register pair, so that products
// and sums take two at a time (N = 1: one by one).
template <int N>
struct Nums {
    uint64_t v[N / 2];
    __device__ __forceinline__ float get(int i) const
    {
        float lo, hi;
        f2_split(v[i / 2], lo, hi);
        return i & 1 ? hi : lo;
    }
    __device__ __forceinline__ void pair(int i, float lo, float hi) { v[i] = f2(lo, hi); }
    static __device__ __forceinline__ Nums splat(float x)
    {
        Nums r;
#pragma unroll
        for (int i = 0; i < N / 2; ++i)
            r.v[i] = f2(x, x);
        return r;
    }
    __device__ __forceinline__ float sum() const
    {
        uint64_t t = v[0];
#pragma unroll
        for (int i = 1; i < N / 2; ++i)
            asm("add.rn.f32x2 %0, %0, %1;" : "+l"(t) : "l"(v[i]));
        float lo, hi;
        f2_split(t, lo, hi);
        return lo + hi;
    }
};
template <>
struct Nums<1> {
    float v;
    __device__ __forceinline__ float get(int) const { return v; }
    static __device__ __forceinline__ Nums splat(float x) { return {x}; }
    __device__ __forceinline__ float sum() const { return v; }
};

template <int N>
__device__ __forceinline__ Nums<N> operator*(const Nums<N> &a, const Nums<N> &b)
{
    Nums<N> r;
    if constexpr (N == 1)
        r.v = a.v * b.v;
    else
#pragma unroll
        for (int i = 0; i < N / 2; ++i)
            r.v[i] = fmul2(a.v[i], b.v[i]);
    return r;
}
template <int N>
__device__ __forceinline__ Nums<N> operator+(const Nums<N> &a, const Nums<N> &b)
{
    Nums<N> r;
    if constexpr (N == 1)
        r.v = a.v + b.v;
    else
#pragma unroll
        for (int i = 0; i < N / 2; ++i)
            asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v[i]) : "l"(a.v[i]), "l"(b.v[i]));
    return r;
}
template <int N>
__device__ __forceinline__ Nums<N> operator-(const Nums<N> &a, const Nums<N> &b)
{
    Nums<N> r;
    if constexpr (N == 1)
        r.v = a.v - b.v;
    else
#pragma unroll
        for (int i = 0; i < N / 2; ++i)
            asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r.v[i]) : "l"(a.v[i]), "l"(b.v[i]));
    return r;
}
template <int N>
__device__ __forceinline__ Nums<N> fma(const Nums<N> &a, const Nums<N> &b, const Nums<N> &c)
{
    Nums<N> r;
    if constexpr (N == 1)
        r.v = fmaf(a.v, b.v, c.v);
    else
#pragma unroll
        for (int i = 0; i < N / 2; ++i)
            r.v[i] = ffma2(a.v[i], b.v[i], c.v[i]);
    return r;
}

// Pairs of a type's numbers as 32 (64 for fp32) bits, to and from fp32.
template <typename T> __device__ __forceinline__ uint64_t pair_f32(const T *x);
template <> __device__ __forceinline__ uint64_t pair_f32(const __nv_bfloat16 *x)
{
    return bf16x2_to_f2(*reinterpret_cast<const uint32_t *>(x));
}
template <> __device__ __forceinline__ uint64_t pair_f32(const __half *x)
{
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(x));
    return f2(f.x, f.y);
}
template <> __device__ __forceinline__ uint64_t pair_f32(const float *x) { return *reinterpret_cast<const uint64_t *>(x); }

__device__ __forceinline__ void pair_store(__nv_bfloat16 *x, uint64_t v) { *reinterpret_cast<uint32_t *>(x) = f2_to_bf16x2(v); }
__device__ __forceinline__ void pair_store(__half *x, uint64_t v)
{
    float lo, hi;
    f2_split(v, lo, hi);
    *reinterpret_cast<__half2 *>(x) = __floats2half2_rn(lo, hi);
}
__device__ __forceinline__ void pair_store(float *x, uint64_t v) { *reinterpret_cast<uint64_t *>(x) = v; }

template <typename T> __device__ __forceinline__ float to_f32(T v);
template <> __device__ __forceinline__ float to_f32(float v) { return v; }
template <> __device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <> __device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_f32(float &x, float v) { x = v; }
__device__ __forceinline__ void from_f32(__half &x, float v) { x = __float2half_rn(v); }
__device__ __forceinline__ void from_f32(__nv_bfloat16 &x, float v) { x = __float2bfloat16_rn(v); }

template <typename T, int N>
__device__ __forceinline__ Nums<N> unpack(const Vec<T, N> &x)
{
    Nums<N> r;
    if constexpr (N == 1)
        r.v = to_f32<T>(x.v[0]);
    else
#pragma unroll
        for (int i = 0; i < N / 2; ++i)
            r.v[i] = pair_f32<T>(&x.v[2 * i]);
    return r;
}
template <typename T, int N>
__device__ __forceinline__ Vec<T, N> pack(const Nums<N> &f)
{
    Vec<T, N> x;
    if constexpr (N == 1)
        from_f32(x.v[0], f.v);
    else
#pragma unroll
        for (int i = 0; i < N / 2; ++i)
            pair_store(&x.v[2 * i], f.v[i]);
    return x;
}

// One vector of a thread from global to shared memory, without a register:
// asynchronously where the hardware can (4, 8 or 16 bytes).
template <int kBytes>
__device__ __forceinline__ void fetch(void *smem, const void *gmem)
{
    if constexpr (kBytes == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(smem_u32(smem)), "l"(gmem) : "memory");
    else if constexpr (kBytes >= 4)
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;"
                     :: "r"(smem_u32(smem)), "l"(gmem), "n"(kBytes) : "memory");
    else
        *static_cast<uint16_t *>(smem) = *static_cast<const uint16_t *>(gmem);
}
__device__ __forceinline__ void fetch_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kPending>
__device__ __forceinline__ void fetch_wait() { asm volatile("cp.async.wait_group %0;" :: "n"(kPending) : "memory"); }

// Sum over the `lanes` (a power of two) neighbouring lanes of a head.
__device__ __forceinline__ float head_sum(float s, int lanes)
{
#pragma unroll
    for (int d = 16; d; d >>= 1)
        if (lanes > d)
            s += __shfl_xor_sync(0xffffffffu, s, d);
    return s;
}

__device__ __forceinline__ float head_max(float m, int lanes)
{
#pragma unroll
    for (int d = 16; d; d >>= 1)
        if (lanes > d)
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    return m;
}

// Position of a row: given (32 or 64 bits), or its place in its sequence.
// False for a row behind the last sequence.
__device__ __forceinline__ bool row_position(const RotaryArgs &a, long long row, long long &pos)
{
    if (a.cu) {
        if (row >= __ldg(a.cu + a.n_seqs))
            return false;
        int lo = 0, hi = a.n_seqs;      // cu[lo] <= row < cu[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (__ldg(a.cu + mid) <= row)
                lo = mid;
            else
                hi = mid;
        }
        pos = row - __ldg(a.cu + lo);
        return true;
    }
    pos = a.pos32 ? __ldg(a.pos32 + row) : a.pos64 ? __ldg(a.pos64 + row) : 0;
    return true;
}

// Sine and cosine of pos * w turns, w a 64-bit binary fraction.  The product's
// upper 32 bits modulo 1 are exact but for a carry (2^-32 turns); as a signed
// number of half turns in [-1, 1) they need no range reduction.  fp32 rows take
// the accurate functions; for 16-bit rows the fast ones' error (2^-20.9
// absolute on [-pi, pi]) is far below the rows' own rounding (2^-11, 2^-8).
template <typename T>
__device__ __forceinline__ void sin_cos(long long pos, uint64_t w, float &s, float &c)
{
    const uint32_t plo = static_cast<uint32_t>(pos), phi = static_cast<uint32_t>(pos >> 32);
    const uint32_t wlo = static_cast<uint32_t>(w), whi = static_cast<uint32_t>(w >> 32);
    const int t = static_cast<int>(__umulhi(plo, wlo) + plo * whi + phi * wlo);
    const float half_turns = static_cast<float>(t) * 0x1p-31f;
    if constexpr (sizeof(T) == 4) {
        sincospif(half_turns, &s, &c);
    } else {
        const float x = half_turns * 3.14159265f;
        s = __sinf(x);
        c = __cosf(x);
    }
}

// Place of pair m in a row's table of cosines (sines follow): with 8 pairs per
// slot, the first 4 of every slot, then the second 4, so that neighbouring
// lanes read neighbouring 16 bytes.
template <int VW>
__device__ __forceinline__ int table_place(int m, int rot_slots)
{
    return VW == 8 ? (((m >> 2 & 1) * rot_slots + (m >> 3)) << 2) + (m & 3) : m;
}

template <int VW>
__device__ __forceinline__ Nums<VW> table_read(const float *t, int slot, int rot_slots)
{
    Nums<VW> c;
    if constexpr (VW >= 4) {
#pragma unroll
        for (int q = 0; q < VW / 4; ++q) {
            const ulonglong2 x = *reinterpret_cast<const ulonglong2 *>(t + 4 * (q * rot_slots + slot));
            c.v[2 * q] = x.x;
            c.v[2 * q + 1] = x.y;
        }
    } else if constexpr (VW == 2) {
        c.v[0] = *reinterpret_cast<const uint64_t *>(t + 2 * slot);
    } else {
        c.v = t[slot];
    }
    return c;
}

// A row's numbers from memory, scaled by the power of two that brings its head's
// largest near 1, at most most_scale; by 1 where that is zero or infinite.  Gives
// the scale.
template <typename T, int VW, int SPL>
__device__ float load_scaled(const T *row, const int (&off0)[SPL], const int (&off1)[SPL], int slots, int slot0,
                             bool mine, float most_scale, int lanes, Nums<VW> (&f0)[SPL], Nums<VW> (&f1)[SPL])
{
    using V = Vec<T, VW>;
    float big = 0.f;
#pragma unroll
    for (int j = 0; j < SPL; ++j) {
        V v{}, w{};
        if (mine && slot0 + 32 * j < slots) {
            v = *reinterpret_cast<const V *>(row + off0[j]);
            w = *reinterpret_cast<const V *>(row + off1[j]);
        }
        f0[j] = unpack(v);
        f1[j] = unpack(w);
#pragma unroll
        for (int i = 0; i < VW; ++i)
            big = fmaxf(big, fmaxf(fabsf(f0[j].get(i)), fabsf(f1[j].get(i))));
    }
    big = head_max(big, lanes);
    const float s = big > 0.f && big < INFINITY ? fminf(scalbnf(1.f, -ilogbf(big)), most_scale) : 1.f;
#pragma unroll
    for (int j = 0; j < SPL; ++j) {
        f0[j] = f0[j] * Nums<VW>::splat(s);
        f1[j] = f1[j] * Nums<VW>::splat(s);
    }
    return s;
}

// VW numbers per vector; SPL slots per lane (more than one only where a head
// has more than 32 slots).
template <typename T, int VW, int SPL, bool kInterleaved, bool kNorm>
__global__ void __launch_bounds__(kMaxThreads, kMinBlocks)
rotary_kernel(const __grid_constant__ RotaryArgs a)
{
    pdl_wait();
    extern __shared__ __align__(16) uint8_t s_dynamic[];
    __shared__ long long s_pos[kMaxRows];
    __shared__ bool s_live[kMaxRows];
    using V = Vec<T, VW>;
    // every thread's rows in flight, [ahead][slot][2][thread], then the table
    V *s_rows = reinterpret_cast<V *>(s_dynamic);
    float *s_table = reinterpret_cast<float *>(s_dynamic + a.table_offset);
    const int tid = threadIdx.x;
    const int half = a.rot >> 1;
    const int slots = a.dim / (2 * VW), rot_slots = a.rot / (2 * VW);
    const long long row0 = static_cast<long long>(blockIdx.x) * a.block_rows;
    const int rows = static_cast<int>(min(static_cast<long long>(a.block_rows), a.tokens - row0));

    // this thread's place: its rows team, team + teams, ..., its head and slot
    const int item = tid >> a.lanes_log2, slot0 = tid & ((1 << a.lanes_log2) - 1);
    const int heads = a.x[0].heads + a.x[1].heads;
    const int head_all = blockIdx.y * a.block_heads + item % a.block_heads;
    const int team = item / a.block_heads;
    const bool placed = team < a.teams && head_all < heads;
    const int which = head_all >= a.x[0].heads;
    const RotaryRows &x = a.x[which];
    const int head = head_all - (which ? a.x[0].heads : 0);
    const T *src = static_cast<const T *>(x.src) + head * x.src_head + (row0 + team) * x.src_row;
    T *dst = static_cast<T *>(x.dst) + head * x.dst_head + (row0 + team) * x.dst_row;
    const long long src_step = a.teams * x.src_row, dst_step = a.teams * x.dst_row;
    int off0[SPL], off1[SPL];
#pragma unroll
    for (int j = 0; j < SPL; ++j) {
        const int s = slot0 + 32 * j;
        const bool turned = s < rot_slots;
        off0[j] = turned && !kInterleaved ? s * VW : 2 * s * VW;
        off1[j] = off0[j] + (turned && !kInterleaved ? half : VW);
    }
    const int threads = blockDim.x;
    auto load = [&](int r, int u) {
#pragma unroll
        for (int j = 0; j < SPL; ++j)
            if (placed && r < rows && slot0 + 32 * j < slots) {
                fetch<sizeof(V)>(&s_rows[((u * SPL + j) * 2) * threads + tid], src + off0[j]);
                fetch<sizeof(V)>(&s_rows[((u * SPL + j) * 2 + 1) * threads + tid], src + off1[j]);
            }
        fetch_commit();
        src += src_step;
    };
    // places that no row fills hold zeros, so that sums need no selection
#pragma unroll
    for (int j = 0; j < SPL; ++j)
        if (!placed || slot0 + 32 * j >= slots) {
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                s_rows[((u * SPL + j) * 2) * threads + tid] = V{};
                s_rows[((u * SPL + j) * 2 + 1) * threads + tid] = V{};
            }
        }
    // the first rows are on their way while the table is made
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
        load(team + u * a.teams, u);

    // cu_seqlens is only data here (a bad one cannot lead outside the rows);
    // one block reports it
    if (a.cu && blockIdx.x == 0 && blockIdx.y == 0) {
        bool bad = tid == 0 && (a.cu[0] != 0 || a.cu[a.n_seqs] > a.tokens);
        for (int s = tid; s < a.n_seqs; s += blockDim.x)
            bad |= a.cu[s + 1] < a.cu[s];
        if (bad)
            atomicOr(a.err, kErrBadCu);
    }
    for (int r = tid; r < rows; r += blockDim.x) {
        long long p = 0;
        s_live[r] = row_position(a, row0 + r, p);
        s_pos[r] = p;
    }
    __syncthreads();
    if (half > 0) {
        // a thread keeps its pair and walks down the rows
        const int per = min(half, threads), down = threads / per;
        if (tid < per * down)
            for (int m = tid % per; m < half; m += per) {
                const uint64_t w = a.turns[m];
                float *place = s_table + table_place<VW>(m, rot_slots);
                for (int r = tid / per; r < rows; r += down) {
                    float s, c;
                    sin_cos<T>(s_pos[r], w, s, c);
                    place[2 * half * r] = c * a.amplitude;
                    place[2 * half * r + half] = s * a.sin_amplitude;
                }
            }
    }
    __syncthreads();

    Nums<VW> w0[SPL], w1[SPL];
    if constexpr (kNorm) {
#pragma unroll
        for (int j = 0; j < SPL; ++j) {
            V w{}, z{};
            if (placed && slot0 + 32 * j < slots) {
                w = *reinterpret_cast<const V *>(static_cast<const T *>(x.weight) + off0[j]);
                z = *reinterpret_cast<const V *>(static_cast<const T *>(x.weight) + off1[j]);
            }
            w0[j] = unpack(w);
            w1[j] = unpack(z);
        }
    }
    const uint32_t least_squares = placed ? a.least_squares : 0u;
    const float inv_dim = 1.f / a.dim;
    const int lanes = 1 << a.lanes_log2;
    // The statistics of a head, in fp32 over its lanes: LayerNorm in two passes
    // (mean, then squared deviations).  Gives the sum of squares, and the factor.
    auto norm = [&](Nums<VW> (&f0)[SPL], Nums<VW> (&f1)[SPL], float eps, float &rs) -> float {
        if (a.norm == MBERT_NORM_LAYER) {
            Nums<VW> t = f0[0] + f1[0];
#pragma unroll
            for (int j = 1; j < SPL; ++j)
                t = t + (f0[j] + f1[j]);
            const Nums<VW> mean = Nums<VW>::splat(head_sum(t.sum(), lanes) * inv_dim);
#pragma unroll
            for (int j = 0; j < SPL; ++j)
                if (slot0 + 32 * j < slots) {
                    f0[j] = f0[j] - mean;
                    f1[j] = f1[j] - mean;
                }
        }
        Nums<VW> q = f0[0] * f0[0];
        q = fma(f1[0], f1[0], q);
#pragma unroll
        for (int j = 1; j < SPL; ++j) {
            q = fma(f0[j], f0[j], q);
            q = fma(f1[j], f1[j], q);
        }
        const float total = head_sum(q.sum(), lanes);
        rs = rsqrtf(fmaf(total, inv_dim, eps));
        return total;
    };
    // Where a head's squares (or their sum, or LayerNorm's first one) are beyond
    // fp32, or below it and not hidden by eps.  (In one comparison, as floats from 0
    // up order like their bits.)  fp16's numbers have no such squares.
    constexpr bool kOdd = kNorm && !std::is_same_v<T, __half>;
    auto is_odd = [&](float total) { return kOdd && __float_as_uint(total) - least_squares >= a.squares; };
    // norm's factor and weight, the rotation and the result
    auto finish = [&](Nums<VW> (&f0)[SPL], Nums<VW> (&f1)[SPL], float rs, const float *table, T *to, bool store) {
        if constexpr (kNorm) {
            const Nums<VW> inv = Nums<VW>::splat(rs);
#pragma unroll
            for (int j = 0; j < SPL; ++j) {
                f0[j] = f0[j] * inv * w0[j];
                f1[j] = f1[j] * inv * w1[j];
            }
        }
        if (store) {
#pragma unroll
            for (int j = 0; j < SPL; ++j) {
                const int s = slot0 + 32 * j;
                if (s >= slots)
                    continue;
                if (s < rot_slots) {
                    const Nums<VW> c = table_read<VW>(table, s, rot_slots);
                    const Nums<VW> sn = table_read<VW>(table + half, s, rot_slots);
                    if constexpr (!kInterleaved) {
                        const Nums<VW> y = f0[j] * c - f1[j] * sn;
                        f1[j] = fma(f0[j], sn, f1[j] * c);
                        f0[j] = y;
                    } else if constexpr (VW == 1) {
                        const float y = f0[j].v * c.v - f1[j].v * sn.v;
                        f1[j].v = f1[j].v * c.v + f0[j].v * sn.v;
                        f0[j].v = y;
                    } else {
                        // pairs are neighbours: (0, 1), (2, 3), ... over both vectors
#pragma unroll
                        for (int m = 0; m < VW; ++m) {
                            Nums<VW> &f = m < VW / 2 ? f0[j] : f1[j];
                            const int at = m % (VW / 2);
                            const float p = f.get(2 * at), q = f.get(2 * at + 1), cm = c.get(m), sm = sn.get(m);
                            f.pair(at, p * cm - q * sm, q * cm + p * sm);
                        }
                    }
                }
                *reinterpret_cast<V *>(to + off0[j]) = pack<T, VW>(f0[j]);
                *reinterpret_cast<V *>(to + off1[j]) = pack<T, VW>(f1[j]);
            }
        }
    };
    const float *trow = s_table + 2 * half * team;          // of the step's row
    const int tstep = 2 * half * a.teams;
    static_assert(kMaxRows <= 64, "a bit per step");
    uint64_t odd_steps = 0, bit = 1;
    auto step = [&](int r0, int u) {
        const int r = r0 + team;
        Nums<VW> f0[SPL], f1[SPL];
        fetch_wait<kAhead - 1>();
#pragma unroll
        for (int j = 0; j < SPL; ++j) {
            f0[j] = unpack(s_rows[((u * SPL + j) * 2) * threads + tid]);
            f1[j] = unpack(s_rows[((u * SPL + j) * 2 + 1) * threads + tid]);
        }
        // the place is free for a later row
        load(r + kAhead * a.teams, u);
        float rs = 1.f;
        bool odd = false;
        if constexpr (kNorm)
            odd = is_odd(norm(f0, f1, a.eps, rs));
        if constexpr (kOdd) {
            odd_steps |= odd ? bit : 0;
            bit <<= 1;
        }
        finish(f0, f1, rs, trow, dst, placed && r < rows && s_live[r] && !odd);
        dst += dst_step;
        trow += tstep;
    };
#pragma unroll 1
    for (int r0 = 0, u = 0; r0 < rows; r0 += a.teams, u = (u + 1) % kAhead)
        step(r0, u);
    if constexpr (kOdd) {
        // The odd heads, which are as they were: scaled by a power of two, which
        // with eps times its square leaves the norm as it is.  (Behind the loop, as
        // a branch within it cost up to 9 %; and by the bits, as the other heads may
        // have been written over their numbers.)
#pragma unroll 1
        for (int r0 = 0; __any_sync(0xffffffffu, odd_steps != 0); r0 += a.teams, odd_steps >>= 1) {
            const bool odd = odd_steps & 1;
            if (!__any_sync(0xffffffffu, odd))
                continue;
            const int r = r0 + team;
            const bool mine = odd && r < rows;
            Nums<VW> f0[SPL], f1[SPL];
            float rs;
            const float s = load_scaled<T, VW, SPL>(
                static_cast<const T *>(x.src) + head * x.src_head + (row0 + r) * x.src_row, off0, off1, slots, slot0,
                mine, a.most_scale, lanes, f0, f1);
            norm(f0, f1, a.eps * s * s, rs);
            finish(f0, f1, rs, s_table + 2 * half * r,
                   static_cast<T *>(x.dst) + head * x.dst_head + (row0 + r) * x.dst_row, mine && s_live[r]);
        }
    }
    pdl_trigger();
}

template <typename T, int VW, int SPL, bool kInterleaved, bool kNorm>
cudaError_t launch_as(RotaryArgs &a, dim3 grid, int threads, cudaStream_t stream)
{
    constexpr int kRowBytes = kAhead * SPL * 2 * VW * static_cast<int>(sizeof(T));   // of a thread
    static PerDeviceOnce smem_once;
    const cudaError_t e = smem_opt_in(smem_once, rotary_kernel<T, VW, SPL, kInterleaved, kNorm>,
                                      kRowBytes * kMaxThreads + kTableBytes);
    if (e != cudaSuccess)
        return e;
    a.table_offset = kRowBytes * threads;
    return launch_chained(rotary_kernel<T, VW, SPL, kInterleaved, kNorm>, grid, dim3(threads),
                          a.table_offset + a.block_rows * a.rot * 4, stream, a);
}

template <typename T, int VW, int SPL>
cudaError_t launch(RotaryArgs &a, int num_sms, cudaStream_t stream)
{
    const int slots = a.dim / (2 * VW);
    a.lanes_log2 = 0;
    while ((1 << a.lanes_log2) < slots && a.lanes_log2 < 5)
        ++a.lanes_log2;
    const int lanes = 1 << a.lanes_log2;
    const int heads = a.x[0].heads + a.x[1].heads;
    // Heads of a block: all, where they fit; else equal shares.  Then as many
    // teams (rows side by side) as leave the fewest lanes of whole warps idle.
    const int fit = kMaxThreads / lanes;
    const int shares = (heads + fit - 1) / fit;
    a.block_heads = (heads + shares - 1) / shares;
    // (no more than a block may have rows: heads of up to 32 numbers, one or two
    // of them, would fit more)
    int most = a.rot ? kTableBytes / (4 * a.rot) : kMaxRows;
    most = most > kMaxRows ? kMaxRows : most;
    int threads = 0;
    double best = -1.0;
    for (int t = 1; t * a.block_heads * lanes <= kMaxThreads && t <= a.tokens && t <= most; ++t) {
        const int th = (t * a.block_heads * lanes + 31) / 32 * 32;
        const double use = static_cast<double>(t * a.block_heads * lanes) / th + (th >= 192 ? 0.5 : th / 384.0);
        if (use > best + 1e-9) {
            best = use;
            threads = th;
            a.teams = t;
        }
    }
    // Rows of a block: what the table holds, fewer while that leaves less than
    // kBlocksPerSm blocks per SM (and at least kAhead per team while that leaves two)
    const int step = a.teams * kAhead;
    int rows = most;
    const long long even = (a.tokens * shares + num_sms * kBlocksPerSm - 1) / (num_sms * kBlocksPerSm);
    if (even < rows)
        rows = static_cast<int>(even);
    if (rows > step)
        rows = rows / step * step;
    a.block_rows = rows < a.teams ? a.teams : rows;
    const dim3 grid(static_cast<unsigned>((a.tokens + a.block_rows - 1) / a.block_rows), shares);
    return a.norm ? (a.interleaved ? launch_as<T, VW, SPL, true, true>(a, grid, threads, stream)
                                   : launch_as<T, VW, SPL, false, true>(a, grid, threads, stream))
                  : (a.interleaved ? launch_as<T, VW, SPL, true, false>(a, grid, threads, stream)
                                   : launch_as<T, VW, SPL, false, false>(a, grid, threads, stream));
}

}  // namespace

// The vector width: the widest (16 bytes at most) that divides the head, its
// turned part, every stride and every address.
cudaError_t launch_rotary(RotaryArgs &a, int num_sms, cudaStream_t stream)
{
    const int es = a.dtype == MBERT_F32 ? 4 : 2;
    uintptr_t addr = 0;
    long long strides = 0;
    for (const RotaryRows &x : a.x) {
        if (x.heads == 0)
            continue;
        addr |= reinterpret_cast<uintptr_t>(x.src) | reinterpret_cast<uintptr_t>(x.dst);
        if (a.norm)
            addr |= reinterpret_cast<uintptr_t>(x.weight);
        strides |= x.src_row | x.src_head | x.dst_row | x.dst_head;
    }
    int vw = 16 / es;
    while (vw > 1 && (a.dim % (2 * vw) || a.rot % (2 * vw) || strides % vw || addr % (vw * es)))
        vw /= 2;
    switch (a.dtype) {
    case MBERT_F32:
        return vw == 4 ? launch<float, 4, 1>(a, num_sms, stream)
               : vw == 2 ? launch<float, 2, 2>(a, num_sms, stream)
                         : launch<float, 1, 4>(a, num_sms, stream);
    case MBERT_F16:
        return vw == 8 ? launch<__half, 8, 1>(a, num_sms, stream)
               : vw == 4 ? launch<__half, 4, 1>(a, num_sms, stream)
               : vw == 2 ? launch<__half, 2, 2>(a, num_sms, stream)
                         : launch<__half, 1, 4>(a, num_sms, stream);
    default:
        return vw == 8 ? launch<__nv_bfloat16, 8, 1>(a, num_sms, stream)
               : vw == 4 ? launch<__nv_bfloat16, 4, 1>(a, num_sms, stream)
               : vw == 2 ? launch<__nv_bfloat16, 2, 2>(a, num_sms, stream)
                         : launch<__nv_bfloat16, 1, 4>(a, num_sms, stream);
    }
}

}  // namespace mbert
