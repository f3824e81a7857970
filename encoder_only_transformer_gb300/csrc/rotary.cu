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
// the signed fraction then goes through sincospif, which needs no range
// reduction.  The error of an angle is that of f_m's double (2^-53 relative)
// and of one fp32 rounding, at any position.
//
// What bounds it: every element is read once and written once, a few flops
// each; the sines are the only dear part, and all heads of a row share them.
// So a warp takes a few whole rows: it computes their cosines and sines once,
// one pair per lane, into shared memory (2 KB per warp), then walks the rows'
// heads.  A head is cut into slots of two vectors of VW numbers (the two
// halves of VW pairs), one slot per lane, the 2^k >= slots lanes of a head
// side by side, so a norm needs k shuffles and no shared memory.  Loads of kU
// heads are in flight per lane before the first is needed.
#include <cuda_fp16.h>

#include "mbert_attn.h"
#include "common.cuh"
#include "internal.h"

namespace mbert {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kTableBytes = 2048;      // cos/sin per warp
constexpr int kTablePairs = kTableBytes / 8;

template <typename T> __device__ __forceinline__ float to_f32(T v);
template <> __device__ __forceinline__ float to_f32(float v) { return v; }
template <> __device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <> __device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32(float v) { return v; }
template <> __device__ __forceinline__ __half from_f32(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32(float v) { return __float2bfloat16_rn(v); }

template <typename T, int N>
struct alignas(sizeof(T) * N) Vec {
    T v[N];
};

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
    if (a.pos32)
        pos = __ldg(a.pos32 + row);
    else if (a.pos64)
        pos = __ldg(a.pos64 + row);
    else
        pos = 0;
    return true;
}

// VW numbers per vector; SPL slots per lane (more than one only where a head
// has more than 32 slots); kU heads in flight per lane.
template <typename T, int VW, int SPL, int kU, bool kInterleaved>
__global__ void __launch_bounds__(kThreads)
rotary_kernel(const __grid_constant__ RotaryArgs a)
{
    pdl_wait();
    __shared__ __align__(16) float2 s_table[kWarps][kTablePairs];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int half = a.rot >> 1;
    using V = Vec<T, VW>;

    // cu_seqlens is only data here (a bad one cannot lead outside the rows);
    // one block reports it
    if (a.cu && blockIdx.x == 0) {
        bool bad = threadIdx.x == 0 && (a.cu[0] != 0 || a.cu[a.n_seqs] > a.tokens);
        for (int s = threadIdx.x; s < a.n_seqs; s += kThreads)
            bad |= a.cu[s + 1] < a.cu[s];
        if (bad)
            atomicOr(a.err, kErrBadCu);
    }

    // this warp's rows [row0, row0 + rows) and its share of their heads
    const long long task = static_cast<long long>(blockIdx.x) * kWarps + warp;
    const int part = static_cast<int>(task % a.parts);
    const long long row0 = task / a.parts * a.rows_per_warp;
    if (row0 < a.tokens) {
        const int rows = static_cast<int>(min(static_cast<long long>(a.rows_per_warp), a.tokens - row0));
        uint32_t live = 0;             // bit i: row row0 + i has a position
        {
            long long pos = 0;
            const bool ok = lane < rows && row_position(a, row0 + lane, pos);
            live = __ballot_sync(0xffffffffu, ok);
            for (int m0 = 0; m0 < half; m0 += 32) {
                const int m = m0 + lane;
                const unsigned long long w = m < half ? a.turns[m] : 0ull;
                for (int i = 0; i < rows; ++i) {
                    const long long p = __shfl_sync(0xffffffffu, pos, i);
                    const unsigned long long t = static_cast<unsigned long long>(p) * w;
                    float s, c;
                    // t / 2^63 half turns, in [-1, 1)
                    sincospif(static_cast<float>(static_cast<long long>(t)) * 0x1p-63f, &s, &c);
                    if (m < half)
                        s_table[warp][i * half + m] = make_float2(c * a.amplitude, s * a.sin_amplitude);
                }
            }
        }
        __syncwarp();

        const int gl = 1 << a.lanes_log2;               // lanes of one head
        const int sub = lane >> a.lanes_log2, slot0 = lane & (gl - 1);
        const int ipw = 32 >> a.lanes_log2;             // heads side by side
        const int slots = a.dim / (2 * VW), rot_slots = a.rot / (2 * VW);
        const int mid_off = kInterleaved ? VW : half;   // second vector of a turned slot
        for (int t = 0; t < 2; ++t) {
            const RotaryRows &x = a.x[t];
            if (x.heads == 0)
                continue;
            // the lane's slots: offsets of its two vectors, the weights
            int off0[SPL], off1[SPL];
            V w0[SPL], w1[SPL];
#pragma unroll
            for (int j = 0; j < SPL; ++j) {
                const int s = slot0 + 32 * j;
                const bool turned = s < rot_slots;
                off0[j] = turned && !kInterleaved ? s * VW : 2 * s * VW;
                off1[j] = off0[j] + (turned ? mid_off : VW);
                if (a.norm && s < slots) {
                    w0[j] = *reinterpret_cast<const V *>(static_cast<const T *>(x.weight) + off0[j]);
                    w1[j] = *reinterpret_cast<const V *>(static_cast<const T *>(x.weight) + off1[j]);
                }
            }
            const int items = rows * x.heads;
            for (int it0 = part * ipw; it0 < items; it0 += a.parts * ipw * kU) {
                V v0[kU][SPL], v1[kU][SPL];
                int row_of[kU];
#pragma unroll
                for (int u = 0; u < kU; ++u) {
                    const int it = it0 + u * a.parts * ipw + sub;
                    const int r = it / x.heads;
                    row_of[u] = it < items && (live >> r & 1) ? r : -1;
                    if (row_of[u] >= 0) {
                        const T *src = static_cast<const T *>(x.src) + (row0 + r) * x.src_row +
                                       static_cast<long long>(it - r * x.heads) * x.src_head;
#pragma unroll
                        for (int j = 0; j < SPL; ++j)
                            if (slot0 + 32 * j < slots) {
                                v0[u][j] = *reinterpret_cast<const V *>(src + off0[j]);
                                v1[u][j] = *reinterpret_cast<const V *>(src + off1[j]);
                            }
                    }
                }
#pragma unroll
                for (int u = 0; u < kU; ++u) {
                    const bool mine = row_of[u] >= 0;
                    float f0[SPL][VW], f1[SPL][VW];
#pragma unroll
                    for (int j = 0; j < SPL; ++j)
#pragma unroll
                        for (int i = 0; i < VW; ++i) {
                            const bool in = mine && slot0 + 32 * j < slots;
                            f0[j][i] = in ? to_f32<T>(v0[u][j].v[i]) : 0.f;
                            f1[j][i] = in ? to_f32<T>(v1[u][j].v[i]) : 0.f;
                        }
                    if (a.norm) {
                        // statistics in fp32 over the head's lanes; LayerNorm in
                        // two passes (mean, then squared deviations)
                        float mean = 0.f;
                        if (a.norm == MBERT_NORM_LAYER) {
                            float s = 0.f;
#pragma unroll
                            for (int j = 0; j < SPL; ++j)
#pragma unroll
                                for (int i = 0; i < VW; ++i)
                                    s += f0[j][i] + f1[j][i];
                            for (int d = gl >> 1; d; d >>= 1)
                                s += __shfl_xor_sync(0xffffffffu, s, d);
                            mean = s / a.dim;
                        }
                        float q = 0.f;
#pragma unroll
                        for (int j = 0; j < SPL; ++j)
                            if (slot0 + 32 * j < slots) {
#pragma unroll
                                for (int i = 0; i < VW; ++i) {
                                    f0[j][i] -= mean;
                                    f1[j][i] -= mean;
                                    q = fmaf(f0[j][i], f0[j][i], q);
                                    q = fmaf(f1[j][i], f1[j][i], q);
                                }
                            }
                        for (int d = gl >> 1; d; d >>= 1)
                            q += __shfl_xor_sync(0xffffffffu, q, d);
                        const float inv = 1.f / sqrtf(q / a.dim + a.eps);
#pragma unroll
                        for (int j = 0; j < SPL; ++j)
#pragma unroll
                            for (int i = 0; i < VW; ++i) {
                                f0[j][i] *= inv * to_f32<T>(w0[j].v[i]);
                                f1[j][i] *= inv * to_f32<T>(w1[j].v[i]);
                            }
                    }
                    if (!mine)
                        continue;
                    const int it = it0 + u * a.parts * ipw + sub;
                    T *dst = static_cast<T *>(x.dst) + (row0 + row_of[u]) * x.dst_row +
                             static_cast<long long>(it - row_of[u] * x.heads) * x.dst_head;
#pragma unroll
                    for (int j = 0; j < SPL; ++j) {
                        const int s = slot0 + 32 * j;
                        if (s >= slots)
                            continue;
                        V o0, o1;
                        if (s < rot_slots) {
                            const float2 *cs = &s_table[warp][row_of[u] * half + s * VW];
                            if (kInterleaved) {
                                // pairs are neighbours: (0, 1), (2, 3), ... over both vectors
                                float y[2 * VW], z[2 * VW];
#pragma unroll
                                for (int i = 0; i < VW; ++i) {
                                    y[i] = f0[j][i];
                                    y[VW + i] = f1[j][i];
                                }
#pragma unroll
                                for (int m = 0; m < VW; ++m) {
                                    const float2 r = cs[m];
                                    z[2 * m] = y[2 * m] * r.x - y[2 * m + 1] * r.y;
                                    z[2 * m + 1] = y[2 * m + 1] * r.x + y[2 * m] * r.y;
                                }
#pragma unroll
                                for (int i = 0; i < VW; ++i) {
                                    o0.v[i] = from_f32<T>(z[i]);
                                    o1.v[i] = from_f32<T>(z[VW + i]);
                                }
                            } else {
#pragma unroll
                                for (int i = 0; i < VW; ++i) {
                                    const float2 r = cs[i];
                                    o0.v[i] = from_f32<T>(f0[j][i] * r.x - f1[j][i] * r.y);
                                    o1.v[i] = from_f32<T>(f1[j][i] * r.x + f0[j][i] * r.y);
                                }
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < VW; ++i) {
                                o0.v[i] = from_f32<T>(f0[j][i]);
                                o1.v[i] = from_f32<T>(f1[j][i]);
                            }
                        }
                        *reinterpret_cast<V *>(dst + off0[j]) = o0;
                        *reinterpret_cast<V *>(dst + off1[j]) = o1;
                    }
                }
            }
        }
    }
    pdl_trigger();
}

template <typename T, int VW, int SPL, int kU>
cudaError_t launch(RotaryArgs &a, int num_sms, cudaStream_t stream)
{
    const int slots = a.dim / (2 * VW);
    a.lanes_log2 = 0;
    while ((1 << a.lanes_log2) < slots && a.lanes_log2 < 5)
        ++a.lanes_log2;
    const int ipw = 32 >> a.lanes_log2;
    const int heads = a.x[0].heads > a.x[1].heads ? a.x[0].heads : a.x[1].heads;
    // rows per warp: enough that a warp's sines serve kU heads per lane, as
    // far as its table goes, and fewer while that leaves SMs without work
    int rows = (kU * ipw + heads - 1) / heads;
    const int fit = a.rot ? kTablePairs / (a.rot / 2) : 32;
    rows = rows > fit ? fit : rows;
    rows = rows > 32 ? 32 : rows;
    while (rows > 1 && (a.tokens + rows - 1) / rows < static_cast<long long>(num_sms) * 16)
        rows = (rows + 1) / 2;
    a.rows_per_warp = rows;
    const long long groups = (a.tokens + rows - 1) / rows;
    // few rows (single tokens): the heads of a row go to several warps
    a.parts = 1;
    if (groups < static_cast<long long>(num_sms) * 4) {
        const int want = (rows * heads + ipw - 1) / ipw;
        a.parts = want > kWarps ? kWarps : want;
    }
    const long long blocks = (groups * a.parts + kWarps - 1) / kWarps;
    auto kernel = a.interleaved ? rotary_kernel<T, VW, SPL, kU, true> : rotary_kernel<T, VW, SPL, kU, false>;
    return launch_chained(kernel, dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0, stream, a);
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
        return vw == 4 ? launch<float, 4, 1, 4>(a, num_sms, stream)
               : vw == 2 ? launch<float, 2, 2, 2>(a, num_sms, stream)
                         : launch<float, 1, 4, 1>(a, num_sms, stream);
    case MBERT_F16:
        return vw == 8 ? launch<__half, 8, 1, 4>(a, num_sms, stream)
               : vw == 4 ? launch<__half, 4, 1, 4>(a, num_sms, stream)
               : vw == 2 ? launch<__half, 2, 2, 2>(a, num_sms, stream)
                         : launch<__half, 1, 4, 1>(a, num_sms, stream);
    default:
        return vw == 8 ? launch<__nv_bfloat16, 8, 1, 4>(a, num_sms, stream)
               : vw == 4 ? launch<__nv_bfloat16, 4, 1, 4>(a, num_sms, stream)
               : vw == 2 ? launch<__nv_bfloat16, 2, 2, 2>(a, num_sms, stream)
                         : launch<__nv_bfloat16, 1, 4, 1>(a, num_sms, stream);
    }
}

}  // namespace mbert
