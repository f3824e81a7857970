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
// each, so memory, as long as the instructions per element stay few.  So a
// thread keeps one place of a row (its tensor, its head, its slot of two
// vectors of VW numbers, the halves of VW pairs) and walks down the rows: no
// index arithmetic but an add, weights in registers.  kU rows are in flight
// per thread before the first is needed.  The 2^k >= slots lanes of a head lie
// side by side, so a norm needs k shuffles and no shared memory.  All heads of
// a row share its cosines and sines: the block computes its rows' once into
// shared memory, laid out so that the lanes' 16-byte reads have no conflicts.
#include <cuda_fp16.h>

#include "mbert_attn.h"
#include "common.cuh"
#include "internal.h"

namespace mbert {
namespace {

constexpr int kMaxThreads = 384;
constexpr int kTableBytes = 16384;      // cosines and sines of a block's rows
constexpr int kMaxRows = 64;            // rows of a block

template <typename T, int N>
struct alignas(sizeof(T) * N) Vec {
    T v[N];
};

template <typename T> __device__ __forceinline__ float to_f32(T v);
template <> __device__ __forceinline__ float to_f32(float v) { return v; }
template <> __device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <> __device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

template <typename T, int N>
__device__ __forceinline__ void unpack(const Vec<T, N> &x, float (&f)[N])
{
#pragma unroll
    for (int i = 0; i < N; ++i)
        f[i] = to_f32<T>(x.v[i]);
}

template <int N>
__device__ __forceinline__ void pack(const float (&f)[N], Vec<float, N> &x)
{
#pragma unroll
    for (int i = 0; i < N; ++i)
        x.v[i] = f[i];
}
template <int N>
__device__ __forceinline__ void pack(const float (&f)[N], Vec<__half, N> &x)
{
    if constexpr (N == 1) {
        x.v[0] = __float2half_rn(f[0]);
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 2)
            *reinterpret_cast<__half2 *>(&x.v[i]) = __floats2half2_rn(f[i], f[i + 1]);
    }
}
template <int N>
__device__ __forceinline__ void pack(const float (&f)[N], Vec<__nv_bfloat16, N> &x)
{
    if constexpr (N == 1) {
        x.v[0] = __float2bfloat16_rn(f[0]);
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 2)
            *reinterpret_cast<__nv_bfloat162 *>(&x.v[i]) = __floats2bfloat162_rn(f[i], f[i + 1]);
    }
}

// Two fp32 products or sums per instruction where N is even.
template <int N>
__device__ __forceinline__ void mul_to(float (&y)[N], const float (&a)[N], const float (&b)[N])
{
    if constexpr (N == 1) {
        y[0] = a[0] * b[0];
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 2)
            f2_split(fmul2(f2(a[i], a[i + 1]), f2(b[i], b[i + 1])), y[i], y[i + 1]);
    }
}
template <int N>
__device__ __forceinline__ void fma_to(float (&y)[N], const float (&a)[N], const float (&b)[N], const float (&c)[N])
{
    if constexpr (N == 1) {
        y[0] = fmaf(a[0], b[0], c[0]);
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 2)
            f2_split(ffma2(f2(a[i], a[i + 1]), f2(b[i], b[i + 1]), f2(c[i], c[i + 1])), y[i], y[i + 1]);
    }
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

// Place of pair m in a row's table of cosines (sines follow): with 8 pairs per
// slot, the first 4 of every slot, then the second 4, so that neighbouring
// lanes read neighbouring 16 bytes.
template <int VW>
__device__ __forceinline__ int table_place(int m, int rot_slots)
{
    return VW == 8 ? (((m >> 2 & 1) * rot_slots + (m >> 3)) << 2) + (m & 3) : m;
}

template <int VW>
__device__ __forceinline__ void table_read(const float *t, int slot, int rot_slots, float (&c)[VW])
{
    if constexpr (VW == 8) {
        *reinterpret_cast<float4 *>(&c[0]) = *reinterpret_cast<const float4 *>(t + 4 * slot);
        *reinterpret_cast<float4 *>(&c[4]) = *reinterpret_cast<const float4 *>(t + 4 * (rot_slots + slot));
    } else {
#pragma unroll
        for (int i = 0; i < VW; ++i)
            c[i] = t[VW * slot + i];
    }
}

// VW numbers per vector; SPL slots per lane (more than one only where a head
// has more than 32 slots); kU rows in flight per thread.
template <typename T, int VW, int SPL, int kU, bool kInterleaved, bool kNorm>
__global__ void __launch_bounds__(kMaxThreads)
rotary_kernel(const __grid_constant__ RotaryArgs a)
{
    pdl_wait();
    __shared__ __align__(16) float s_table[kTableBytes / 4];
    __shared__ long long s_pos[kMaxRows];
    __shared__ bool s_live[kMaxRows];
    using V = Vec<T, VW>;
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
    auto load = [&](int r, V (&v0)[SPL], V (&v1)[SPL]) {
#pragma unroll
        for (int j = 0; j < SPL; ++j) {
            v0[j] = v1[j] = V{};
            if (placed && r < rows && slot0 + 32 * j < slots) {
                v0[j] = *reinterpret_cast<const V *>(src + off0[j]);
                v1[j] = *reinterpret_cast<const V *>(src + off1[j]);
            }
        }
        src += src_step;
    };
    // the first rows are on their way while the table is made
    V v0[kU][SPL], v1[kU][SPL];
#pragma unroll
    for (int u = 0; u < kU; ++u)
        load(team + u * a.teams, v0[u], v1[u]);

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
    for (int i = tid; i < rows * half; i += blockDim.x) {
        const int r = i / half, m = i - r * half;
        // t / 2^63 half turns, in [-1, 1)
        const unsigned long long t = static_cast<unsigned long long>(s_pos[r]) * a.turns[m];
        float s, c;
        sincospif(static_cast<float>(static_cast<long long>(t)) * 0x1p-63f, &s, &c);
        float *row = s_table + 2 * half * r + table_place<VW>(m, rot_slots);
        row[0] = c * a.amplitude;
        row[half] = s * a.sin_amplitude;
    }
    __syncthreads();

    float w0[SPL][VW], w1[SPL][VW];
    if constexpr (kNorm) {
#pragma unroll
        for (int j = 0; j < SPL; ++j) {
            V w{}, z{};
            if (placed && slot0 + 32 * j < slots) {
                w = *reinterpret_cast<const V *>(static_cast<const T *>(x.weight) + off0[j]);
                z = *reinterpret_cast<const V *>(static_cast<const T *>(x.weight) + off1[j]);
            }
            unpack(w, w0[j]);
            unpack(z, w1[j]);
        }
    }
    const float inv_dim = 1.f / a.dim;
    for (int r0 = 0; r0 < rows; r0 += kU * a.teams) {
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int r = r0 + team + u * a.teams;
            float f0[SPL][VW], f1[SPL][VW];
#pragma unroll
            for (int j = 0; j < SPL; ++j) {
                unpack(v0[u][j], f0[j]);
                unpack(v1[u][j], f1[j]);
            }
            // this slot's next row
            load(r + kU * a.teams, v0[u], v1[u]);
            if constexpr (kNorm) {
                // statistics in fp32 over the head's lanes; LayerNorm in two
                // passes (mean, then squared deviations)
                if (a.norm == MBERT_NORM_LAYER) {
                    float s = 0.f;
#pragma unroll
                    for (int j = 0; j < SPL; ++j)
#pragma unroll
                        for (int i = 0; i < VW; ++i)
                            s += f0[j][i] + f1[j][i];
                    for (int d = 1 << a.lanes_log2 >> 1; d; d >>= 1)
                        s += __shfl_xor_sync(0xffffffffu, s, d);
                    const float mean = s * inv_dim;
#pragma unroll
                    for (int j = 0; j < SPL; ++j)
                        if (slot0 + 32 * j < slots) {
#pragma unroll
                            for (int i = 0; i < VW; ++i) {
                                f0[j][i] -= mean;
                                f1[j][i] -= mean;
                            }
                        }
                }
                float q[VW];
#pragma unroll
                for (int i = 0; i < VW; ++i)
                    q[i] = 0.f;
#pragma unroll
                for (int j = 0; j < SPL; ++j) {
                    fma_to(q, f0[j], f0[j], q);
                    fma_to(q, f1[j], f1[j], q);
                }
                float sum = q[0];
#pragma unroll
                for (int i = 1; i < VW; ++i)
                    sum += q[i];
                for (int d = 1 << a.lanes_log2 >> 1; d; d >>= 1)
                    sum += __shfl_xor_sync(0xffffffffu, sum, d);
                const float inv = rsqrtf(fmaf(sum, inv_dim, a.eps));
                float scale[VW];
#pragma unroll
                for (int i = 0; i < VW; ++i)
                    scale[i] = inv;
#pragma unroll
                for (int j = 0; j < SPL; ++j) {
                    mul_to(f0[j], f0[j], scale);
                    mul_to(f1[j], f1[j], scale);
                    mul_to(f0[j], f0[j], w0[j]);
                    mul_to(f1[j], f1[j], w1[j]);
                }
            }
            if (placed && r < rows && s_live[r]) {
                const float *row = s_table + 2 * half * r;
#pragma unroll
                for (int j = 0; j < SPL; ++j) {
                    const int s = slot0 + 32 * j;
                    if (s >= slots)
                        continue;
                    if (s < rot_slots) {
                        float c[VW], sn[VW];
                        table_read<VW>(row, s, rot_slots, c);
                        table_read<VW>(row + half, s, rot_slots, sn);
                        if constexpr (kInterleaved) {
                            // pairs are neighbours: (0, 1), (2, 3), ... over both vectors
                            float y[2 * VW];
#pragma unroll
                            for (int i = 0; i < VW; ++i) {
                                y[i] = f0[j][i];
                                y[VW + i] = f1[j][i];
                            }
#pragma unroll
                            for (int m = 0; m < VW; ++m) {
                                const float p = y[2 * m], q2 = y[2 * m + 1];
                                y[2 * m] = p * c[m] - q2 * sn[m];
                                y[2 * m + 1] = q2 * c[m] + p * sn[m];
                            }
#pragma unroll
                            for (int i = 0; i < VW; ++i) {
                                f0[j][i] = y[i];
                                f1[j][i] = y[VW + i];
                            }
                        } else {
                            float p[VW], q2[VW], ns[VW];
#pragma unroll
                            for (int i = 0; i < VW; ++i)
                                ns[i] = -sn[i];
                            mul_to(p, f0[j], c);
                            mul_to(q2, f1[j], c);
                            fma_to(p, f1[j], ns, p);
                            fma_to(q2, f0[j], sn, q2);
#pragma unroll
                            for (int i = 0; i < VW; ++i) {
                                f0[j][i] = p[i];
                                f1[j][i] = q2[i];
                            }
                        }
                    }
                    V o0, o1;
                    pack(f0[j], o0);
                    pack(f1[j], o1);
                    *reinterpret_cast<V *>(dst + off0[j]) = o0;
                    *reinterpret_cast<V *>(dst + off1[j]) = o1;
                }
            }
            dst += dst_step;
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
    const int lanes = 1 << a.lanes_log2;
    const int heads = a.x[0].heads + a.x[1].heads;
    // Heads of a block: all, where they fit; else equal shares.  Then as many
    // teams (rows side by side) as leave the fewest lanes of whole warps idle.
    const int fit = kMaxThreads / lanes;
    const int shares = (heads + fit - 1) / fit;
    a.block_heads = (heads + shares - 1) / shares;
    int threads = 0;
    double best = -1.0;
    for (int t = 1; t * a.block_heads * lanes <= kMaxThreads && t <= a.tokens; ++t) {
        const int th = (t * a.block_heads * lanes + 31) / 32 * 32;
        const double use = static_cast<double>(t * a.block_heads * lanes) / th + (th >= 192 ? 0.5 : th / 384.0);
        if (use > best + 1e-9) {
            best = use;
            threads = th;
            a.teams = t;
        }
    }
    // Rows of a block: what the table holds, fewer while that leaves less than
    // six blocks per SM (and at least kU per team while that leaves two)
    const int step = a.teams * kU;
    int rows = a.rot ? kTableBytes / (4 * a.rot) : kMaxRows;
    rows = rows > kMaxRows ? kMaxRows : rows;
    const long long even = (a.tokens * shares + num_sms * 6 - 1) / (num_sms * 6);
    if (even < rows)
        rows = static_cast<int>(even);
    if (rows > step)
        rows = rows / step * step;
    if (rows < a.teams)
        rows = a.teams;
    const int most = a.rot ? kTableBytes / (4 * a.rot) : kMaxRows;
    a.block_rows = rows > most ? most : rows;
    const dim3 grid(static_cast<unsigned>((a.tokens + a.block_rows - 1) / a.block_rows), shares);
    void (*kernel)(RotaryArgs) =
        a.norm ? (a.interleaved ? rotary_kernel<T, VW, SPL, kU, true, true> : rotary_kernel<T, VW, SPL, kU, false, true>)
               : (a.interleaved ? rotary_kernel<T, VW, SPL, kU, true, false>
                                : rotary_kernel<T, VW, SPL, kU, false, false>);
    return launch_chained(kernel, grid, dim3(threads), 0, stream, a);
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
