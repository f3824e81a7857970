// What the two kernels of the products of any width share: the walk over the
// units of ragged groups, the check of the groups' offsets, the activations.
#pragma once

#include <type_traits>

#include "common.cuh"
#include "linear.h"
#include "mbert_attn.h"
#include "roles.cuh"

namespace mbert {

// ---------------------------------------------------------------------------
// units: `block` rows x a block of output columns, group after group
// ---------------------------------------------------------------------------
struct Unit {
    int group, column;          // group, block of columns
    long long row, end;         // first row, the group's end
    bool first;                 // the group's first rows
};

// The units of a call in order.  Within a group they go by bands of `band` row
// blocks, column after column of a band, so that the units that run at the same
// time share rows and weights in L2.  Offsets are read as the walk comes to
// them, 128 groups at a time, four a lane, so any number of groups will do and no kernel
// has to write a list first.
class UnitWalk {
public:
    __device__ UnitWalk(const LinearArgs &a, int block, int columns, int band)
        : cu_(a.cu), groups_(a.groups), rows_(a.rows), block_(block), columns_(columns), band_(band)
    {
        if (cu_)
            window(0, 0);
    }

    // Unit u (not below the last one asked for); false behind the last unit.
    // Called by all lanes of a warp, with the same u.
    __device__ bool find(int u, Unit &out)
    {
        if (!cu_) {
            const int blocks = static_cast<int>((rows_ + block_ - 1) / block_);
            if (u >= blocks * columns_)
                return false;
            out.group = 0;
            place(u, blocks, 0, rows_, out);
            return true;
        }
        for (;;) {
            const int last = __shfl_sync(0xffffffffu, upto_, 31);
            if (u < last)
                break;
            if (first_ + kWindow >= groups_)
                return false;
            window(first_ + kWindow, last);
        }
        // the lane whose groups hold the unit, and the group
        const int l = __ffs(__ballot_sync(0xffffffffu, u < upto_)) - 1;
        int at = __shfl_sync(0xffffffffu, upto_ - units_, l), g = first_ + l * kPerLane, row = 0, end = 0;
        bool found = false;
#pragma unroll
        for (int i = 0; i < kPerLane; ++i) {
            const int x = __shfl_sync(0xffffffffu, cut_[i], l), y = __shfl_sync(0xffffffffu, cut_[i + 1], l);
            const int n = (y - x + block_ - 1) / block_ * columns_;
            if (!found && u < at + n) {
                found = true;
                g += i;
                row = x;
                end = y;
            }
            at += found ? 0 : n;
        }
        out.group = g;
        place(u - at, (end - row + block_ - 1) / block_, row, end, out);
        return true;
    }

private:
    __device__ void place(int i, int blocks, long long row, long long end, Unit &out) const
    {
        int r, b = 0, h = blocks;
        if (blocks > band_) {
            b = i / (band_ * columns_);
            i -= b * band_ * columns_;
            h = min(band_, blocks - b * band_);
        }
        out.column = i / h;
        r = b * band_ + i - out.column * h;
        out.row = row + static_cast<long long>(r) * block_;
        out.end = end;
        out.first = r == 0;
    }

    // groups first .. first + 127, whose units begin at `before`
    __device__ void window(int first, int before)
    {
        const int lane = threadIdx.x & 31, g = first + lane * kPerLane;
        first_ = first;
#pragma unroll
        for (int i = 0; i <= kPerLane; ++i)
            cut_[i] = cu_[min(g + i, groups_)];
        units_ = 0;
#pragma unroll
        for (int i = 0; i < kPerLane; ++i)
            units_ += (cut_[i + 1] - cut_[i] + block_ - 1) / block_ * columns_;
        upto_ = units_;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, upto_, o);
            upto_ += lane >= o ? x : 0;
        }
        upto_ += before;
    }

    static constexpr int kPerLane = 4, kWindow = 32 * kPerLane;
    const int32_t *cu_;
    int groups_;
    long long rows_;
    int block_, columns_, band_;
    int first_ = 0;
    // this lane's groups: where they begin and end, their units, the units up to their end
    int cut_[kPerLane + 1] = {}, units_ = 0, upto_ = 0;
};

// The units of a call, of `columns` a block of rows; -1 if the groups' offsets are not in
// order and within the rows (reported once).  Called by all lanes of a warp.
__device__ __forceinline__ long long count_units(const LinearArgs &a, int block, int columns)
{
    if (!a.cu)
        return (a.rows + block - 1) / block * columns;
    long long n = 0;
    bool bad = false;
    for (int g = threadIdx.x & 31; g < a.groups; g += 32) {
        const int x = a.cu[g], y = a.cu[g + 1];
        bad |= y < x || (g == 0 && x != 0) || (g == a.groups - 1 && y > a.rows);
        n += (static_cast<long long>(y) - x + block - 1) / block;
    }
    bad = __any_sync(0xffffffffu, bad);
    if (bad && blockIdx.x == 0 && (threadIdx.x & 31) == 0)
        atomicOr(a.err, kErrBadCu);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        n += __shfl_xor_sync(0xffffffffu, n, o);
    return bad ? -1 : n * columns;
}

// Are the groups' offsets in order and within the rows?  Called by all threads
// of a block; a bad list is reported once, and the kernel then writes nothing.
__device__ __forceinline__ bool offsets_ok(const LinearArgs &a)
{
    if (!a.cu)
        return true;
    bool bad = false;
    for (int g = threadIdx.x; g <= a.groups; g += blockDim.x) {
        const int x = a.cu[g];
        bad |= g == 0 ? x != 0 : x < a.cu[g - 1];
        bad |= g == a.groups && x > a.rows;
    }
    bad = __syncthreads_or(bad) != 0;
    if (bad && blockIdx.x == 0 && threadIdx.x == 0)
        atomicOr(a.err, kErrBadCu);
    return !bad;
}

// mbar_wait for a whole warp: one answer for all lanes, so that none leaves its
// warp alone before an instruction of all of them.
__device__ __forceinline__ bool mbar_wait_warp(uint32_t bar, uint32_t parity, int *err)
{
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, err));
}

constexpr uint32_t make_idesc_f16(int M, int N, bool half)
{
    // fp16 is format 0 where bf16 is 1
    return make_idesc_bf16(M, N, false) & ~(half ? (1u << 7) | (1u << 10) : 0u);
}

// ---------------------------------------------------------------------------
// activations, on pairs of fp32 numbers
// ---------------------------------------------------------------------------
__device__ __forceinline__ float max_nan(float a, float b)
{
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

__device__ __forceinline__ float rcp_approx(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint64_t bc2(float x) { return f2(x, x); }

// z Phi(z) with Phi the normal distribution (the erf form): max(z, 0) - |z| q(|z|),
// where q(t) = 1 - Phi(t) = 2^(-t^2 log2(e) / 2 + Q(t)).  Q, the logarithm of
// e^(t^2/2) (1 - Phi(t)), bends so little that a polynomial of degree 8 gives it to
// 5.3e-6 on 0 .. 8 (least squares on Chebyshev points, reweighted until the errors
// were even); beyond, its value at 8 is taken, where q < 7e-16.  Together 1e-5 of the
// result (a half step of fp16 is 4.9e-4 of it) from z = -8 on, where 1 + erf would cancel
// for negative z; below -8, where the result is under 6e-15, q stays too large: by 12 % at
// -9, 49 % at -12.  One exponential and about 10 instructions a number against 25
// for erff.  (On single numbers instead of pairs 358 us against 331, 32768 x 1024 ->
// 8192.  Degree 11, 4.7e-7: 30367 x 40 -> 2 x 5656 210 us against 197, 65536 rows of 8
// experts, 768 -> 2 x 1152, 136.4 / 134.2; bf16 results of the latter that are not the exact
// ones' roundings 0.08 % against 0.10, most of them by the sums of products.)
__device__ __forceinline__ uint64_t gelu2(uint64_t z)
{
    float a, b;
    f2_split(z, a, b);
    const float ta = fabsf(a), tb = fabsf(b);
    const uint64_t t = f2(fminf(ta, 8.f), fminf(tb, 8.f)), w = f2(fminf(ta, 64.f), fminf(tb, 64.f));
    uint64_t p = ffma2(t, bc2(7.42839461e-08f), bc2(-3.65532651e-06f));
    p = ffma2(p, t, bc2(7.95740707e-05f));
    p = ffma2(p, t, bc2(-0.00102197588f));
    p = ffma2(p, t, bc2(0.0087621659f));
    p = ffma2(p, t, bc2(-0.0543373488f));
    p = ffma2(p, t, bc2(0.263151854f));
    p = ffma2(p, t, bc2(-1.15132189f));
    p = ffma2(p, t, bc2(-0.999992371f));
    p = ffma2(fmul2(w, w), bc2(-0.72134752f), p);       // (q is 0 at 64: 2^-2955)
    float qa, qb;
    f2_split(p, qa, qb);
    return ffma2(w, f2(-ex2_approx(qa), -ex2_approx(qb)), f2(max_nan(a, 0.f), max_nan(b, 0.f)));
}

// z / (1 + 2^e); z below -1e4 counts as -1e4, where the result is 0 (so that
// minus infinity does not meet a factor of 0)
__device__ __forceinline__ float over_1_plus_ex2(float z, float e)
{
    return max_nan(z, -1e4f) * rcp_approx(1.f + ex2_approx(e));
}

__device__ __forceinline__ uint64_t silu2(uint64_t z)
{
    float a, b;
    f2_split(z, a, b);
    return f2(over_1_plus_ex2(a, -1.44269504f * a), over_1_plus_ex2(b, -1.44269504f * b));
}

// z (1 + tanh(u)) / 2 = z / (1 + e^(-2u)), u = sqrt(2 / pi) (z + 0.044715 z^3)
__device__ __forceinline__ uint64_t gelu_tanh2(uint64_t z)
{
    constexpr float k1 = -2.30220819f, k3 = k1 * 0.044715f;     // -2 sqrt(2 / pi) log2(e)
    float a, b, ea, eb;
    f2_split(z, a, b);
    const uint64_t e = fmul2(z, ffma2(fmul2(z, z), bc2(k3), bc2(k1)));
    f2_split(e, ea, eb);
    return f2(over_1_plus_ex2(a, ea), over_1_plus_ex2(b, eb));
}

template <int kAct>
__device__ __forceinline__ uint64_t activate2(uint64_t z)
{
    if constexpr (kAct == MBERT_ACT_GELU)
        return gelu2(z);
    else if constexpr (kAct == MBERT_ACT_GELU_TANH)
        return gelu_tanh2(z);
    else if constexpr (kAct == MBERT_ACT_SILU)
        return silu2(z);
    else if constexpr (kAct == MBERT_ACT_RELU) {
        float a, b;
        f2_split(z, a, b);
        return f2(max_nan(a, 0.f), max_nan(b, 0.f));
    } else
        return z;
}

// f(integral constant) for the call's activation
template <typename F>
__device__ __forceinline__ void with_activation(int activation, F &&f)
{
    switch (activation) {
    case MBERT_ACT_GELU: f(std::integral_constant<int, MBERT_ACT_GELU>()); break;
    case MBERT_ACT_GELU_TANH: f(std::integral_constant<int, MBERT_ACT_GELU_TANH>()); break;
    case MBERT_ACT_SILU: f(std::integral_constant<int, MBERT_ACT_SILU>()); break;
    case MBERT_ACT_RELU: f(std::integral_constant<int, MBERT_ACT_RELU>()); break;
    default: f(std::integral_constant<int, MBERT_ACT_NONE>()); break;
    }
}

__device__ __forceinline__ uint64_t fadd2p(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// two 16-bit numbers of a word as fp32
template <bool kHalf>
__device__ __forceinline__ uint64_t unpack2(uint32_t w)
{
    if constexpr (kHalf) {
        float lo, hi;
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
            : "=f"(lo), "=f"(hi) : "r"(w));
        return f2(lo, hi);
    } else
        return bf16x2_to_f2(w);
}

template <bool kHalf>
__device__ __forceinline__ float load16(const void *p, long long i)
{
    const uint32_t v = static_cast<const uint16_t *>(p)[i];
    float lo, hi;
    f2_split(unpack2<kHalf>(v), lo, hi);
    return lo;
}

}  // namespace mbert
