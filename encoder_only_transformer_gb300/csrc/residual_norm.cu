// The norms after one block and before the next, with the gate and the residual
// between them, in one pass (sm_103a): for every row t
//     h_t = alpha x_t + g_t P(branch_t),   y_t = N(h_t)
// P and N: LayerNorm, (v - mean) / sqrt(var + eps) w + b with the population
// variance, or RMS, v / sqrt(mean(v^2) + eps) w + b; either may be absent, and so may
// the branch (y = N(x)) and the gate (of a channel, a row, or a row's sequence).
// bf16, fp16 or fp32; everything between loading and storing is fp32, y is of the
// h that has not been rounded.
//
// Bound by HBM: x and branch in, h and y out.  A row stays in registers from its
// load to its store: 16-byte vectors, up to four (eight in fp32) a lane, by 1 to 32
// lanes a row up to 1024 numbers and 2 to 16 warps beyond, which add their sums up in
// shared memory; the weights come from L1 or L2 each time, which costs no DRAM traffic
// and leaves the registers to the rows.  A norm's statistics are sums over the
// registers, the LayerNorm's in two passes (mean, then squares about it).
//
// Where the squares add up to what fp32 does not hold (or, beside a small eps, to
// what it holds badly), the row is scaled by a power of two first: see Norm.
#include "internal.h"
#include "residual_norm.h"
#include "linear.cuh"

namespace mbert {
namespace {

constexpr int kLaneNumbers = 32;    // numbers of a row that a lane holds, at most
constexpr int kMostThreads = kResidualNormMaxWidth / kLaneNumbers;

// The numbers of a row that lane `lane` of `step` holds: vectors of 16 bytes, the
// lanes' side by side, or (rows that such vectors do not fit) single numbers, again
// side by side.  load() fills with 0 behind the row's end.
template <int kType, bool kVectors>
struct Row {
    static constexpr int kN = kType == MBERT_F32 ? 4 : 8;
    int lane, step, width;

    // number e of vector j is number at(j, e) of the row
    __device__ int at(int j, int e) const
    {
        return kVectors ? (lane + j * step) * kN + e : lane + (j * kN + e) * step;
    }
    __device__ bool in(int j, int e) const { return at(j, kVectors ? 0 : e) < width; }

    __device__ void load(const void *p, long long row, int j, float (&v)[kN]) const
    {
        if constexpr (kVectors) {
            uint4 x = make_uint4(0, 0, 0, 0);
            if (in(j, 0))
                x = *reinterpret_cast<const uint4 *>(static_cast<const char *>(p) + (row + at(j, 0)) * (16 / kN));
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if constexpr (kType == MBERT_F32)
                    v[e] = __uint_as_float(w[e]);
                else
                    f2_split(unpack2<kType == MBERT_F16>(w[e]), v[2 * e], v[2 * e + 1]);
            }
        } else {
#pragma unroll
            for (int e = 0; e < kN; ++e) {
                v[e] = 0.f;
                if (in(j, e)) {
                    if constexpr (kType == MBERT_F32)
                        v[e] = static_cast<const float *>(p)[row + at(j, e)];
                    else
                        v[e] = load16<kType == MBERT_F16>(p, row + at(j, e));
                }
            }
        }
    }

    __device__ void store(void *p, long long row, int j, const float (&v)[kN]) const
    {
        if constexpr (kVectors) {
            if (!in(j, 0))
                return;
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if constexpr (kType == MBERT_F32)
                    w[e] = __float_as_uint(v[e]);
                else
                    w[e] = pack2<kType == MBERT_F16>(v[2 * e], v[2 * e + 1]);
            }
            *reinterpret_cast<uint4 *>(static_cast<char *>(p) + (row + at(j, 0)) * (16 / kN)) =
                make_uint4(w[0], w[1], w[2], w[3]);
        } else {
#pragma unroll
            for (int e = 0; e < kN; ++e) {
                if (!in(j, e))
                    continue;
                if constexpr (kType == MBERT_F32)
                    static_cast<float *>(p)[row + at(j, e)] = v[e];
                else
                    static_cast<uint16_t *>(p)[row + at(j, e)] = static_cast<uint16_t>(pack2<kType == MBERT_F16>(v[e], 0.f));
            }
        }
    }
};

// The lanes of a row: `lanes` of a warp, or `warps` whole warps of a block.
struct Team {
    int lanes, warps;
    float *scratch;     // [2][warps]
    int turn;

    template <typename Op>
    __device__ float all(float v, Op op)
    {
        for (int o = lanes >> 1; o > 0; o >>= 1)
            v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
        if (warps > 1) {
            // two places in turn, so that one barrier a sum will do
            float *s = scratch + (turn ^= 1) * 32;
            if ((threadIdx.x & 31) == 0)
                s[threadIdx.x >> 5] = v;
            __syncthreads();
            v = s[0];
            for (int w = 1; w < warps; ++w)
                v = op(v, s[w]);
        }
        return v;
    }
    __device__ float sum(float v) { return all(v, [](float x, float y) { return x + y; }); }
    __device__ float most(float v) { return all(v, [](float x, float y) { return fmaxf(x, y); }); }
};

// v[] of a row -> its norm times w plus b.  Called by all lanes of a warp.
//
// LayerNorm works on half of each number, so that no difference from the mean
// overflows (the sum of numbers times sum_scale, at most 1 / width, does not either),
// and with eps / 4.  Squares that add up to more than 2^126, or, beside an eps below
// 2^-40, to less than 2^-90 (those that round to nothing are then off by 2^-45 of the
// sum at most), are taken again of the row times a power of two that brings its
// largest number to 1 .. 2, or as near as keeps eps times its square at 2^100.
template <int kType, bool kVectors, int kVecs, bool kLayer>
__device__ __forceinline__ void norm_row(const ResidualNormArgs &a, const Row<kType, kVectors> &at,
                                         float (&v)[kVecs][Row<kType, kVectors>::kN], const void *w, const void *b,
                                         Team &team)
{
    constexpr int kN = Row<kType, kVectors>::kN;
    auto centre = [&](bool keep) {
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < kVecs; ++j)
#pragma unroll
            for (int e = 0; e < kN; ++e)
                s = fmaf(v[j][e], a.sum_scale, s);
        const float half_mean = team.sum(s) * a.half_mean_scale;
#pragma unroll
        for (int j = 0; j < kVecs; ++j)
#pragma unroll
            for (int e = 0; e < kN; ++e)
                if (!keep)
                    v[j][e] = at.in(j, e) ? fmaf(v[j][e], 0.5f, -half_mean) : 0.f;
    };
    auto squares = [&] {
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < kVecs; ++j)
#pragma unroll
            for (int e = 0; e < kN; ++e)
                s = fmaf(v[j][e], v[j][e], s);
        return team.sum(s);
    };
    float eps = a.eps;
    if constexpr (kLayer) {
        centre(false);
        eps *= 0.25f;
    }
    float q = squares();
    bool again = !(q >= a.least_squares && q <= 0x1p126f);      // (NaN too, which stay)
    if (__any_sync(0xffffffffu, again)) {
        float m = 0.f;
#pragma unroll
        for (int j = 0; j < kVecs; ++j)
#pragma unroll
            for (int e = 0; e < kN; ++e)
                m = fmaxf(m, fabsf(v[j][e]));
        m = team.most(m);
        again = again && m > 0.f && m < INFINITY;
        const int k = min(127 - (__float_as_int(m) >> 23), a.most_scale);
        const float up = again ? __int_as_float((max(k, -126) + 127) << 23) : 1.f;
        eps = eps * up * up;
#pragma unroll
        for (int j = 0; j < kVecs; ++j)
#pragma unroll
            for (int e = 0; e < kN; ++e)
                v[j][e] *= up;
        if constexpr (kLayer) {
            centre(!again);
            eps *= again ? 0.25f : 1.f;
        }
        const float sum = squares();
        q = again ? sum : q;
    }
    const float r = rsqrtf(fmaf(q, a.inv_width, eps));
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
        float wv[kN];
        at.load(w, 0, j, wv);
#pragma unroll
        for (int e = 0; e < kN; ++e)
            v[j][e] = v[j][e] * r * wv[e];
        if (b) {
            at.load(b, 0, j, wv);
#pragma unroll
            for (int e = 0; e < kN; ++e)
                v[j][e] += wv[e];
        }
    }
}

// kVecs 16-byte vectors a lane.
template <int kType, bool kVectors, int kVecs, bool kLayer>
__global__ void __launch_bounds__(kMostThreads) residual_norm_kernel(const ResidualNormArgs a)
{
    constexpr int kN = Row<kType, kVectors>::kN;
    __shared__ float scratch[64];
    pdl_wait();
    Team team{a.lanes, a.warps, scratch, 0};
    // rows side by side in a block, this thread's place among them and in its row
    const int step = a.lanes * a.warps, beside = blockDim.x / step;
    const Row<kType, kVectors> at{static_cast<int>(threadIdx.x) % step, step, a.width};
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
    const long long rows = bad ? 0 : a.cu ? a.cu[a.n_seqs] : a.rows;
    // (every thread makes the same rounds, so that its warp and block stay together)
    for (long long t0 = static_cast<long long>(blockIdx.x) * beside; t0 < rows;
         t0 += static_cast<long long>(gridDim.x) * beside) {
        const long long row = t0 + threadIdx.x / step;
        const bool on = row < rows;
        const long long t = on ? row : rows - 1;
        float h[kVecs][kN], v[kVecs][kN];
#pragma unroll
        for (int j = 0; j < kVecs; ++j)
            at.load(a.x, t * a.x_row, j, h[j]);
        if (a.branch) {
#pragma unroll
            for (int j = 0; j < kVecs; ++j)
                at.load(a.branch, t * a.branch_row, j, v[j]);
            long long gate = t * a.gate_row;
            if (a.cu) {
                // the sequence of the row: the last that begins there or before
                int lo = 0, hi = a.n_seqs;
                while (hi - lo > 1) {
                    const int mid = (lo + hi) >> 1;
                    (a.cu[mid] <= t ? lo : hi) = mid;
                }
                gate = lo * a.gate_row;
            }
            if (a.after_weight)
                norm_row<kType, kVectors, kVecs, kLayer>(a, at, v, a.after_weight, a.after_bias, team);
#pragma unroll
            for (int j = 0; j < kVecs; ++j) {
                if (a.gate) {
                    float g[kN];
                    at.load(a.gate, gate, j, g);
#pragma unroll
                    for (int e = 0; e < kN; ++e)
                        v[j][e] *= g[e];
                }
#pragma unroll
                for (int e = 0; e < kN; ++e)
                    h[j][e] = fmaf(a.residual_scale, h[j][e], v[j][e]);
                if (on)
                    at.store(a.h, t * a.h_row, j, h[j]);
            }
        }
        if (a.weight) {
            norm_row<kType, kVectors, kVecs, kLayer>(a, at, h, a.weight, a.bias, team);
#pragma unroll
            for (int j = 0; j < kVecs; ++j)
                if (on)
                    at.store(a.y, t * a.y_row, j, h[j]);
        }
    }
    pdl_trigger();
}

template <int kType, bool kVectors, int kVecs, bool kLayer>
cudaError_t launch(const ResidualNormArgs &a, int num_sms, cudaStream_t stream)
{
    static PerDeviceOnce once;
    const int step = a.lanes * a.warps;
    const int threads = a.warps > 1 ? step : 256;
    int fit = 0;
    auto *kernel = residual_norm_kernel<kType, kVectors, kVecs, kLayer>;
    const cudaError_t e = per_device_once(once, &fit, [&](int *out) {
        int regs = 0;
        cudaFuncAttributes f;
        const cudaError_t r = cudaFuncGetAttributes(&f, kernel);
        regs = f.numRegs > 0 ? f.numRegs : 64;
        *out = 65536 / (32 * ((regs + 7) / 8 * 8));       // warps on one SM
        return r;
    });
    if (e != cudaSuccess)
        return e;
    const int beside = threads / step;
    const long long need = (a.rows + beside - 1) / beside;
    const int per_sm = fit * 32 / threads > 0 ? fit * 32 / threads : 1;
    const long long most = static_cast<long long>(num_sms) * (per_sm < 2048 / threads ? per_sm : 2048 / threads);
    return launch_chained(kernel, dim3(static_cast<unsigned>(need < most ? need : most)), dim3(threads), 0, stream, a);
}

template <int kType, bool kVectors, bool kLayer>
cudaError_t launch(const ResidualNormArgs &a, int vecs, int num_sms, cudaStream_t stream)
{
    if constexpr (kType == MBERT_F32) {
        if (vecs > 6)
            return launch<kType, kVectors, 8, kLayer>(a, num_sms, stream);
        if (vecs > 4)
            return launch<kType, kVectors, 6, kLayer>(a, num_sms, stream);
    }
    switch (vecs) {
    case 1: return launch<kType, kVectors, 1, kLayer>(a, num_sms, stream);
    case 2: return launch<kType, kVectors, 2, kLayer>(a, num_sms, stream);
    case 3: return launch<kType, kVectors, 3, kLayer>(a, num_sms, stream);
    default: return launch<kType, kVectors, 4, kLayer>(a, num_sms, stream);
    }
}

template <int kType>
cudaError_t launch(ResidualNormArgs &a, bool layer, int num_sms, cudaStream_t stream)
{
    constexpr int kN = Row<kType, true>::kN, kMost = kLaneNumbers / kN;
    const int vecs = (a.width + kN - 1) / kN;           // of a row
    // up to 32 lanes take a row, then more vectors each, then more warps
    a.lanes = 1;
    while (a.lanes < 32 && a.lanes < vecs)
        a.lanes *= 2;
    a.warps = (vecs + 32 * kMost - 1) / (32 * kMost);
    const int step = a.lanes * a.warps, each = (vecs + step - 1) / step;
    if (a.vectors)
        return layer ? launch<kType, true, true>(a, each, num_sms, stream)
                     : launch<kType, true, false>(a, each, num_sms, stream);
    return layer ? launch<kType, false, true>(a, each, num_sms, stream)
                 : launch<kType, false, false>(a, each, num_sms, stream);
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
