// Products of any width for few rows (sm_103a): the same as linear.cu, whose head
// has the formulas, for calls and groups of up to about a hundred rows.
//
// Bound by the weights, which are read once: 2 N K bytes against 2 T N K operations.
// So the operands change places: D^T = W x^T with 128 weight rows as M and 16 to 128
// rows of x as N, which wastes little of an MMA on rows that are not there, and the
// bytes of W are spread over all SMs:
//  * one CTA per 128 output columns (and `tile` rows of x), one or two CTAs an SM,
//    so that 90 KB or more of weights are on their way to each SM;
//  * where that leaves SMs idle, the inner dimension is cut among 2, 4 or 8 CTAs of
//    a cluster.  Each writes its sums into the others' shared memory, rows of x dealt
//    out among them, and each adds up its rows' parts in the order of the CTAs: the
//    result does not depend on timing, and there is no second kernel and no workspace.
// Roles: warp 0 producer (TMA, a ring of stages of 64 numbers of K), warp 1 MMA
// issuer, warps 2 - 5 epilogue, one output column per thread, the rows one after
// another: a warp writes 64 bytes of a row at a time.
// Without a cut the CTAs are persistent, with two accumulators in turn.  Within a
// group the units go column by column with the row tiles inside, so a weight tile that
// several row tiles need is read from L2.
#include "linear.cuh"
#include "internal.h"
#include "pair.cuh"

namespace mbert {
namespace {

constexpr int kThreads = 192;
constexpr int kEpiThreads = 128;
constexpr int kM = kLinearRowsColumns;
constexpr int kBK = 64;
constexpr uint32_t kWBytes = kM * kBK * 2;

template <int kNB, bool kGated>
struct Layout {
    static constexpr int kSides = kGated ? 2 : 1;
    static constexpr uint32_t kStageBytes = kSides * kWBytes + kNB * kBK * 2;
    static constexpr int kCtas = linear_rows_ctas(kNB, kGated);
    // two CTAs: up to 108 KB each; one: up to 192 KB
    static constexpr int kStages = kCtas == 2 ? 108 * 1024 / kStageBytes : kNB == 64 ? 4 : 192 * 1024 / kStageBytes;
    static constexpr uint32_t kOffBar = kStages * kStageBytes;
    static constexpr uint32_t kOffParts = kOffBar + 256;
    // with a cut: every CTA's sums of this CTA's share of the rows
    static constexpr uint32_t kPartsBytes = kSides * kNB * kM * 4;
    static constexpr uint32_t smem(int split) { return kOffParts + (split > 1 ? kPartsBytes : 0) + 1024; }
    static constexpr uint32_t kTmemCols = 2 * kSides * kNB;
    static constexpr int kFull = 0, kEmpty = kStages, kAccFull = 2 * kStages, kAccEmpty = kAccFull + 2,
                         kBars = kAccEmpty + 2;
    static_assert(8 * kBars <= 256 && smem(linear_rows_most_split(kNB, kGated)) + 16 <= 227 * 1024, "shared memory");
    static_assert(kCtas * (smem(1) + 1040) <= 228 * 1024 && kCtas * kTmemCols <= 512, "CTAs on one SM");
};

__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v)
{
    asm volatile("st.shared::cluster.f32 [%0], %1;" :: "r"(addr), "f"(v) : "memory");
}

__device__ __forceinline__ float lds_f32(uint32_t addr)
{
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ uint32_t cluster_nctarank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}

// What an epilogue thread writes: its output column of some rows.
template <bool kGated, bool kHalf>
struct Column {
    const LinearArgs &a;
    long long f;            // output column
    float bg = 0.f, bu = 0.f;

    __device__ Column(const LinearArgs &args, const Unit &u) : a(args)
    {
        f = static_cast<long long>(u.column) * kM + 32 * (threadIdx.x / 32 % 4) + threadIdx.x % 32;
        const long long width = kGated ? 2 * a.outer : a.outer;
        if (a.bias && f < a.outer) {
            bg = load16<kHalf>(a.bias, u.group * width + f);
            if constexpr (kGated)
                bu = load16<kHalf>(a.bias, u.group * width + a.outer + f);
        }
    }

    // rows `row` and the next one, where they lie before `end`
    __device__ void put(long long row, long long end, uint64_t z, uint64_t w) const
    {
        z = fadd2p(z, bc2(bg));
        if constexpr (kGated)
            w = fadd2p(w, bc2(bu));
        with_activation(a.activation, [&](auto act) { z = activate2<decltype(act)::value>(z); });
        if constexpr (kGated)
            z = fmul2(z, w);
        float y[2];
        f2_split(z, y[0], y[1]);
        if (f >= a.outer)
            return;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            if (row + e >= end)
                return;
            if (a.row_scale)
                y[e] *= a.row_scale[row + e];
            if (a.residual)
                y[e] += load16<kHalf>(a.residual, (row + e) * a.residual_row + f);
            static_cast<uint16_t *>(a.out)[(row + e) * a.out_row + f] = static_cast<uint16_t>(pack2<kHalf>(y[e], 0.f));
        }
    }
};

template <int kNB, bool kGated, bool kHalf>
__global__ void __launch_bounds__(kThreads, linear_rows_ctas(kNB, kGated))
linear_rows_kernel(const __grid_constant__ LinearArgs a)
{
    using L = Layout<kNB, kGated>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint32_t s_tmem;
    pdl_wait();
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;    // the same offset in every CTA of a cluster
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int split = static_cast<int>(cluster_nctarank()), rank = static_cast<int>(cluster_ctarank());
    const int first = blockIdx.x / split, stride = gridDim.x / split;
    auto bar = [&](int i) { return base + L::kOffBar + 8u * i; };

    if (warp == 1) {
        tmem_alloc(smem_u32(&s_tmem), L::kTmemCols);
        tmem_relinquish();
    } else if (tid == 0) {
        tma_prefetch_desc(&a.tm_x);
        tma_prefetch_desc(&a.tm_w);
        for (int i = 0; i < L::kBars; ++i)
            mbar_init(bar(i), i >= L::kAccEmpty ? kEpiThreads / 32 : 1);
        fence_mbar_init();
    }
    const bool valid = offsets_ok(a);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    const int columns = (a.outer + kM - 1) / kM;
    const int steps = (a.inner + kBK - 1) / kBK;
    const int k0 = steps * rank / split, k1 = steps * (rank + 1) / split;
    int *const err = a.err;
    bool ok = valid;
    UnitWalk walk(a, kNB, columns, INT32_MAX);
    Unit u;
    // with a cut every CTA of the cluster is there before another writes to it
    if (split > 1)
        cluster_sync();

    if (valid && warp == 0) {
        // ------------------------------------------------------ producer
        int g = 0;
        for (int i = first; ok && walk.find(i, u); i += stride) {
            for (int k = k0; k < k1; ++k, ++g) {
                const int st = g % L::kStages;
                if (!(ok = mbar_wait_warp(bar(L::kEmpty + st), ((g / L::kStages) & 1) ^ 1u, err)))
                    break;
                if (elect_one_sync()) {
                    const uint32_t dst = base + st * L::kStageBytes, full = bar(L::kFull + st);
                    mbar_arrive_expect_tx(full, L::kStageBytes);
#pragma unroll
                    for (int s = 0; s < L::kSides; ++s)
                        tma_load_3d(dst + s * kWBytes, &a.tm_w, k * kBK, s * a.outer + u.column * kM, u.group, full);
                    tma_load_2d(dst + L::kSides * kWBytes, &a.tm_x, k * kBK, static_cast<int>(u.row), full);
                }
                __syncwarp();
            }
        }
        // the loads have landed and the MMAs have read them
        for (int t = max(0, g - L::kStages); t < g; ++t)
            drain_wait(bar(L::kFull + t % L::kStages), (t / L::kStages) & 1);
    } else if (valid && warp == 1) {
        // ------------------------------------------------------ MMA issuer
        constexpr uint32_t kIdesc = make_idesc_f16(kM, kNB, kHalf);
        int g = 0, n = 0;
        for (int i = first; ok && walk.find(i, u); i += stride, ++n) {
            const int acc = n & 1;
            const uint32_t d = tmem + acc * L::kSides * kNB;
            if (!(ok = mbar_wait_warp(bar(L::kAccEmpty + acc), ((n >> 1) & 1) ^ 1u, err)))
                break;
            tc_fence_after();
            for (int k = k0; k < k1; ++k, ++g) {
                const int st = g % L::kStages;
                if (!(ok = mbar_wait_warp(bar(L::kFull + st), (g / L::kStages) & 1, err)))
                    break;
                tc_fence_after();
                const uint32_t sw = base + st * L::kStageBytes, sx = sw + L::kSides * kWBytes;
#pragma unroll
                for (int s = 0; s < L::kSides; ++s)
#pragma unroll
                    for (int kk = 0; kk < kBK / 16; ++kk)
                        mma_bf16_ss_warp(d + s * kNB, make_sdesc_sw128(sw + s * kWBytes + 32 * kk, 16, 1024),
                                         make_sdesc_sw128(sx + 32 * kk, 16, 1024), kIdesc, k > k0 || kk > 0);
                mma_commit_warp(bar(L::kEmpty + st));
            }
            if (ok)
                mma_commit_warp(bar(L::kAccFull + acc));
        }
        // every MMA issued has completed before TMEM is released
        for (int t = max(0, g - L::kStages); t < g; ++t)
            drain_wait(bar(L::kEmpty + t % L::kStages), (t / L::kStages) & 1);
    } else if (valid) {
        // ------------------------------------------------------ epilogue
        const int q = warp & 3;
        const uint32_t lanes = static_cast<uint32_t>(32 * q) << 16;
        int n = 0;
        for (int i = first; ok && walk.find(i, u); i += stride, ++n) {
            const int acc = n & 1;
            const Column<kGated, kHalf> col(a, u);
            if (!(ok = mbar_wait_warp(bar(L::kAccFull + acc), static_cast<uint32_t>(n >> 1) & 1u, err)))
                break;
            tc_fence_after();
            const uint32_t d = tmem + acc * L::kSides * kNB + lanes;
            const int rows = static_cast<int>(min(u.end - u.row, static_cast<long long>(kNB)));
            const int share = kNB / split;
#pragma unroll 1
            for (int j = 0; j < kNB; j += 16) {
                if (j >= rows)
                    break;
                uint32_t zg[16], zu[16];
                tmem_ld16(d + j, zg);
                if constexpr (kGated)
                    tmem_ld16(d + kNB + j, zu);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    asm volatile("" : "+r"(zg[e]));
                    if constexpr (kGated)
                        asm volatile("" : "+r"(zu[e]));
                }
                if (split > 1) {
                    // to the CTA whose share of the rows it is: [CTA][side][row][column]
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const int to = (j + e) / share, c = (j + e) % share;
                        const uint32_t at = base + L::kOffParts +
                            (((rank * L::kSides * share) + c) * kM + 32 * q + lane) * 4;
                        const uint32_t p = map_to_rank(at, to);
                        st_cluster_f32(p, __uint_as_float(zg[e]));
                        if constexpr (kGated)
                            st_cluster_f32(p + share * kM * 4, __uint_as_float(zu[e]));
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 16; e += 2)
                        col.put(u.row + j + e, u.row + rows, f2(__uint_as_float(zg[e]), __uint_as_float(zg[e + 1])),
                                kGated ? f2(__uint_as_float(zu[e]), __uint_as_float(zu[e + 1])) : 0ull);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(bar(L::kAccEmpty + acc));
        }
    }
    __syncwarp();
    if (split > 1) {
        // all parts are written (the launch gives a cluster one unit at most)
        cluster_sync();
        const int all_ok = __syncthreads_and(ok);
        UnitWalk again(a, kNB, columns, INT32_MAX);
        if (valid && warp >= 2 && all_ok && again.find(first, u)) {
            const Column<kGated, kHalf> col(a, u);
            const int share = kNB / split, rows = static_cast<int>(min(u.end - u.row, static_cast<long long>(kNB)));
            const uint32_t mine = base + L::kOffParts + (32 * (warp & 3) + lane) * 4;
            for (int c = 0; c < share && rank * share + c < rows; c += 2) {
                float z[2][2] = {};
                for (int s = 0; s < split; ++s)
#pragma unroll
                    for (int side = 0; side < L::kSides; ++side)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            z[side][e] += lds_f32(mine + ((s * L::kSides + side) * share + c + e) * kM * 4);
                const long long row = u.row + rank * share + c;
                col.put(row, u.row + rows, f2(z[0][0], z[0][1]), f2(z[1][0], z[1][1]));
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, L::kTmemCols);
    }
    pdl_trigger();
}

template <int kNB, bool kGated, bool kHalf>
cudaError_t launch(const LinearArgs &a, int split, long long units, int num_sms, cudaStream_t stream)
{
    using L = Layout<kNB, kGated>;
    static PerDeviceOnce once;
    auto *kernel = linear_rows_kernel<kNB, kGated, kHalf>;
    const cudaError_t e = smem_opt_in(once, kernel, L::smem(linear_rows_most_split(kNB, kGated)));
    if (e != cudaSuccess)
        return e;
    const long long most = static_cast<long long>(num_sms) * L::kCtas;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = split;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(split > 1 ? units * split : units < most ? units : most));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = L::smem(split);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <int kNB>
cudaError_t launch(const LinearArgs &a, int split, bool gated, bool half, long long units, int num_sms,
                   cudaStream_t stream)
{
    return gated ? half ? launch<kNB, true, true>(a, split, units, num_sms, stream)
                        : launch<kNB, true, false>(a, split, units, num_sms, stream)
                 : half ? launch<kNB, false, true>(a, split, units, num_sms, stream)
                        : launch<kNB, false, false>(a, split, units, num_sms, stream);
}

}  // namespace

cudaError_t launch_linear_rows(const LinearArgs &a, int tile, int split, bool gated, bool half, long long units,
                               int num_sms, cudaStream_t stream)
{
    switch (tile) {
    case 16: return launch<16>(a, split, gated, half, units, num_sms, stream);
    case 32: return launch<32>(a, split, gated, half, units, num_sms, stream);
    case 64: return launch<64>(a, split, gated, half, units, num_sms, stream);
    default: return launch<128>(a, split, gated, half, units, num_sms, stream);
    }
}

}  // namespace mbert
