// Products of any width for few rows (sm_103a): the same as linear.cu, whose head
// has the formulas, for calls and groups of few rows: up to 2048 in the mean, where it is
// estimated to be the faster (host_linear.cu).
//
// Bound by the weights, which are read once: 2 N K bytes against 2 T N K operations.
// So the operands change places: D^T = W x^T with 128 weight rows as M and 16 to 128
// rows of x as N, which wastes little of an MMA on rows that are not there, and the
// bytes of W are spread evenly over the SMs:
//  * output columns go by granules of 32, in pieces of 1 to 4 granules, as many as
//    leave the CTAs (one or two an SM) the least to do.  All pieces, row tile after row tile
//    and group after group, are dealt out in even runs.  An MMA of fewer than 4 granules
//    leaves the rest of its 128 rows to whatever shared memory holds behind them, and
//    nobody reads those.  (24 rows, 768 -> 50368 bf16, 525 pieces of 3 granules on 304 CTAs:
//    16.0 us, 4.9 TB/s; pieces of 4 in turn 18.4; even runs of granules, cut into pieces by
//    each CTA, 17.1, and 25.8 against 23.1 for -> 80000.)
//  * where there are too few columns to fill the SMs, the inner dimension is cut among 2,
//    4 or 8 CTAs of a cluster.  Each writes its sums into the others' shared memory, rows
//    of x dealt out among them, and each adds up its rows' parts in the order of the
//    CTAs: the result does not depend on timing, and there is no second kernel and no
//    workspace.
//  * stages of the ring are as large as the call's pieces, so that short pieces do not
//    leave the SM waiting for a few bytes at a time.
// Roles: warp 0 producer (TMA, a ring of stages of 64 numbers of K), warp 1 MMA
// issuer, warps 2 - 9 epilogue, one output column per thread and 16 rows at a time, which
// a warp writes as whole vectors through a tile of its own in shared memory (four warps
// that wrote number by number took 10 us for 128 rows).  Two accumulators in turn.
// 4001 rows of 64 experts, 768 -> 2 x 1152 fp16 with SiLU and biases: 44 to 45 us (242 MB,
// 5.4 TB/s) against 63 with those four warps and 68 by linear.cu.
// What bounds short calls: a warp needs 330 clocks from one step to the next, whatever
// it loads or multiplies (half of the MMAs, or one load for two, change nothing, nor do
// more warps that load), and a call 5 us beside its steps.
#include "linear.cuh"
#include "internal.h"
#include "pair.cuh"

namespace mbert {
namespace {

constexpr int kEpiWarps = 8;
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr int kM = kLinearGranule * kLinearGranules;
constexpr int kBK = 64;
constexpr uint32_t kGranuleBytes = kLinearGranule * kBK * 2;
constexpr int kMostStages = kLinearRowsStages;
constexpr int kBlock = 16;              // rows of x that an epilogue warp takes at a time
static_assert(kLinearGranule == 32, "a warp's columns");

template <int kNB, bool kGated>
struct Layout {
    static constexpr int kSides = kGated ? 2 : 1;
    static constexpr uint32_t kXBytes = kNB * kBK * 2;
    static constexpr int kCtas = linear_rows_ctas(kNB, kGated);
    static constexpr uint32_t kTmemCols = 2 * kSides * kNB;
    // shared memory: barriers, the epilogue warps' tiles of 16 rows x 32 results, the sums
    // that a cluster's CTAs exchange, the ring (x, then the granules of each side), and as
    // much behind it as an MMA reads beyond its piece
    static constexpr uint32_t kOffTiles = 1024, kTileBytes = kBlock * kLinearGranule * 2;
    static constexpr uint32_t kOffParts = kOffTiles + kEpiWarps * kTileBytes;
    static_assert(kOffParts + 1024 == kLinearRowsFixed, "shared memory");
    static constexpr uint32_t parts_bytes(int granules, int split)
    {
        return linear_rows_parts(kNB, kGated, granules, split);
    }
    static constexpr uint32_t stage_bytes(int granules) { return linear_rows_stage(kNB, kGated, granules); }
    static constexpr uint32_t behind(int granules) { return (kLinearGranules - granules) * kGranuleBytes; }
    static constexpr int stages(int granules, int split) { return linear_rows_stages(kNB, kGated, granules, split); }
    static constexpr uint32_t smem(int granules, int split)
    {
        return kLinearRowsFixed + parts_bytes(granules, split) + stages(granules, split) * stage_bytes(granules) +
               behind(granules);
    }
    static constexpr int kFull = 0, kEmpty = kMostStages, kAccFull = 2 * kMostStages, kAccEmpty = kAccFull + 2,
                         kBars = kAccEmpty + 2;
    static_assert(8 * kBars <= kOffTiles, "barriers");
    static_assert(stages(kLinearGranules, 1) >= 2 && kCtas * (linear_rows_budget(kNB, kGated) + 1040) <= 228 * 1024 &&
                  kCtas * kTmemCols <= 512,
                  "CTAs on one SM");
};

__device__ __forceinline__ void st_cluster_pair(uint32_t addr, uint32_t a, uint32_t b)
{
    asm volatile("st.shared::cluster.v2.b32 [%0], {%1, %2};" :: "r"(addr), "r"(a), "r"(b) : "memory");
}

__device__ __forceinline__ uint64_t lds_pair(uint32_t addr)
{
    uint64_t v;
    asm volatile("ld.shared.b64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ uint32_t cluster_nctarank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}

// A place in a ring of stages, and the stages gone through.
struct Ring {
    int done, slot;
    uint32_t parity;

    __device__ void step(int stages)
    {
        ++done;
        if (++slot == stages) {
            slot = 0;
            parity ^= 1;
        }
    }
};

// A CTA's pieces: granules `at` .. `at` + n of the unit's row tile, one after another.
// Called by all lanes of a warp.
class PieceWalk {
public:
    __device__ PieceWalk(const LinearArgs &a, int block, int split)
        : all_((a.outer + kLinearGranule - 1) / kLinearGranule), most_(a.granules),
          walk_(a, block, (all_ + most_ - 1) / most_, 1)
    {
        const long long units = count_units(a, block, (all_ + most_ - 1) / most_);
        const unsigned b = blockIdx.x / split, n = gridDim.x / split;
        valid_ = units >= 0;
        at_ = valid_ ? static_cast<int>(units * b / n) : 0;
        end_ = valid_ ? static_cast<int>(units * (b + 1ll) / n) : 0;
    }

    __device__ bool next(Unit &u, int &at, int &n)
    {
        if (at_ >= end_ || !walk_.find(at_, u))
            return false;
        at = u.column * most_;
        n = min(most_, all_ - at);
        ++at_;
        return true;
    }

    __device__ bool valid() const { return valid_; }

private:
    int all_, most_;
    UnitWalk walk_;
    bool valid_;
    int at_, end_;
};

// An epilogue thread's output column, in a warp's 32 of them.
template <bool kGated, bool kHalf>
struct Column {
    const LinearArgs &a;
    int f0, f;              // the warp's first column, this thread's
    bool on;                // within the row
    float bg = 0.f, bu = 0.f;

    __device__ Column(const LinearArgs &args, const Unit &u, int at, int quadrant) : a(args)
    {
        f0 = (at + quadrant) * kLinearGranule;
        f = f0 + threadIdx.x % 32;
        on = f < a.outer;
        const long long width = kGated ? 2ll * a.outer : a.outer;
        if (a.bias && on) {
            bg = load16<kHalf>(a.bias, u.group * width + f);
            if constexpr (kGated)
                bu = load16<kHalf>(a.bias, u.group * width + a.outer + f);
        }
    }

    // z (and w) of rows `row` and the next one, their weights -> the results as 16-bit
    // numbers; rows from `end` on are of no matter
    template <int kAct>
    __device__ uint32_t finish(long long row, long long end, uint64_t z, uint64_t w, uint64_t scale) const
    {
        z = activate2<kAct>(fadd2p(z, bc2(bg)));
        if constexpr (kGated)
            z = fmul2(z, fadd2p(w, bc2(bu)));
        if (a.row_scale)
            z = fmul2(z, scale);
        if (a.residual && on)
            z = fadd2p(z, f2(row < end ? load16<kHalf>(a.residual, row * a.residual_row + f) : 0.f,
                             row + 1 < end ? load16<kHalf>(a.residual, (row + 1) * a.residual_row + f) : 0.f));
        float lo, hi;
        f2_split(z, lo, hi);
        return pack2<kHalf>(lo, hi);
    }

    __device__ void put(long long row, long long end, uint32_t y) const
    {
        uint16_t *o = static_cast<uint16_t *>(a.out) + row * a.out_row + f;
        if (on && row < end)
            o[0] = static_cast<uint16_t>(y);
        if (on && row + 1 < end)
            o[a.out_row] = static_cast<uint16_t>(y >> 16);
    }
};

template <int kNB, bool kGated, bool kHalf>
__global__ void __launch_bounds__(kThreads, linear_rows_ctas(kNB, kGated))
linear_rows_kernel(const __grid_constant__ LinearArgs a)
{
    using L = Layout<kNB, kGated>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint32_t s_tmem, s_gave_up;
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;    // the same offset in every CTA of a cluster
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int split = static_cast<int>(cluster_nctarank()), rank = static_cast<int>(cluster_ctarank());
    const int stages = a.stages;
    const uint32_t ring = base + L::kOffParts + L::parts_bytes(a.granules, split);
    auto bar = [&](int i) { return base + 8u * i; };

    if (warp == 1) {
        // TMEM is taken when the kernel before has ended: one that lets this kernel start
        // before it has its own would wait for TMEM that is held here until it ends (0.1
        // to 0.2 us of a call)
        pdl_wait();
        tmem_alloc(smem_u32(&s_tmem), L::kTmemCols);
        tmem_relinquish();
    } else if (warp == 0) {
        if (lane == 0) {
            s_gave_up = 0;
            tma_prefetch_desc(&a.tm_x);
            tma_prefetch_desc(&a.tm_w);
        }
        for (int i = lane; i < L::kBars; i += 32)
            mbar_init(bar(i), i >= L::kAccEmpty ? kEpiWarps : 1);
        fence_mbar_init();
    }
    tc_fence_before();
    // with a cut every CTA of the cluster is there before another writes to it
    if (split > 1)
        cluster_sync();
    else
        __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    const int steps = (a.inner + kBK - 1) / kBK;
    const int k0 = steps * rank / split, k1 = steps * (rank + 1) / split;
    int *const err = a.err;
    const uint32_t gave_up = smem_u32(&s_gave_up);
    pdl_wait();
    PieceWalk walk(a, kNB, split);
    Unit u;
    int at, n;

    if (warp == 0) {
        // ------------------------------------------------------ producer
        Ring r{0, 0, 1};
        while (!any_gave_up(gave_up) && walk.next(u, at, n)) {
            for (int k = k0; k < k1; ++k, r.step(stages)) {
                // (after a wait that gives up nothing more is loaded)
                const bool go = mbar_wait_mark(bar(L::kEmpty + r.slot), r.parity, err, gave_up);
                const uint32_t dst = ring + r.slot * a.stage_bytes, full = bar(L::kFull + r.slot);
                if (elect_one_sync() && go) {
                    // (a row tile's last piece may have fewer granules: nobody reads the rest)
                    mbar_arrive_expect_tx(full, a.stage_bytes);
#pragma unroll
                    for (int s = 0; s < L::kSides; ++s)
                        tma_load_3d(dst + L::kXBytes + s * a.granules * kGranuleBytes, &a.tm_w, k * kBK,
                                    s * a.outer + at * kLinearGranule, u.group, full);
                    tma_load_2d(dst, &a.tm_x, k * kBK, static_cast<int>(u.row), full);
                }
                __syncwarp();
            }
        }
        // the loads have landed
        ring_drain(bar(L::kFull), r.done, stages);
    } else if (warp == 1) {
        // ------------------------------------------------------ MMA issuer
        constexpr uint32_t kIdesc = make_idesc_f16(kM, kNB, kHalf);
        // the descriptors of stage 0; a stage, a side and 16 numbers of K further on
        const uint64_t dx0 = make_sdesc_sw128(ring, 16, 1024), dw0 = make_sdesc_sw128(ring + L::kXBytes, 16, 1024);
        const uint32_t d_stage = a.stage_bytes >> 4, d_side = a.granules * kGranuleBytes >> 4;
        Ring r{0, 0, 0};
        for (int units = 0; !any_gave_up(gave_up) && walk.next(u, at, n); ++units) {
            const int acc = units & 1;
            const uint32_t d = tmem + acc * L::kSides * kNB;
            mbar_wait_mark(bar(L::kAccEmpty + acc), ((units >> 1) & 1) ^ 1u, err, gave_up);
            tc_fence_after();
            for (int k = k0; k < k1; ++k, r.step(stages)) {
                const uint64_t dx = dx0 + r.slot * d_stage, dw = dw0 + r.slot * d_stage;
                mbar_wait_mark(bar(L::kFull + r.slot), r.parity, err, gave_up);
                tc_fence_after();
                if (elect_one_sync()) {
#pragma unroll
                    for (int s = 0; s < L::kSides; ++s)
#pragma unroll
                        for (int kk = 0; kk < kBK / 16; ++kk)
                            mma_bf16_ss(d + s * kNB, dw + s * d_side + 2 * kk, dx + 2 * kk, kIdesc, k > k0 || kk > 0);
                    mma_commit(bar(L::kEmpty + r.slot));
                }
                __syncwarp();
            }
            mma_commit_warp(bar(L::kAccFull + acc));
        }
        // every MMA issued has completed before TMEM is released
        ring_drain(bar(L::kEmpty), r.done, stages);
        __syncwarp();
    } else {
        // ------------------------------------------------------ epilogue
        // TMEM quadrant q, that is a granule, and every other block of rows
        const int q = warp & 3, half = (warp - 2) >> 2;
        const int share = kNB / split, columns = a.granules * kLinearGranule;
        const uint32_t tile = base + L::kOffTiles + (warp - 2) * L::kTileBytes;
        for (int units = 0; walk.next(u, at, n); ++units) {
            const int acc = units & 1;
            const Column<kGated, kHalf> col(a, u, at, q);
            mbar_wait_mark(bar(L::kAccFull + acc), static_cast<uint32_t>(units >> 1) & 1u, err, gave_up);
            if (any_gave_up(gave_up))
                break;
            tc_fence_after();
            const uint32_t d = tmem + acc * L::kSides * kNB + (static_cast<uint32_t>(32 * q) << 16);
            const int rows = static_cast<int>(min(u.end - u.row, static_cast<long long>(kNB)));
            if (q < n) {
                with_activation(split > 1 ? MBERT_ACT_NONE : a.activation, [&](auto act) {
#pragma unroll 1
                    for (int j = kBlock * half; j < rows; j += 2 * kBlock) {
                        uint32_t zg[16], zu[16];
                        const float weight = a.row_scale && split == 1 && lane < kBlock && j + lane < rows
                                                 ? a.row_scale[u.row + j + lane] : 0.f;
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
                            // to the CTA whose share of the rows it is, two rows at a time:
                            // [CTA][side][pair of rows][column][2]
#pragma unroll
                            for (int e = 0; e < 16; e += 2) {
                                const int to = (j + e) / share, c = (j + e) % share;
                                const uint32_t p = map_to_rank(base + L::kOffParts +
                                    ((rank * L::kSides * share + c) * columns + 2 * (32 * q + lane)) * 4, to);
                                st_cluster_pair(p, zg[e], zg[e + 1]);
                                if constexpr (kGated)
                                    st_cluster_pair(p + share * columns * 4, zu[e], zu[e + 1]);
                            }
                            continue;
                        }
                        const long long row = u.row + j, end = u.row + rows;
                        uint32_t y[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            y[e] = col.template finish<decltype(act)::value>(
                                row + 2 * e, end, f2(__uint_as_float(zg[2 * e]), __uint_as_float(zg[2 * e + 1])),
                                kGated ? f2(__uint_as_float(zu[2 * e]), __uint_as_float(zu[2 * e + 1])) : 0ull,
                                f2(__shfl_sync(0xffffffffu, weight, 2 * e), __shfl_sync(0xffffffffu, weight, 2 * e + 1)));
                        if (!a.out_vectors) {
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                col.put(row + 2 * e, end, y[e]);
                            continue;
                        }
                        // through the warp's tile, to 8 columns of a row a thread
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            asm volatile("st.shared.b16 [%0], %1;"
                                         :: "r"(tile + e * 64 + 2 * lane), "h"(static_cast<uint16_t>(y[e / 2] >> 16 * (e & 1)))
                                         : "memory");
                        __syncwarp();
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            const int r = 8 * t + lane / 4, c = 8 * (lane & 3), left = a.outer - col.f0 - c;
                            uint4 v;
                            asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                                         : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(tile + r * 64 + 2 * c) : "memory");
                            uint16_t *o = static_cast<uint16_t *>(a.out) + (row + r) * a.out_row + col.f0 + c;
                            if (row + r < end && left >= 8) {
                                *reinterpret_cast<uint4 *>(o) = v;
                            } else if (row + r < end) {
                                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                                for (int e = 0; e < 8; ++e)
                                    if (e < left)
                                        o[e] = static_cast<uint16_t>(w[e / 2] >> 16 * (e & 1));
                            }
                        }
                        __syncwarp();
                    }
                });
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(bar(L::kAccEmpty + acc));
        }
    }
    __syncwarp();
    if (split > 1) {
        // all parts are written (a cluster has one piece at most)
        cluster_sync();
        __syncthreads();
        PieceWalk again(a, kNB, split);
        if (warp >= 2 && !any_gave_up(gave_up) && again.next(u, at, n) && (warp & 3) < n) {
            const int q = warp & 3, half = (warp - 2) >> 2;
            const Column<kGated, kHalf> col(a, u, at, q);
            const int share = kNB / split, columns = a.granules * kLinearGranule;
            const int rows = static_cast<int>(min(u.end - u.row, static_cast<long long>(kNB)));
            const uint32_t mine = base + L::kOffParts + 2 * (32 * q + lane) * 4;
            with_activation(a.activation, [&](auto act) {
                for (int c = 2 * half; c < share && rank * share + c < rows; c += 4) {
                    uint64_t z[2] = {};
                    for (int s = 0; s < split; ++s)
#pragma unroll
                        for (int side = 0; side < L::kSides; ++side)
                            z[side] = fadd2p(z[side], lds_pair(mine + ((s * L::kSides + side) * share + c) * columns * 4));
                    const long long row = u.row + rank * share + c, end = u.row + rows;
                    const uint64_t scale = a.row_scale ? f2(a.row_scale[row], row + 1 < end ? a.row_scale[row + 1] : 0.f) : 0ull;
                    col.put(row, end, col.template finish<decltype(act)::value>(row, end, z[0], z[1], scale));
                }
            });
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
cudaError_t launch(LinearArgs a, const LinearRowsPlan &p, cudaStream_t stream)
{
    using L = Layout<kNB, kGated>;
    static PerDeviceOnce once;
    auto *kernel = linear_rows_kernel<kNB, kGated, kHalf>;
    const cudaError_t e = smem_opt_in(once, kernel, linear_rows_budget(kNB, kGated));
    if (e != cudaSuccess)
        return e;
    a.granules = p.granules;
    a.stages = L::stages(p.granules, p.split);
    a.stage_bytes = static_cast<int>(L::stage_bytes(p.granules));
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = p.split;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.ctas * p.split));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = L::smem(p.granules, p.split);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <int kNB>
cudaError_t launch(const LinearArgs &a, const LinearRowsPlan &p, bool gated, bool half, cudaStream_t stream)
{
    return gated ? half ? launch<kNB, true, true>(a, p, stream) : launch<kNB, true, false>(a, p, stream)
                 : half ? launch<kNB, false, true>(a, p, stream) : launch<kNB, false, false>(a, p, stream);
}

}  // namespace

cudaError_t launch_linear_rows(const LinearArgs &a, const LinearRowsPlan &p, bool gated, bool half, cudaStream_t stream)
{
    switch (p.tile) {
    case 16: return launch<16>(a, p, gated, half, stream);
    case 32: return launch<32>(a, p, gated, half, stream);
    case 64: return launch<64>(a, p, gated, half, stream);
    default: return launch<128>(a, p, gated, half, stream);
    }
}

}  // namespace mbert
