// Products of any width with their epilogue (sm_103a): for every row t of a group
// with weight W [N][K] ([2N][K] where gated), bias b and row weight s
//     z = x_t W^T + b,   out_t = residual_t + s_t act(z)
//     gated: out_t = residual_t + s_t act(z_g) z_u,   z_g, z_u the halves of z
// bf16 or fp16, products and epilogue in fp32, one rounding.  One group (a linear
// layer) or ragged groups of rows with a weight each (experts), whose offsets are
// on the device.
//
// 2 T K N operations on (T K + N K + T N) numbers: bound by the tensor cores from a
// few hundred rows on.  As in projections.cu a pair of SMs shares an MMA of 256 rows
// x 256 columns (an SM's copy engine would feed a tile of 128 x 128 at half the
// MMA's rate only), D in two accumulators of TMEM, so that a unit's epilogue runs
// beside the next unit's products:
//   warp 0      producer (both CTAs): the CTA's 128 rows of x and its half of the
//               unit's weight rows, 64 numbers of K a stage; where gated the leader
//               holds rows of Wg and its peer those of Wu, so that D has z_g in its
//               left half and z_u in its right
//   warp 1      MMA issuer (leader)
//   the others  epilogue (both CTAs), a row of a TMEM lane per thread: quadrant
//               w % 4, a part of the unit's chunks of columns: 16 warps and chunks of 32
//               columns, 8 warps and chunks of 64 where gated, whose two halves of z
//               leave no registers for 16
// Each epilogue warp has two staging buffers of 32 rows x a chunk of its own and its own TMA
// stores from them (clipped at the last row and column by the tensor map), so no warp
// waits for another's rows; a residual comes into the buffer by TMA, the first two chunks'
// at the start and then each as the chunk before it is begun, and is overwritten by the
// result, so `out` may be the residual.
// A warp's bias numbers, 64 at most, come in a register or two while the unit's products run
// and go round by shuffles; read where they are added, as vectors, their latency shows: 62
// experts of about 127 rows, 80 -> 2 x 6720 with GELU, 187 us against 247.
// Rows that TMA cannot address (strides or addresses off 16 bytes) and the last rows
// of a group, behind which another group's begin, are copied from the buffer by
// plain loads and stores.
//
// Units go to the pairs in turn, group after group, by bands of 8 row blocks and
// within a band column after column: the units that run at one time then touch
// about 8 x 10 blocks, whose rows and weights stay in L2.
// Units of 256 x 128 accumulators serve calls with too few units for every pair.
//
// 32768 x 1024 -> 2 x 4096 bf16, GELU and gate: 277 to 289 us by board, 1.9 to 1.98
// PFLOP/s (1.62 to 1.66 under the power cap, where the same calls follow each other for
// seconds); without a gate the
// epilogue, 5000 clocks of a unit and 3700 more for GELU, shows: 325 us with it, 290
// without.  65536 rows of 8 experts, 768 -> 2 x 1152: 133 to 139 us by board; 1152 -> 768: 74 us,
// 780 units on 76 pairs in 11 rounds.
// Not kept (before the bias came ahead, when these calls took 140 and 331 us): the
// accumulators through fp32 tiles, 8 columns of a row a thread, plain stores: 150 and 351;
// 8 warps without a gate 339; an arrival at the leader's barrier with a release at the
// cluster's scope, which waits for stores: 144.
#include "linear.cuh"
#include "internal.h"
#include "pair.cuh"

namespace mbert {
namespace {

constexpr int kBM = kLinearRows / 2;            // rows per CTA
constexpr int kBK = 64;
constexpr int kBand = 8;
constexpr uint32_t kXBytes = kBM * kBK * 2;
constexpr uint16_t kPairMask = 0x3;
constexpr unsigned long long kDrainLimitNs = 100000000ull;

template <int kBN, bool kGated>
struct Layout {
    // epilogue warps, and the output columns of one's staging buffers of 32 rows
    static constexpr int kEpiWarps = kGated ? 8 : 16, kChunk = linear_chunk(kGated);
    static constexpr int kParts = kEpiWarps / 4, kThreads = 64 + 32 * kEpiWarps;
    static constexpr uint32_t kBufBytes = 32 * kChunk * 2;
    static constexpr int kStages = kBN == 256 ? 5 : 6;
    static constexpr uint32_t kStageBytes = kXBytes + kBN / 2 * kBK * 2;
    static constexpr uint32_t kOffBuf = kStages * kStageBytes;
    static constexpr uint32_t kOffBar = kOffBuf + 2 * kEpiWarps * kBufBytes;
    static constexpr uint32_t kSmemBytes = kOffBar + 512 + 1024;
    static constexpr int kOutCols = kGated ? kBN / 2 : kBN;
    // the chunks of a unit's columns are dealt to the warps of a quadrant; where there are
    // half as many, half of the warps take every other unit
    static constexpr int kChunks = kOutCols / kChunk;
    static constexpr int kWarpChunks = kChunks > kParts ? kChunks / kParts : 1;
    static constexpr bool kInTurns = kChunks < kParts;
    static_assert(kWarpChunks * kChunk <= 64, "a warp's bias");
    static_assert(kInTurns ? 2 * kChunks == kParts : kChunks % kParts == 0, "chunks");
    static constexpr int kReaders = 2 * kEpiWarps / (kInTurns ? 2 : 1);
    // barriers
    static constexpr int kFull = 0, kEmpty = kStages, kAccFull = 2 * kStages, kAccEmpty = kAccFull + 2,
                         kDrain = kAccEmpty + 2, kResidual = kDrain + 1, kBars = kResidual + 2 * kEpiWarps;
    static_assert(8 * kBars <= 512 && kSmemBytes + 16 <= 227 * 1024, "shared memory");
};

__device__ __forceinline__ void bulk_wait_read1() { asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory"); }

// vector c of a row of a staging buffer, in the order of the 128-byte swizzle (rows of
// 64 columns: bits 4 to 6 of the address exclusive-or bits 7 to 9) or of the 64-byte one
// (32 columns: bits 4 and 5, bits 7 and 8)
template <int kChunk>
__device__ __forceinline__ uint32_t chunk_addr(uint32_t buf, int row, int c)
{
    return kChunk == 64 ? buf + row * 128 + ((c ^ (row & 7)) << 4) : buf + row * 64 + ((c ^ (row >> 1 & 3)) << 4);
}

// Bias numbers of 64 columns from n on, two a lane, 0 behind `width`.
__device__ __forceinline__ uint32_t bias_lanes(const void *bias, long long base, int n, int width)
{
    const uint16_t *b = static_cast<const uint16_t *>(bias) + base;
    n += 2 * (threadIdx.x & 31);
    return (n < width ? b[n] : 0u) | (n + 1 < width ? b[n + 1] : 0u) << 16;
}

// z += b for 8 columns, whose bias numbers four lanes from `from` on hold
template <bool kHalf>
__device__ __forceinline__ void add_bias(uint64_t (&z)[4], uint32_t lanes, int from)
{
#pragma unroll
    for (int e = 0; e < 4; ++e)
        z[e] = fadd2p(z[e], unpack2<kHalf>(__shfl_sync(0xffffffffu, lanes, from + e)));
}

// A warp's copy of 32 rows x kChunk columns of 16-bit numbers by words of kBytes, lane
// by lane along the rows.  Words that reach beyond the last column go number by number.
template <int kChunk, int kBytes>
struct Copy {
    static constexpr int kN = kBytes / 2, kWords = kChunk / kN;     // of a row
    static constexpr int kTimes = kWords;                           // words of a lane
    // words of a lane in a row, rows from one row of a lane to its next
    static constexpr int kInRow = kWords > 32 ? kWords / 32 : 1, kRowStep = kWords > 32 ? 1 : 32 / kWords;
    using Word = std::conditional_t<kBytes == 8, uint64_t, std::conditional_t<kBytes == 4, uint32_t, uint16_t>>;

    static __device__ int row(int t) { return (32 * t + (threadIdx.x & 31)) / kWords; }
    static __device__ int column(int t) { return (32 * t + (threadIdx.x & 31)) % kWords * kN; }

    static __device__ Word load(const uint16_t *p, int c, bool on, int columns)
    {
        Word w = 0;
        if (on && c + kN <= columns) {
            w = *reinterpret_cast<const Word *>(p + c);
        } else if (on) {
#pragma unroll
            for (int e = 0; e < kN; ++e)
                if (c + e < columns)
                    w |= static_cast<Word>(static_cast<Word>(p[c + e]) << 16 * e);
        }
        return w;
    }
    static __device__ void store(uint16_t *p, int c, bool on, int columns, Word w)
    {
        if (on && c + kN <= columns) {
            *reinterpret_cast<Word *>(p + c) = w;
        } else if (on) {
#pragma unroll
            for (int e = 0; e < kN; ++e)
                if (c + e < columns)
                    p[c + e] = static_cast<uint16_t>(w >> 16 * e);
        }
    }
    static __device__ void to_shared(uint32_t addr, Word w)
    {
        if constexpr (kBytes == 8)
            asm volatile("st.shared.b64 [%0], %1;" :: "r"(addr), "l"(w) : "memory");
        else if constexpr (kBytes == 4)
            asm volatile("st.shared.b32 [%0], %1;" :: "r"(addr), "r"(w) : "memory");
        else
            asm volatile("st.shared.b16 [%0], %1;" :: "r"(addr), "h"(w) : "memory");
    }
    static __device__ Word from_shared(uint32_t addr)
    {
        Word w;
        if constexpr (kBytes == 8)
            asm volatile("ld.shared.b64 %0, [%1];" : "=l"(w) : "r"(addr) : "memory");
        else if constexpr (kBytes == 4)
            asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w) : "r"(addr) : "memory");
        else
            asm volatile("ld.shared.b16 %0, [%1];" : "=h"(w) : "r"(addr) : "memory");
        return w;
    }
};

// f(integral constant) for words of 8, 4 or 2 bytes
template <typename F>
__device__ __forceinline__ void with_bytes(int bytes, F &&f)
{
    if (bytes >= 8)
        f(std::integral_constant<int, 8>());
    else if (bytes == 4)
        f(std::integral_constant<int, 4>());
    else
        f(std::integral_constant<int, 2>());
}

template <int kBN, bool kGated, bool kHalf>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Layout<kBN, kGated>::kThreads, 1)
linear_kernel(const __grid_constant__ LinearArgs a)
{
    using L = Layout<kBN, kGated>;
    constexpr int kChunk = L::kChunk;
    constexpr uint32_t kBufBytes = L::kBufBytes;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint32_t s_tmem;
    pdl_wait();
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;    // the same offset in both CTAs
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = static_cast<int>(cluster_ctarank());
    const bool leader = rank == 0;
    const int cluster = blockIdx.x >> 1, clusters = gridDim.x >> 1;
    auto bar = [&](int i) { return base + L::kOffBar + 8u * i; };

    if (warp == 1) {
        tmem_alloc_pair(smem_u32(&s_tmem), 2 * kBN);
        tmem_relinquish_pair();
    } else if (tid == 0) {
        tma_prefetch_desc(&a.tm_x);
        tma_prefetch_desc(&a.tm_w);
        for (int i = 0; i < L::kBars; ++i)
            mbar_init(bar(i), i == L::kAccEmpty || i == L::kAccEmpty + 1 ? L::kReaders : 1);
        fence_mbar_init();
    }
    bool ok = offsets_ok(a);                             // (the same in both CTAs)
    tc_fence_before();
    cluster_sync();                                      // both CTAs' barriers and TMEM exist
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    // The pair's accumulators must sit at the same TMEM address in both CTAs.
    if (ld_shared_cluster_u32(map_to_rank(smem_u32(&s_tmem), rank ^ 1)) != tmem) {
        if (tid == 0)
            atomicOr(a.err, kErrPairTmem);
        ok = false;
    }
    const int columns = (a.outer + L::kOutCols - 1) / L::kOutCols;
    const int steps = (a.inner + kBK - 1) / kBK;
    int *const err = a.err;
    if (ok) {
        UnitWalk walk(a, kLinearRows, columns, kBand);
        Unit u;
        if (warp == 0) {
            // -------------------------------------------------- producer
            const uint64_t keep = l2_policy_evict_last();    // rows and weights: read again by other units
            int g = 0;
            auto x_row = [&](const Unit &v) { return static_cast<int>(v.row) + rank * kBM; };
            auto w_row = [&](const Unit &v) {
                return kGated ? rank * a.outer + v.column * L::kOutCols : v.column * kBN + rank * (kBN / 2);
            };
            bool more = walk.find(cluster, u);
            for (int i = cluster; ok && more; i += clusters) {
                const int m0 = x_row(u), w0 = w_row(u), group = u.group;
                // the next unit's boxes go to L2 a unit ahead, by the unit that is the first to
                // need them
                more = i <= INT32_MAX - clusters && walk.find(i + clusters, u);
                const bool next_x = more && u.column == 0, next_w = more && u.first;
                for (int k = 0; k < steps; ++k, ++g) {
                    const int st = g % L::kStages;
                    if (!(ok = mbar_wait_warp(bar(L::kEmpty + st), ((g / L::kStages) & 1) ^ 1u, err)))
                        break;
                    if (elect_one_sync()) {
                        const uint32_t dst = base + st * L::kStageBytes;
                        const uint32_t full = map_to_rank(bar(L::kFull + st), 0);
                        if (leader)                      // both CTAs' boxes land on the leader's barrier
                            mbar_arrive_expect_tx(bar(L::kFull + st), 2 * L::kStageBytes);
                        tma_load_2d_pair(dst, &a.tm_x, k * kBK, m0, full, keep);
                        tma_load_3d_pair(dst + kXBytes, &a.tm_w, k * kBK, w0, group, full, keep);
                        if (next_x)
                            tma_prefetch_2d(&a.tm_x, k * kBK, x_row(u));
                        if (next_w)
                            tma_prefetch_3d(&a.tm_w, k * kBK, w_row(u), u.group);
                    }
                    __syncwarp();
                }
            }
            // every stage this CTA loaded has been read by the pair's MMAs
            for (int t = max(0, g - L::kStages); t < g; ++t)
                mbar_wait(bar(L::kEmpty + t % L::kStages), (t / L::kStages) & 1, err, kDrainLimitNs);
        } else if (warp == 1) {
            // -------------------------------------------------- MMA issuer
            if (leader) {
                constexpr uint32_t kIdesc = make_idesc_f16(kLinearRows, kBN, kHalf);
                int g = 0, n = 0;
                for (int i = cluster; ok && walk.find(i, u); i += clusters, ++n) {
                    const int acc = n & 1;
                    const uint32_t d = tmem + acc * kBN;
                    if (!(ok = mbar_wait_warp(bar(L::kAccEmpty + acc), ((n >> 1) & 1) ^ 1u, err)))
                        break;
                    tc_fence_after();
                    for (int k = 0; k < steps; ++k, ++g) {
                        const int st = g % L::kStages;
                        if (!(ok = mbar_wait_warp(bar(L::kFull + st), (g / L::kStages) & 1, err)))
                            break;
                        tc_fence_after();
                        const uint32_t sx = base + st * L::kStageBytes, sw = sx + kXBytes;
#pragma unroll
                        for (int kk = 0; kk < kBK / 16; ++kk)
                            mma_pair_warp(d, make_sdesc_sw128(sx + 32 * kk, 16, 1024),
                                          make_sdesc_sw128(sw + 32 * kk, 16, 1024), kIdesc, k > 0 || kk > 0);
                        mma_commit_pair_warp(bar(L::kEmpty + st), kPairMask);
                    }
                    if (ok)
                        mma_commit_pair_warp(bar(L::kAccFull + acc), kPairMask);
                }
                // every MMA issued has completed before TMEM is released
                mma_commit_pair_warp(bar(L::kDrain), 0x1);
                mbar_wait(bar(L::kDrain), 0, err, kDrainLimitNs);
            }
        } else {
            // -------------------------------------------------- epilogue
            const int q = warp & 3, part = (warp - 2) >> 2;
            const uint32_t buf0 = base + L::kOffBuf + (warp - 2) * 2 * kBufBytes;
            const int rbar = L::kResidual + 2 * (warp - 2);
            const bool residual = a.residual != nullptr, residual_vectors = residual && a.residual_vectors;
            const int width = kGated ? 2 * a.outer : a.outer;
            // chunk `ch` of this warp's in a unit
            auto column_of = [&](const Unit &v, int ch) {
                const int chunk = L::kInTurns ? part % L::kChunks : part * L::kWarpChunks + ch;
                return v.column * L::kOutCols + kChunk * chunk;
            };
            // the residual of this warp's chunk `seq`, over the units that come to it (one
            // group only)
            auto load_residual = [&](int seq) {
                const int n = L::kInTurns ? 2 * seq + part / L::kChunks : seq / L::kWarpChunks;
                Unit v;
                const long long i = cluster + static_cast<long long>(n) * clusters;
                if (i > INT32_MAX || !walk.find(static_cast<int>(i), v))
                    return false;
                if (lane == 0) {
                    const uint32_t b = bar(rbar + (seq & 1));
                    mbar_arrive_expect_tx(b, kBufBytes);
                    tma_load_2d(buf0 + (seq & 1) * kBufBytes, &a.tm_residual, column_of(v, seq % L::kWarpChunks),
                                static_cast<int>(v.row) + rank * kBM + 32 * q, b);
                }
                return true;
            };
            int seq = 0, loads = 0;
            if (residual_vectors) {
                while (loads < 2 && load_residual(loads))
                    ++loads;
            }
            int n = 0;
            for (int i = cluster; ok && walk.find(i, u); i += clusters, ++n) {
                if (L::kInTurns && (n & 1) != part / L::kChunks)
                    continue;
                const int acc = n & 1;
                const long long row0 = u.row + rank * kBM + 32 * q;
                const int left = static_cast<int>(min(u.end - row0, 32ll));      // rows of this warp (may be < 1)
                const float scale = a.row_scale && lane < left ? a.row_scale[row0 + lane] : 1.f;
                // the bias of this warp's columns, on its way while the products are
                uint32_t bg = 0, bu = 0;
                if (a.bias) {
                    const long long bias0 = static_cast<long long>(u.group) * width;
                    bg = bias_lanes(a.bias, bias0, column_of(u, 0), a.outer);
                    if constexpr (kGated)
                        bu = bias_lanes(a.bias, bias0 + a.outer, column_of(u, 0), a.outer);
                }
                if (!(ok = mbar_wait_warp(bar(L::kAccFull + acc), static_cast<uint32_t>(n >> 1) & 1u, err)))
                    break;
                tc_fence_after();
                const uint32_t d = tmem + acc * kBN + (static_cast<uint32_t>(32 * q) << 16);
#pragma unroll 1
                for (int ch = 0; ch < L::kWarpChunks; ++ch, ++seq) {
                    const int n0 = column_of(u, ch);
                    const uint32_t buf = buf0 + (seq & 1) * kBufBytes;
                    // the buffer: the residual is in it, or its last store has been read
                    if (residual_vectors) {
                        if (seq > 0) {
                            if (lane == 0)
                                bulk_wait_read0();
                            __syncwarp();
                            if (load_residual(seq + 1))
                                ++loads;
                        }
                        if (!(ok = mbar_wait_warp(bar(rbar + (seq & 1)), static_cast<uint32_t>(seq >> 1) & 1u, err)))
                            break;
                    } else {
                        if (lane == 0)
                            bulk_wait_read1();
                        __syncwarp();
                        if (residual) {
                            with_bytes(a.residual_bytes, [&](auto bytes) {
                                using C = Copy<kChunk, decltype(bytes)::value>;
                                typename C::Word w[C::kTimes];
                                const uint16_t *p = static_cast<const uint16_t *>(a.residual) +
                                                    (row0 + C::row(0)) * a.residual_row + n0;
#pragma unroll
                                for (int t = 0; t < C::kTimes; ++t) {
                                    w[t] = C::load(p, C::column(t), C::row(t) < left, a.outer - n0);
                                    if ((t + 1) % C::kInRow == 0)
                                        p += C::kRowStep * a.residual_row;
                                }
#pragma unroll
                                for (int t = 0; t < C::kTimes; ++t)
                                    C::to_shared(chunk_addr<kChunk>(buf, C::row(t), C::column(t) / 8) + 2 * (C::column(t) & 7), w[t]);
                            });
                            __syncwarp();
                        }
                    }
                    const bool last = ch == L::kWarpChunks - 1;
                    auto release = [&] {
                        // the accumulator may be used again: one arrival per warp at the leader
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0)
                            mbar_arrive_cluster(map_to_rank(bar(L::kAccEmpty + acc), 0));
                    };
                    if (left <= 0 || n0 >= a.outer) {
                        // no row or no column of this chunk is there
                        if (last)
                            release();
                        if (lane == 0)
                            bulk_commit();
                        continue;
                    }
#pragma unroll 1
                    for (int piece = 0; piece < kChunk / 32; ++piece) {
                        const int p0 = n0 + 32 * piece;
                        uint32_t zg[32], zu[kGated ? 32 : 1];
                        tmem_ld32(d + p0 - u.column * L::kOutCols, zg);
                        if constexpr (kGated)
                            tmem_ld32(d + L::kOutCols + p0 - u.column * L::kOutCols, zu);
                        tmem_wait_ld();
                        reg_fence32(zg);
                        if constexpr (kGated)
                            reg_fence32(zu);
                        if (piece == kChunk / 32 - 1 && last)
                            release();
                        with_activation(a.activation, [&](auto act) {
#pragma unroll
                            for (int c = 0; c < 4; ++c) {
                                uint64_t z[4], w[4];
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    z[e] = f2(__uint_as_float(zg[8 * c + 2 * e]), __uint_as_float(zg[8 * c + 2 * e + 1]));
                                    if constexpr (kGated)
                                        w[e] = f2(__uint_as_float(zu[8 * c + 2 * e]), __uint_as_float(zu[8 * c + 2 * e + 1]));
                                }
                                if (a.bias) {
                                    const int from = ch * (kChunk / 2) + 16 * piece + 4 * c;
                                    add_bias<kHalf>(z, bg, from);
                                    if constexpr (kGated)
                                        add_bias<kHalf>(w, bu, from);
                                }
                                const uint32_t at = chunk_addr<kChunk>(buf, lane, 4 * piece + c);
                                uint32_t x[4] = {};
                                if (residual)
                                    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                                                 : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(at));
                                uint32_t y[4];
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    z[e] = activate2<decltype(act)::value>(z[e]);
                                    if constexpr (kGated)
                                        z[e] = fmul2(z[e], w[e]);
                                    z[e] = fmul2(z[e], bc2(scale));
                                    if (residual)
                                        z[e] = fadd2p(z[e], unpack2<kHalf>(x[e]));
                                    float lo, hi;
                                    f2_split(z[e], lo, hi);
                                    y[e] = pack2<kHalf>(lo, hi);
                                }
                                asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};"
                                             :: "r"(at), "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3]) : "memory");
                            }
                        });
                    }
                    // the chunk to global memory: by TMA where the map ends with the rows (one
                    // group) and with the columns (it clips whole vectors of 16 bytes only)
                    const bool whole = (left == 32 || !a.cu) && (n0 + kChunk <= a.outer || a.outer % 8 == 0);
                    if (a.out_vectors && whole) {
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0)
                            tma_store_2d(&a.tm_out, buf, n0, static_cast<int>(row0));
                    } else {
                        __syncwarp();
                        with_bytes(a.out_bytes, [&](auto bytes) {
                            using C = Copy<kChunk, decltype(bytes)::value>;
                            uint16_t *p = static_cast<uint16_t *>(a.out) + (row0 + C::row(0)) * a.out_row + n0;
#pragma unroll
                            for (int t = 0; t < C::kTimes; ++t) {
                                C::store(p, C::column(t), C::row(t) < left, a.outer - n0,
                                         C::from_shared(chunk_addr<kChunk>(buf, C::row(t), C::column(t) / 8) + 2 * (C::column(t) & 7)));
                                if ((t + 1) % C::kInRow == 0)
                                    p += C::kRowStep * a.out_row;
                            }
                        });
                        __syncwarp();
                        fence_proxy_async_smem();                // before a load or store by TMA
                        __syncwarp();
                    }
                    if (lane == 0)
                        bulk_commit();      // one group a chunk, if an empty one: the waits above count them
                }
            }
            tmem_wait_ld();
            if (lane == 0) {
                // residuals still on their way after a wait that gave up
                for (int t = seq; t < loads; ++t)
                    mbar_wait(bar(rbar + (t & 1)), static_cast<uint32_t>(t >> 1) & 1u, err, kDrainLimitNs);
                bulk_wait0();                                    // the stores have completed
            }
        }
        __syncwarp();
    }

    tc_fence_before();
    cluster_sync();                   // neither CTA exits while the other may still signal it
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, 2 * kBN);
    }
    pdl_trigger();
}

template <int kBN, bool kGated, bool kHalf>
cudaError_t launch(const LinearArgs &a, long long units, int num_sms, cudaStream_t stream)
{
    using L = Layout<kBN, kGated>;
    static PerDeviceOnce once;
    auto *kernel = linear_kernel<kBN, kGated, kHalf>;
    int fit = 0;
    const cudaError_t e = per_device_once(once, &fit, [&](int *out) {
        cudaError_t r = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(L::kSmemBytes));
        if (r != cudaSuccess)
            return r;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(2 * (num_sms / 2));
        cfg.blockDim = dim3(L::kThreads);
        cfg.dynamicSmemBytes = L::kSmemBytes;
        int n = 0;
        r = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
        *out = n > 0 ? n : 1;
        return r;
    });
    if (e != cudaSuccess)
        return e;
    const int pairs = static_cast<int>(units < fit ? units : fit);
    return launch_chained(kernel, dim3(2 * pairs), dim3(L::kThreads), L::kSmemBytes, stream, a);
}

}  // namespace

cudaError_t launch_linear(const LinearArgs &a, int columns, bool gated, bool half, long long units, int num_sms,
                          cudaStream_t stream)
{
    if (columns == 256)
        return gated ? half ? launch<256, true, true>(a, units, num_sms, stream)
                            : launch<256, true, false>(a, units, num_sms, stream)
                     : half ? launch<256, false, true>(a, units, num_sms, stream)
                            : launch<256, false, false>(a, units, num_sms, stream);
    return gated ? half ? launch<128, true, true>(a, units, num_sms, stream)
                        : launch<128, true, false>(a, units, num_sms, stream)
                 : half ? launch<128, false, true>(a, units, num_sms, stream)
                        : launch<128, false, false>(a, units, num_sms, stream);
}

}  // namespace mbert
