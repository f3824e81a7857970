// Attention of packed queries over keys and values of another length, for
// blocks of queries: a persistent, warp-specialised tcgen05 pipeline.
//
//   out_i = sum_j softmax_j(scale q_i . k_j) v_j,  j over the visible keys of
//   i's sequence; 0 where there is none
//
// Work: a unit is 256 query rows of one sequence and head (two tiles of 128);
// units and their 128-key tiles are split among one CTA per SM by cost
// (cross_sched.cuh), and units cut between CTAs are joined by a second kernel
// (cross_join.cu) in a fixed order.  Query heads that share a key head read
// the same key columns; the copies after the first come from L2.
//
// CTA (12 warps):
//   warps 0-3   softmax group 0 (query tile 0, TMEM lanes 0..127, a thread a row)
//   warps 4-7   softmax group 1 (query tile 1)
//   warp  8     TMA producer: Q, K and V rings
//   warps 9,10  MMA issuers, one per query tile
//   warp  11    masks: the key bits of a tile to shared memory, and zeros over
//               the V rows that nothing may see (a weight of 0 times an
//               infinity there would be NaN)
// TMEM (512 columns), fp32 except P (16-bit pairs):
//   D = 64:   S0 S1 (128 each), P0 P1 (64 each), O0 O1 (64 each); S of the next
//             tile is computed while the softmax works on this one
//   D = 128:  S0 S1, O0 O1 (128 each); P takes the first half of its S, so S
//             of the next tile follows P V of this one, and the two query
//             tiles fill each other's gaps
//
// Softmax: online, in base 2, held in fp32.  The reference m moves (and O is
// rescaled) only when a tile's maximum passes it by more than 8, so weights
// stay below 2^8.  In fp16 they are taken times 2^7: the largest is 2^15,
// inside fp16's range, and the smallest normal one is 2^-21 of the largest
// instead of 2^-14, so a long tail of small weights keeps its share.
#include <type_traits>

#include "common.cuh"
#include "cross_sched.cuh"
#include "internal.h"

namespace mbert {
namespace {

constexpr int kThreads = 384;
constexpr int kRegsSoftmax = 216;   // 4 x 72 + 8 x 216 = 12 x 168 (the launch budget)
constexpr int kRegsControl = 72;
constexpr int kMaskSlots = 4;

// A unit's fixed work costs about four key tiles (the query load, the refill
// of the pipeline, the end of the softmax, the output).
using Split = CrossSplit<kThreads, kCrossBlockRows, kBlockN, 4, 4>;

template <int D>
struct Layout {
    static constexpr bool kAlias = D == 128;            // P lies in its S
    static constexpr int kHalves = D / 64;              // 64-column boxes of a tile
    static constexpr uint32_t kTile = kHalves * kTileBytes;
    static constexpr int kQSets = D == 64 ? 2 : 1;      // of two query tiles
    static constexpr int kStages = D == 64 ? 3 : 2;     // of K and of V
    static constexpr uint32_t kOffK = kQSets * 2 * kTile;
    static constexpr uint32_t kOffV = kOffK + kStages * kTile;
    static constexpr uint32_t kOffBar = kOffV + kStages * kTile;
    static constexpr uint32_t kOffWords = kOffBar + 512;            // key bits, kMaskSlots x 4 words
    static constexpr uint32_t kOffScratch = kOffWords + 16 * kMaskSlots;
    static constexpr uint32_t kSmemBytes = kOffScratch + sizeof(Split::Scratch) + 1024;
    static constexpr uint32_t col_s(int w) { return 128u * w; }
    static constexpr uint32_t col_p(int w) { return kAlias ? 128u * w : 256u + 64u * w; }
    static constexpr uint32_t col_o(int w) { return kAlias ? 256u + 128u * w : 384u + 64u * w; }
};
static_assert(Layout<64>::kSmemBytes <= 232448 && Layout<128>::kSmemBytes <= 232448, "shared memory");

// barrier slots (8 bytes each)
constexpr int kBarQFull = 0;      // + set (2)
constexpr int kBarQEmpty = 2;     // + set
constexpr int kBarKFull = 4;      // + stage (3)
constexpr int kBarKEmpty = 7;
constexpr int kBarVFull = 10;
constexpr int kBarVEmpty = 13;
constexpr int kBarSFull = 16;     // + group (2)
constexpr int kBarSEmpty = 18;    // D = 64 only
constexpr int kBarPFull = 20;
constexpr int kBarODone = 22;
constexpr int kBarOFree = 24;
constexpr int kBarBitsFull = 26;  // + mask slot (4): a tile's key bits are in shared memory
constexpr int kBarBitsEmpty = 30; // + mask slot: read by all 256 softmax threads
constexpr int kBarVClean = 34;    // + mask slot: a tile's unseen V rows are zeros
constexpr int kNumBars = 38;
constexpr uint32_t kSlotInBars = 8 * kNumBars;                 // TMEM address
static_assert(kSlotInBars + 4 <= 512, "barriers");

constexpr uint32_t kTmemCols = 512;
constexpr float kRescaleThreshold = 8.0f;

// kind::f16 instruction descriptor for either 16-bit type (A and B alike)
__device__ __forceinline__ constexpr uint32_t idesc(int M, int N, bool b_mn_major, bool half)
{
    const uint32_t d = make_idesc_bf16(M, N, b_mn_major);
    return half ? d & ~((7u << 7) | (7u << 10)) : d;
}

struct Ctx {
    uint32_t base;          // 1024-aligned shared address
    uint32_t tmem;
    uint8_t *sbase;         // generic pointer to the same address
    const CrossArgs &a;
    const Split &split;
    uint32_t bars;
};

__device__ __forceinline__ uint32_t bar(const Ctx &c, int i) { return c.bars + 8u * i; }

// A tile whose keys are not all visible (or not known to be).
__device__ __forceinline__ bool needs_mask(const Ctx &c, const Split::Seg &s, int k)
{
    return c.a.key_bits != nullptr || s.s.k_len - k * kBlockN < kBlockN;
}

// The unit's second query tile holds rows.
__device__ __forceinline__ bool second_tile(const Split::Seg &s) { return s.s.q_len - s.q0 > kBlockM; }

// ---------------------------------------------------------------- producer
template <int D>
__device__ void producer(const Ctx &c)
{
    using L = Layout<D>;
    int *err = c.a.err;
    auto it = c.split.begin();
    Split::Seg s;
    uint32_t g = 0;          // key tiles issued by this CTA so far
    for (uint32_t sg = 0; c.split.next(it, s); ++sg) {
        const int qs = sg % L::kQSets;
        const bool two = second_tile(s);
        if (sg >= L::kQSets && !mbar_wait(bar(c, kBarQEmpty + qs), (sg / L::kQSets - 1) & 1, err))
            return;
        const int col_q = s.head * D, col_k = s.head / c.a.group * D;
        const int qrow = s.s.q_row + s.q0;
        const uint32_t qdst = c.base + qs * 2 * L::kTile;
        mbar_arrive_expect_tx(bar(c, kBarQFull + qs), (two ? 2 : 1) * L::kTile);
        for (int w = 0; w < (two ? 2 : 1); ++w)
            for (int h = 0; h < L::kHalves; ++h)
                tma_load_2d(qdst + w * L::kTile + h * kTileBytes, &c.a.tm_q, col_q + 64 * h, qrow + w * kBlockM,
                            bar(c, kBarQFull + qs));
        for (int k = s.kb; k < s.ke; ++k, ++g) {
            const int st = g % L::kStages;
            const uint32_t u = g / L::kStages;
            const int krow = s.s.k_row + k * kBlockN;
            if (u > 0 && !mbar_wait(bar(c, kBarKEmpty + st), (u - 1) & 1, err))
                return;
            mbar_arrive_expect_tx(bar(c, kBarKFull + st), L::kTile);
            for (int h = 0; h < L::kHalves; ++h)
                tma_load_2d(c.base + L::kOffK + st * L::kTile + h * kTileBytes, &c.a.tm_k, col_k + 64 * h, krow,
                            bar(c, kBarKFull + st));
            if (u > 0 && !mbar_wait(bar(c, kBarVEmpty + st), (u - 1) & 1, err))
                return;
            mbar_arrive_expect_tx(bar(c, kBarVFull + st), L::kTile);
            for (int h = 0; h < L::kHalves; ++h)
                tma_load_2d(c.base + L::kOffV + st * L::kTile + h * kTileBytes, &c.a.tm_v, col_k + 64 * h, krow,
                            bar(c, kBarVFull + st));
        }
    }
}

// ---------------------------------------------------------------- MMA issuers
template <int D, bool kHalf>
__device__ __forceinline__ void issue_s(const Ctx &c, int w, int qs, int st)
{
    using L = Layout<D>;
    constexpr uint32_t kIdesc = idesc(128, 128, false, kHalf);
    const uint32_t q = c.base + (qs * 2 + w) * L::kTile;
    const uint32_t k = c.base + L::kOffK + st * L::kTile;
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = (kk / 4) * kTileBytes + 32 * (kk % 4);
        mma_bf16_ss_warp(c.tmem + L::col_s(w), make_sdesc_sw128(q + off, 16, 1024),
                         make_sdesc_sw128(k + off, 16, 1024), kIdesc, kk > 0);
    }
}

template <int D, bool kHalf>
__device__ __forceinline__ void issue_o(const Ctx &c, int w, int st, bool accumulate)
{
    using L = Layout<D>;
    // 64 columns of O per instruction: with P read from TMEM they run at the
    // full rate
    constexpr uint32_t kIdesc = idesc(128, 64, true, kHalf);
    const uint32_t v = c.base + L::kOffV + st * L::kTile;
#pragma unroll
    for (int kk = 0; kk < kBlockN / 16; ++kk)
#pragma unroll
        for (int h = 0; h < L::kHalves; ++h)
            mma_bf16_ts_warp(c.tmem + L::col_o(w) + 64 * h, c.tmem + L::col_p(w) + 8 * kk,
                             make_sdesc_sw128(v + h * kTileBytes + 2048 * kk, 1024, 1024), kIdesc,
                             (accumulate || kk > 0) ? 1u : 0u);
}

// A segment whose second query tile is empty: issuer 1 hands the ring slots
// back as they fill (each phase only once it has begun).
template <int D>
__device__ bool pass_segment(const Ctx &c, const Split::Seg &s, int qs, uint32_t sg, uint32_t g0, int lane)
{
    using L = Layout<D>;
    int *err = c.a.err;
    if (!mbar_wait(bar(c, kBarQFull + qs), (sg / L::kQSets) & 1, err))
        return false;
    for (int t = 0; t < s.ke - s.kb; ++t) {
        const uint32_t g = g0 + t;
        const int st = g % L::kStages;
        if (!mbar_wait(bar(c, kBarKFull + st), (g / L::kStages) & 1, err) ||
            !mbar_wait(bar(c, kBarVFull + st), (g / L::kStages) & 1, err))
            return false;
        if (lane == 0) {
            mbar_arrive(bar(c, kBarKEmpty + st));
            mbar_arrive(bar(c, kBarVEmpty + st));
        }
        __syncwarp();
    }
    if (lane == 0)
        mbar_arrive(bar(c, kBarQEmpty + qs));
    __syncwarp();
    return true;
}

// Issuer for query tile w.  `gw` counts the tiles of this query tile (its S,
// P and O barriers), `g` all tiles of the CTA (the rings).
template <int D, bool kHalf>
__device__ void mma_issuer(const Ctx &c, int w, int lane)
{
    using L = Layout<D>;
    int *err = c.a.err;
    auto it = c.split.begin();
    Split::Seg s;
    uint32_t g0 = 0, gw0 = 0, sw = 0, masked = 0;
    for (uint32_t sg = 0; c.split.next(it, s); ++sg) {
        const int qs = sg % L::kQSets;
        const int n = s.ke - s.kb;
        if (w == 1 && !second_tile(s)) {
            if (!pass_segment<D>(c, s, qs, sg, g0, lane))
                return;
            for (int t = 0; t < n; ++t)
                masked += needs_mask(c, s, s.kb + t);
            g0 += n;
            continue;
        }
        if (!mbar_wait(bar(c, kBarQFull + qs), (sg / L::kQSets) & 1, err))
            return;
        // P V of tile t
        auto step_o = [&](int t) -> bool {
            const uint32_t g = g0 + t, gw = gw0 + t;
            const int st = g % L::kStages;
            if (!mbar_wait(bar(c, kBarVFull + st), (g / L::kStages) & 1, err))
                return false;
            if (needs_mask(c, s, s.kb + t)) {
                if (!mbar_wait(bar(c, kBarVClean + masked % kMaskSlots), (masked / kMaskSlots) & 1, err))
                    return false;
                ++masked;
            }
            if (!mbar_wait(bar(c, kBarPFull + w), gw & 1, err))
                return false;
            if (t == 0 && sw > 0 && !mbar_wait(bar(c, kBarOFree + w), (sw - 1) & 1, err))
                return false;
            __syncwarp();
            tc_fence_after();
            issue_o<D, kHalf>(c, w, st, t > 0);
            mma_commit_warp(bar(c, kBarODone + w));
            mma_commit_warp(bar(c, kBarVEmpty + st));
            return true;
        };
        for (int t = 0; t < n; ++t) {
            const uint32_t g = g0 + t, gw = gw0 + t;
            const int st = g % L::kStages;
            if (!mbar_wait(bar(c, kBarKFull + st), (g / L::kStages) & 1, err))
                return;
            if constexpr (L::kAlias) {
                // S takes the place of the last tile's P
                if (gw > 0 && !mbar_wait(bar(c, kBarODone + w), (gw - 1) & 1, err))
                    return;
            } else {
                if (gw > 0 && !mbar_wait(bar(c, kBarSEmpty + w), (gw - 1) & 1, err))
                    return;
            }
            __syncwarp();
            tc_fence_after();
            issue_s<D, kHalf>(c, w, qs, st);
            mma_commit_warp(bar(c, kBarSFull + w));
            mma_commit_warp(bar(c, kBarKEmpty + st));
            if (t == n - 1)
                mma_commit_warp(bar(c, kBarQEmpty + qs));
            // D = 64: P V one tile behind, while the softmax works on tile t
            if (L::kAlias ? !step_o(t) : (t > 0 && !step_o(t - 1)))
                return;
        }
        if (!L::kAlias && !step_o(n - 1))
            return;
        g0 += n;
        gw0 += n;
        ++sw;
    }
}

// ---------------------------------------------------------------- masks
// The visible keys of tile k as 4 words.
__device__ __forceinline__ uint32_t tile_word(const Ctx &c, const Split::Seg &s, int k, int i)
{
    const int left = s.s.k_len - k * kBlockN - 32 * i;
    uint32_t w = left >= 32 ? 0xffffffffu : left > 0 ? (1u << left) - 1u : 0u;
    if (w && c.a.key_bits)
        w &= __ldg(c.a.key_bits + key_bit_word(s.s.k_row, s.seq) + 4 * k + i);
    return w;
}

template <int D>
__device__ void mask_stager(const Ctx &c, int lane)
{
    using L = Layout<D>;
    int *err = c.a.err;
    auto it = c.split.begin();
    Split::Seg s;
    uint32_t g = 0, masked = 0;
    for (uint32_t sg = 0; c.split.next(it, s); ++sg) {
        for (int k = s.kb; k < s.ke; ++k, ++g) {
            const int st = g % L::kStages;
            // every tile is waited for and handed back, seen or not, so that
            // this warp neither runs ahead of the ring nor falls behind it
            if (!needs_mask(c, s, k)) {
                if (!mbar_wait(bar(c, kBarVFull + st), (g / L::kStages) & 1, err))
                    return;
                if (lane == 0)
                    mbar_arrive(bar(c, kBarVEmpty + st));
                __syncwarp();
                continue;
            }
            const uint32_t slot = masked % kMaskSlots, u = masked / kMaskSlots;
            ++masked;
            const uint32_t mine = lane < 4 ? tile_word(c, s, k, lane) : 0u;
            if (c.a.key_bits) {
                if (u > 0 && !mbar_wait(bar(c, kBarBitsEmpty + slot), (u - 1) & 1, err))
                    return;
                if (lane < 4)
                    reinterpret_cast<uint32_t *>(c.sbase + L::kOffWords)[4 * slot + lane] = mine;
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(bar(c, kBarBitsFull + slot));
            }
            if (!mbar_wait(bar(c, kBarVFull + st), (g / L::kStages) & 1, err))
                return;
            __syncwarp();
#pragma unroll 1
            for (int i = 0; i < 4; ++i) {
                const uint32_t word = __shfl_sync(0xffffffffu, mine, i);
                if (word == 0xffffffffu)
                    continue;
                // 16 bytes of each of 32 rows per step (rows' order does not
                // matter for zeros: a row is 128 contiguous bytes per half)
                uint8_t *v = c.sbase + L::kOffV + st * L::kTile + 32 * i * 128;
                for (int j = lane; j < 32 * 8 * L::kHalves; j += 32) {
                    const int row = j / 8 % 32, part = j % 8, half = j / 256;
                    if (!(word >> row & 1))
                        *reinterpret_cast<uint4 *>(v + half * kTileBytes + row * 128 + part * 16) =
                            make_uint4(0u, 0u, 0u, 0u);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(bar(c, kBarVClean + slot));
                mbar_arrive(bar(c, kBarVEmpty + st));
            }
            __syncwarp();
        }
    }
}

// ---------------------------------------------------------------- softmax
template <bool kHalf>
__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    uint32_t r;
    if constexpr (kHalf)
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

template <int D, bool kHalf>
__device__ void softmax_group(const Ctx &c, int w, int warp_in_group, int lane, int cta)
{
    using L = Layout<D>;
    constexpr float kLift = kHalf ? 7.f : 0.f;        // weights times 2^7 in fp16
    int *err = c.a.err;
    const uint32_t lane_off = static_cast<uint32_t>(32 * warp_in_group) << 16;
    const uint32_t tS = c.tmem + L::col_s(w) + lane_off;
    const uint32_t tP = c.tmem + L::col_p(w) + lane_off;
    const uint32_t tO = c.tmem + L::col_o(w) + lane_off;
    const int rr = kBlockM * w + 32 * warp_in_group + lane;      // row within the unit
    const float scale = c.a.scale_log2;
    auto it = c.split.begin();
    Split::Seg s;
    uint32_t gw = 0, masked = 0;
    while (c.split.next(it, s)) {
        const int n = s.ke - s.kb;
        if (w == 1 && !second_tile(s)) {
            // nothing to do but hand the key bits on
            for (int t = 0; t < n; ++t) {
                if (!needs_mask(c, s, s.kb + t))
                    continue;
                if (c.a.key_bits) {
                    const uint32_t slot = masked % kMaskSlots;
                    if (!mbar_wait(bar(c, kBarBitsFull + slot), (masked / kMaskSlots) & 1, err))
                        return;
                    mbar_arrive(bar(c, kBarBitsEmpty + slot));
                }
                ++masked;
            }
            continue;
        }
        float m = -INFINITY;    // reference (scaled, base 2)
        float l = 0.f;          // sum of exp2(score - m + kLift)
        for (int t = 0; t < n; ++t, ++gw) {
            if (!mbar_wait(bar(c, kBarSFull + w), gw & 1, err))
                return;
            __syncwarp();
            tc_fence_after();
            float sc[kBlockN];
            {
                uint32_t r0[32], r1[32], r2[32], r3[32];
                tmem_ld32(tS, r0);
                tmem_ld32(tS + 32, r1);
                tmem_ld32(tS + 64, r2);
                tmem_ld32(tS + 96, r3);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    sc[i] = __uint_as_float(r0[i]);
                    sc[32 + i] = __uint_as_float(r1[i]);
                    sc[64 + i] = __uint_as_float(r2[i]);
                    sc[96 + i] = __uint_as_float(r3[i]);
                }
            }
            tc_fence_before();
            if constexpr (!L::kAlias)
                mbar_arrive(bar(c, kBarSEmpty + w));   // S may be overwritten now

            if (needs_mask(c, s, s.kb + t)) {
                if (c.a.key_bits) {
                    const uint32_t slot = masked % kMaskSlots;
                    if (!mbar_wait(bar(c, kBarBitsFull + slot), (masked / kMaskSlots) & 1, err))
                        return;
                    const uint4 b = reinterpret_cast<const uint4 *>(c.sbase + L::kOffWords)[slot];
                    mbar_arrive(bar(c, kBarBitsEmpty + slot));
                    if ((b.x & b.y & b.z & b.w) != 0xffffffffu) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            if (!(b.x >> i & 1))
                                sc[i] = -INFINITY;
                            if (!(b.y >> i & 1))
                                sc[32 + i] = -INFINITY;
                            if (!(b.z >> i & 1))
                                sc[64 + i] = -INFINITY;
                            if (!(b.w >> i & 1))
                                sc[96 + i] = -INFINITY;
                        }
                    }
                } else {
                    const int kvalid = s.s.k_len - (s.kb + t) * kBlockN;
#pragma unroll
                    for (int i = 0; i < kBlockN; ++i)
                        if (i >= kvalid)
                            sc[i] = -INFINITY;
                }
                ++masked;
            }
            // row maximum: 8 independent chains
            float mp[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
                mp[k] = fmaxf(sc[k], sc[8 + k]);
#pragma unroll
            for (int i = 16; i < kBlockN; i += 16)
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    mp[k] = fmax3(mp[k], sc[i + k], sc[i + 8 + k]);
            const float mc = fmaxf(fmax3(mp[0], mp[1], mp[2]),
                                   fmaxf(fmax3(mp[3], mp[4], mp[5]), fmaxf(mp[6], mp[7]))) * scale;
            const bool need = mc > m + kRescaleThreshold;
            const float mn = need ? mc : m;
            const float alpha = need ? ex2_approx(m - mn) : 1.f;
            // no visible key so far: every exponent is -inf, not -inf + inf
            const float neg = mn == -INFINITY ? 0.f : kLift - mn;

            // p = 2^(s scale - m), packed to 16-bit pairs; the row sum in 4
            // packed fp32x2 accumulators
            uint32_t pk[kBlockN / 2];
            uint64_t acc2[4] = {0ull, 0ull, 0ull, 0ull};
            const uint64_t sc2 = f2(scale, scale), nm2 = f2(neg, neg);
#pragma unroll
            for (int i = 0; i < kBlockN / 2; ++i) {
                if constexpr (kHalf)
                    asm("{\n\t.reg .b64 y, pp;\n\t.reg .f32 y0, y1, p0, p1;\n\t"
                        "mov.b64 y, {%2, %3};\n\t"
                        "fma.rn.f32x2 y, y, %4, %5;\n\t"
                        "mov.b64 {y0, y1}, y;\n\t"
                        "ex2.approx.ftz.f32 p0, y0;\n\t"
                        "ex2.approx.ftz.f32 p1, y1;\n\t"
                        "mov.b64 pp, {p0, p1};\n\t"
                        "add.f32x2 %1, %1, pp;\n\t"
                        "cvt.rn.f16x2.f32 %0, p1, p0;\n\t}"
                        : "=r"(pk[i]), "+l"(acc2[i & 3])
                        : "f"(sc[2 * i]), "f"(sc[2 * i + 1]), "l"(sc2), "l"(nm2));
                else
                    asm("{\n\t.reg .b64 y, pp;\n\t.reg .f32 y0, y1, p0, p1;\n\t"
                        "mov.b64 y, {%2, %3};\n\t"
                        "fma.rn.f32x2 y, y, %4, %5;\n\t"
                        "mov.b64 {y0, y1}, y;\n\t"
                        "ex2.approx.ftz.f32 p0, y0;\n\t"
                        "ex2.approx.ftz.f32 p1, y1;\n\t"
                        "mov.b64 pp, {p0, p1};\n\t"
                        "add.f32x2 %1, %1, pp;\n\t"
                        "cvt.rn.bf16x2.f32 %0, p1, p0;\n\t}"
                        : "=r"(pk[i]), "+l"(acc2[i & 3])
                        : "f"(sc[2 * i]), "f"(sc[2 * i + 1]), "l"(sc2), "l"(nm2));
            }
            uint64_t accs = acc2[0];
            asm("add.f32x2 %0, %0, %1;" : "+l"(accs) : "l"(acc2[1]));
            asm("add.f32x2 %0, %0, %1;" : "+l"(accs) : "l"(acc2[2]));
            asm("add.f32x2 %0, %0, %1;" : "+l"(accs) : "l"(acc2[3]));
            float acc0, acc1;
            f2_split(accs, acc0, acc1);

            if (t > 0) {
                // P and O are free once the last P V has completed (D = 128:
                // S of this tile was only issued after that)
                if constexpr (!L::kAlias) {
                    if (!mbar_wait(bar(c, kBarODone + w), (gw - 1) & 1, err))
                        return;
                    __syncwarp();
                    tc_fence_after();
                }
                if (__any_sync(0xffffffffu, need)) {
#pragma unroll
                    for (int h = 0; h < D / 32; ++h) {
                        uint32_t o[32];
                        tmem_ld32(tO + 32 * h, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                        tmem_st32(tO + 32 * h, o);
                    }
                }
            }
            l = l * alpha + (acc0 + acc1);
            m = mn;
            tmem_st64(tP, pk);
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(bar(c, kBarPFull + w));
        }

        // ---- end of the segment: O / l to the output, or the state to this
        // CTA's part slot
        if (!mbar_wait(bar(c, kBarODone + w), (gw - 1) & 1, err))
            return;
        __syncwarp();
        tc_fence_after();
        const bool whole = s.ke - s.kb == s.s.tiles;
        const bool in = s.q0 + rr < s.s.q_len;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        float *part = c.a.parts + (2ll * cta + (s.kb == 0)) * cross_slot_floats(kCrossBlockRows, D);
        uint16_t *out = static_cast<uint16_t *>(c.a.out) +
                        (static_cast<long long>(s.s.q_row) + s.q0 + rr) * c.a.out_row + s.head * D;
#pragma unroll
        for (int h = 0; h < D / 64; ++h) {
            float o[64];
            {
                uint32_t x[32], y[32];
                tmem_ld32(tO + 64 * h, x);
                tmem_ld32(tO + 64 * h + 32, y);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    o[i] = __uint_as_float(x[i]);
                    o[32 + i] = __uint_as_float(y[i]);
                }
            }
            if (h == D / 64 - 1) {
                tc_fence_before();
                mbar_arrive(bar(c, kBarOFree + w));   // the next segment may reset O
            }
            if (whole) {
                if (in) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        reinterpret_cast<uint4 *>(out)[8 * h + i] =
                            make_uint4(pack2<kHalf>(o[8 * i] * inv, o[8 * i + 1] * inv),
                                       pack2<kHalf>(o[8 * i + 2] * inv, o[8 * i + 3] * inv),
                                       pack2<kHalf>(o[8 * i + 4] * inv, o[8 * i + 5] * inv),
                                       pack2<kHalf>(o[8 * i + 6] * inv, o[8 * i + 7] * inv));
                }
            } else {
                // [D/4][256 rows] float4: neighbouring rows side by side
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    reinterpret_cast<float4 *>(part)[(16 * h + i) * kCrossBlockRows + rr] =
                        make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
            }
        }
        if (!whole)
            reinterpret_cast<float2 *>(part + kCrossBlockRows * D)[rr] = make_float2(m, l);
        if (!whole && s.kb == 0 && rr == 0) {
            CrossRecord rec;
            rec.row0 = static_cast<long long>(s.s.q_row) + s.q0;
            rec.rows = min(kCrossBlockRows, s.s.q_len - s.q0);
            rec.head0 = s.head;
            rec.group = 1;
            rec.parts = c.split.parts(s);
            c.a.records[cta] = rec;
        }
    }
}

template <int D, bool kHalf>
__global__ void __launch_bounds__(kThreads, 1)
attn_cross_kernel(const __grid_constant__ CrossArgs a)
{
    using L = Layout<D>;
    pdl_wait();
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *sbase = smem_raw + (base - raw);
    uint32_t *slot = reinterpret_cast<uint32_t *>(sbase + L::kOffBar + kSlotInBars);
    const int cta = blockIdx.x;

    if (threadIdx.x == 0)
        a.records[cta].parts = 0;
    Split split(a, a.heads);
    // at least 6 cost units (2 tiles of one unit) per CTA
    const bool work = split.find(*reinterpret_cast<Split::Scratch *>(sbase + L::kOffScratch), gridDim.x, 6);
    if (work) {
        Ctx c{base, 0u, sbase, a, split, base + L::kOffBar};
        const int warp = threadIdx.x >> 5;
        const int lane = threadIdx.x & 31;
        if (threadIdx.x == 0) {
            tma_prefetch_desc(&a.tm_q);
            tma_prefetch_desc(&a.tm_k);
            tma_prefetch_desc(&a.tm_v);
            for (int q = 0; q < L::kQSets; ++q) {
                mbar_init(bar(c, kBarQFull + q), 1);
                mbar_init(bar(c, kBarQEmpty + q), 2);   // one commit per issuer
            }
            for (int st = 0; st < L::kStages; ++st) {
                mbar_init(bar(c, kBarKFull + st), 1);
                mbar_init(bar(c, kBarKEmpty + st), 2);
                mbar_init(bar(c, kBarVFull + st), 1);
                mbar_init(bar(c, kBarVEmpty + st), 3);  // and the mask warp
            }
            for (int w = 0; w < 2; ++w) {
                mbar_init(bar(c, kBarSFull + w), 1);
                mbar_init(bar(c, kBarSEmpty + w), kBlockM);
                mbar_init(bar(c, kBarPFull + w), kBlockM);
                mbar_init(bar(c, kBarODone + w), 1);
                mbar_init(bar(c, kBarOFree + w), kBlockM);
            }
            for (int i = 0; i < kMaskSlots; ++i) {
                mbar_init(bar(c, kBarBitsFull + i), 1);
                mbar_init(bar(c, kBarBitsEmpty + i), 2 * kBlockM);
                mbar_init(bar(c, kBarVClean + i), 1);
            }
            fence_mbar_init();
        }
        if (warp == 0) {
            tmem_alloc(smem_u32(slot), kTmemCols);
            tmem_relinquish();
        }
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        c.tmem = *slot;

        if (warp >= 8) {
            asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(kRegsControl));
            if (warp == 8) {
                if (lane == 0)
                    producer<D>(c);
            } else if (warp == 9 || warp == 10) {
                mma_issuer<D, kHalf>(c, warp - 9, lane);
            } else {
                mask_stager<D>(c, lane);
            }
            __syncwarp();
        } else {
            asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(kRegsSoftmax));
            softmax_group<D, kHalf>(c, warp >> 2, warp & 3, lane, cta);
            __syncwarp();
        }

        tc_fence_before();
        __syncthreads();
        if (warp == 0) {
            tc_fence_after();
            tmem_dealloc(c.tmem, kTmemCols);
        }
    }
    pdl_trigger();
}

template <int D, bool kHalf>
cudaError_t launch(const CrossArgs &a, int ctas, cudaStream_t stream)
{
    static PerDeviceOnce smem_once;
    cudaError_t e = smem_opt_in(smem_once, attn_cross_kernel<D, kHalf>, Layout<D>::kSmemBytes);
    if (e != cudaSuccess)
        return e;
    return launch_chained(attn_cross_kernel<D, kHalf>, dim3(ctas), dim3(kThreads), Layout<D>::kSmemBytes, stream, a);
}

}  // namespace

cudaError_t launch_cross_blocks(const CrossArgs &a, int dim, bool half, int ctas, cudaStream_t stream)
{
    if (dim == 64)
        return half ? launch<64, true>(a, ctas, stream) : launch<64, false>(a, ctas, stream);
    return half ? launch<128, true>(a, ctas, stream) : launch<128, false>(a, ctas, stream);
}

}  // namespace mbert
