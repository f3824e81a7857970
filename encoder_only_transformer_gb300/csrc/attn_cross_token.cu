// Attention of a few query rows (new tokens) of each sequence over long keys
// and values of another length: at most 16 rows per (sequence, key head), the
// query rows times the query heads that share the key head.
//
// What bounds it: K and V are read once, 4 D bytes a key and head for
// 4 D x rows flops, so memory.  A tensor-core tile of 128 rows would be empty
// but for the 16; mma.sync's 16 x 8 tiles fit the rows, and their rate is far
// above what the loads allow.  So everything serves the loads: a TMA warp
// keeps a ring of 64-key tiles of K and V full across the borders of units,
// three (D = 64) or two (D = 128) CTAs an SM (130 KB in flight), and the units
// (sequence, key head) are split by cost over all CTAs (cross_sched.cuh), long
// ones into many parts, which a second kernel joins.  32 sequences of 128 to
// 8192 keys, 12 heads of 64 in rows of 24: 88 us and 3 us of joining for
// 488 MB, 5.4 TB/s (82 in all on another board); the same keys with each head's rows together, 6.2 TB/s, so
// what is left is DRAM's price for 128 bytes out of each row of 24 heads.  (Four heads to a
// CTA, 512 bytes in one place, gave 3 to 8 % there and lost up to 45 % on few
// sequences, whose units then are cut into four times as many parts.)
//
// CTA: warps 0-3 take 16 keys of every tile each, with a softmax state of
// their own; at the end of a segment the four states are joined in shared
// memory.  Warp 4 is the producer: it finds the segments (64-bit divisions and
// global loads that would otherwise stand before each of them), hands them on
// through a ring with their query rows, and keeps the K and V ring full.
#include "common.cuh"
#include "cross_sched.cuh"
#include "internal.h"
#include "roles.cuh"

namespace mbert {
namespace {

constexpr int kWarps = 4;                 // that compute
constexpr int kThreads = 32 * (kWarps + 1);
constexpr int kTileKeys = 16 * kWarps;
constexpr int kRows = kCrossTokenRows;
constexpr uint32_t kBoxBytes = kTileKeys * 128;       // 64 keys x 64 columns

// A unit's fixed work (the query rows, joining four states, the output) costs
// about two tiles.
using Split = CrossSplit<kThreads, 0, kTileKeys, 1, 1, 2, kCrossTokenWholeKeys / kTileKeys>;

// A segment (a unit and a run of its key tiles) as the producer hands it on.
struct alignas(16) Rec {
    int q_row, q_len, k_row, k_len;
    int kb, ke, tiles;      // key tiles [kb, ke) of tiles; ke = 0: no more segments
    int head, seq;          // key head, sequence
    int parts;              // of a cut unit whose first part this is
    int k_full;             // keys before the first hidden one
    int pad;
};
static_assert(sizeof(Rec) == 48, "record");
constexpr int kRecs = 2;

template <int D>
struct Layout {
    static constexpr int kHalves = D / 64;
    static constexpr uint32_t kTile = kHalves * kBoxBytes;          // of K or of V
    static constexpr int kStages = D == 64 ? 3 : 2;
    static constexpr uint32_t kOffState = kStages * 2 * kTile;      // [4][16][D + 2] floats
    static constexpr int kStateRow = D + 4;                         // floats; rows 16 bytes aligned
    static constexpr uint32_t kOffQ = kOffState + 4u * kWarps * kRows * kStateRow;   // [kRecs][16][D] query rows
    static constexpr uint32_t kQBytes = kRows * D * 2;
    static constexpr uint32_t kOffBar = kOffQ + kRecs * kQBytes;
    static constexpr uint32_t kOffRecs = kOffBar + 128;
    static constexpr uint32_t kOffScratch = kOffRecs + 48 * kRecs;
    static constexpr uint32_t kSmemBytes = kOffScratch + sizeof(Split::Scratch) + 1024;
};

constexpr int kBarFull = 0;       // + stage: K and V of a tile
constexpr int kBarEmpty = 3;      // + stage: read by the four warps
constexpr int kBarStates = 6;     // the four states are in shared memory
constexpr int kBarJoined = 7;     // they have been read
constexpr int kBarRecFull = 8;    // + record slot: a segment and its query rows
constexpr int kBarRecEmpty = 10;  // + record slot: read by the four warps
constexpr int kNumBars = 12;
constexpr uint32_t kGaveUpInBars = 8 * kNumBars;    // a wait has given up

__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

// c (16 x 8, fp32) += a (16 x 16) b (16 x 8)
template <bool kHalf>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    if constexpr (kHalf)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
                     "{%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
                     "{%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// (m, l) of two states: weights of each for the joined reference.  A state
// without a visible key has m = -inf and weighs nothing (unless its sum is
// NaN, which stays).
__device__ __forceinline__ float state_weight(float m, float l, float m_new)
{
    return m == -INFINITY ? (l == 0.f ? 0.f : 1.f) : ex2_approx(m - m_new);
}

struct Ctx {
    uint32_t base;
    uint8_t *sbase;
    const CrossArgs &a;
    uint32_t bars;
};

__device__ __forceinline__ uint32_t bar(const Ctx &c, int i) { return c.bars + 8u * i; }

// Waits for a phase of barrier i.  The warps that compute go on where it gives
// up, and ask (stop) where that matters.
__device__ __forceinline__ bool wait(const Ctx &c, int i, uint32_t parity)
{
    return mbar_wait_mark(bar(c, i), parity, c.a.err, c.bars + kGaveUpInBars);
}
__device__ __forceinline__ bool stop(const Ctx &c) { return any_gave_up(c.bars + kGaveUpInBars); }

// 16-byte aligned bulk copy of `bytes` (a multiple of 16) into shared memory.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t mbar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 :: "r"(dst), "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(mbar) : "memory");
}

// What the producer has issued so far.
struct Issued {
    uint32_t recs = 0, kv = 0;  // records (with their queries, but for the last), key tiles
};

template <int D>
__device__ void produce(const Ctx &c, const Split &split, Issued &n)
{
    using L = Layout<D>;
    const CrossArgs &a = c.a;
    auto it = split.begin();
    Split::Seg seg;
    for (uint32_t sg = 0;; ++sg) {
        Rec r{};
        const bool more = split.next(it, seg);
        if (more) {
            r.q_row = seg.s.q_row;
            r.q_len = seg.s.q_len;
            r.k_row = seg.s.k_row;
            r.k_len = seg.s.k_len;
            r.k_full = seg.s.k_full;
            r.kb = seg.kb;
            r.ke = seg.ke;
            r.tiles = seg.s.tiles;
            r.head = seg.head;
            r.seq = seg.seq;
            r.parts = seg.kb == 0 && seg.ke < seg.s.tiles ? split.parts(seg) : 0;
        }
        const int slot = sg % kRecs;
        if (sg >= kRecs && !wait(c, kBarRecEmpty + slot, (sg / kRecs - 1) & 1))
            return;
        reinterpret_cast<Rec *>(c.sbase + L::kOffRecs)[slot] = r;
        ++n.recs;
        if (!more) {
            mbar_arrive(bar(c, kBarRecFull + slot));
            return;
        }
        // row i: query i / group, head i % group of the key head's (a query's
        // heads lie side by side); rows behind the last keep what they held
        const uint32_t row = 2 * D * a.group;
        mbar_arrive_expect_tx(bar(c, kBarRecFull + slot), r.q_len * row);
        for (int i = 0; i < r.q_len; ++i)
            bulk_load(c.base + L::kOffQ + slot * L::kQBytes + i * row,
                      static_cast<const uint16_t *>(a.q) + (static_cast<long long>(r.q_row) + i) * a.q_row +
                          static_cast<long long>(r.head) * a.group * D,
                      row, bar(c, kBarRecFull + slot));
        const int col = r.head * D;
        for (int k = r.kb; k < r.ke; ++k, ++n.kv) {
            const int st = n.kv % L::kStages;
            const uint32_t u = n.kv / L::kStages;
            if (u > 0 && !wait(c, kBarEmpty + st, (u - 1) & 1))
                return;
            const uint32_t dst = c.base + st * 2 * L::kTile;
            mbar_arrive_expect_tx(bar(c, kBarFull + st), 2 * L::kTile);
            for (int h = 0; h < L::kHalves; ++h) {
                tma_load_2d(dst + h * kBoxBytes, &a.tm_k, col + 64 * h, r.k_row + k * kTileKeys,
                            bar(c, kBarFull + st));
                tma_load_2d(dst + L::kTile + h * kBoxBytes, &a.tm_v, col + 64 * h, r.k_row + k * kTileKeys,
                            bar(c, kBarFull + st));
            }
        }
    }
}

// Every copy has landed before the CTA can exit, wherever the producer stopped.
template <int D>
__device__ void producer(const Ctx &c, const Split &split)
{
    Issued n;
    produce<D>(c, split, n);
    ring_drain(bar(c, kBarRecFull), n.recs, kRecs);
    ring_drain(bar(c, kBarFull), n.kv, Layout<D>::kStages);
}

// The 16 keys of this warp in tile k that are visible, as bits.
__device__ __forceinline__ uint32_t warp_keys(const Ctx &c, const Rec &s, int k, int warp)
{
    const int j0 = k * kTileKeys + 16 * warp;
    const int left = s.k_len - j0;
    uint32_t b = left >= 16 ? 0xffffu : left > 0 ? (1u << left) - 1u : 0u;
    if (b && j0 + 16 > s.k_full && s.k_full < s.k_len)
        b &= __ldg(c.a.key_bits + key_bit_word(s.k_row, s.seq) + j0 / 32) >> (j0 & 31);
    return b;
}

template <int D, bool kHalf>
__device__ void compute(const Ctx &c, int warp, int lane, int cta)
{
    using L = Layout<D>;
    constexpr int kSteps = D / 16;
    constexpr float kLift = kHalf ? 7.f : 0.f;      // fp16: weights times 2^7, at most 2^15
    const CrossArgs &a = c.a;
    const int gr = lane >> 2, cq = lane & 3;        // rows gr, gr + 8; columns 2 cq, 2 cq + 1
    const int group = a.group;
    const float scale = a.scale_log2;
    float *states = reinterpret_cast<float *>(c.sbase + L::kOffState);
    uint32_t g = 0;
    for (uint32_t sg = 0;; ++sg) {
        const int slot = sg % kRecs;
        wait(c, kBarRecFull + slot, (sg / kRecs) & 1);
        if (stop(c))
            return;
        const Rec s = reinterpret_cast<const Rec *>(c.sbase + L::kOffRecs)[slot];
        if (s.ke == 0)
            return;
        const int rows = s.q_len * group;           // <= 16 (checked: q_len <= max_q)
        // query rows as A fragments: lane i addresses row i % 16 and the
        // 16-byte chunk 2 step + i / 16
        uint32_t qf[kSteps][4];
        {
            const uint32_t addr = c.base + L::kOffQ + slot * L::kQBytes + (lane & 15) * 2 * D + (lane >> 4) * 16;
#pragma unroll
            for (int k = 0; k < kSteps; ++k)
                ldmatrix_x4(addr + 32 * k, qf[k]);
        }
        __syncwarp();
        if (lane == 0)
            mbar_arrive(bar(c, kBarRecEmpty + slot));
        float o[D / 8][4];
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                o[i][j] = 0.f;
        float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;   // rows gr, gr + 8
        uint32_t keys = warp_keys(c, s, s.kb, warp);
        for (int k = s.kb; k < s.ke; ++k, ++g) {
            const uint32_t now = keys;
            if (k + 1 < s.ke)
                keys = warp_keys(c, s, k + 1, warp);      // a tile ahead
            const int st = g % L::kStages;
            wait(c, kBarFull + st, (g / L::kStages) & 1);
            __syncwarp();
            const uint32_t kt = c.base + st * 2 * L::kTile, vt = kt + L::kTile;
            if (now) {
                // S (16 rows x 16 keys): lane i addresses key (i/16) 8 + i%8 and
                // the 16-byte chunk 2 step + (i/8 & 1); chunk j of row r lies at
                // j ^ (r & 7) (128-byte swizzle)
                float sc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
                {
                    const int row = 16 * warp + (lane >> 4) * 8 + (lane & 7);
                    const uint32_t addr = kt + row * 128;
#pragma unroll
                    for (int q = 0; q < kSteps; ++q) {
                        const int chunk = (2 * q) % 8 + ((lane >> 3) & 1);
                        uint32_t b[4];
                        ldmatrix_x4(addr + (q / 4) * kBoxBytes + ((chunk ^ (row & 7)) << 4), b);
                        mma16816<kHalf>(sc[0], qf[q], b[0], b[1]);
                        mma16816<kHalf>(sc[1], qf[q], b[2], b[3]);
                    }
                }
                // this lane's keys: 2 cq, 2 cq + 1, and those + 8
                uint32_t vm0 = 0xffffffffu, vm1 = 0xffffffffu;
                if (now != 0xffffu) {
                    const uint32_t kb = now >> (2 * cq);
                    vm0 = ((kb & 1u) ? 0x0000ffffu : 0u) | ((kb & 2u) ? 0xffff0000u : 0u);
                    vm1 = ((kb & 0x100u) ? 0x0000ffffu : 0u) | ((kb & 0x200u) ? 0xffff0000u : 0u);
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (!(kb >> (8 * n + (j & 1)) & 1u))
                                sc[n][j] = -INFINITY;
                }
                float x0 = fmaxf(fmaxf(sc[0][0], sc[0][1]), fmaxf(sc[1][0], sc[1][1]));
                float x1 = fmaxf(fmaxf(sc[0][2], sc[0][3]), fmaxf(sc[1][2], sc[1][3]));
                x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 1));
                x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 1));
                x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 2)) * scale;
                x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 2)) * scale;
                // the reference moves when a maximum passes it by 8 (weights up to 2^8)
                const bool n0 = x0 > m0 + 8.f, n1 = x1 > m1 + 8.f;
                if (__any_sync(0xffffffffu, n0 || n1)) {
                    const float a0 = n0 ? ex2_approx(m0 - x0) : 1.f, a1 = n1 ? ex2_approx(m1 - x1) : 1.f;
                    m0 = n0 ? x0 : m0;
                    m1 = n1 ? x1 : m1;
                    l0 *= a0;
                    l1 *= a1;
#pragma unroll
                    for (int i = 0; i < D / 8; ++i) {
                        o[i][0] *= a0;
                        o[i][1] *= a0;
                        o[i][2] *= a1;
                        o[i][3] *= a1;
                    }
                }
                const float neg0 = m0 == -INFINITY ? 0.f : kLift - m0;
                const float neg1 = m1 == -INFINITY ? 0.f : kLift - m1;
                float p[2][4];
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    p[n][0] = ex2_approx(fmaf(sc[n][0], scale, neg0));
                    p[n][1] = ex2_approx(fmaf(sc[n][1], scale, neg0));
                    p[n][2] = ex2_approx(fmaf(sc[n][2], scale, neg1));
                    p[n][3] = ex2_approx(fmaf(sc[n][3], scale, neg1));
                }
                l0 += (p[0][0] + p[0][1]) + (p[1][0] + p[1][1]);
                l1 += (p[0][2] + p[0][3]) + (p[1][2] + p[1][3]);
                const uint32_t pf[4] = {pack2<kHalf>(p[0][0], p[0][1]), pack2<kHalf>(p[0][2], p[0][3]),
                                        pack2<kHalf>(p[1][0], p[1][1]), pack2<kHalf>(p[1][2], p[1][3])};
                // O += P V: lane i addresses key (i/8 & 1) 8 + i%8, chunk i/16
                {
                    const int row = 16 * warp + ((lane >> 3) & 1) * 8 + (lane & 7);
                    const uint32_t addr = vt + row * 128;
#pragma unroll
                    for (int n = 0; n < D / 16; ++n) {
                        const int chunk = (2 * n) % 8 + (lane >> 4);
                        uint32_t b[4];
                        ldmatrix_x4_trans(addr + (n / 4) * kBoxBytes + ((chunk ^ (row & 7)) << 4), b);
                        // unseen keys may hold anything: 0 times it must be 0
                        mma16816<kHalf>(o[2 * n], pf, b[0] & vm0, b[1] & vm1);
                        mma16816<kHalf>(o[2 * n + 1], pf, b[2] & vm0, b[3] & vm1);
                    }
                }
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(bar(c, kBarEmpty + st));
        }
        // ---- the segment's end: sums over the lanes of a row, then the four
        // warps' states through shared memory
        l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
        l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
        l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
        l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
        if (sg > 0)
            wait(c, kBarJoined, (sg - 1) & 1);
        __syncwarp();
        float *mine = states + warp * kRows * L::kStateRow;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = gr + 8 * h;
            if (r < rows) {
#pragma unroll
                for (int i = 0; i < D / 8; ++i)
                    *reinterpret_cast<float2 *>(mine + r * L::kStateRow + 8 * i + 2 * cq) =
                        make_float2(o[i][2 * h], o[i][2 * h + 1]);
                if (cq == 0)
                    *reinterpret_cast<float2 *>(mine + r * L::kStateRow + D) = h ? make_float2(m1, l1) : make_float2(m0, l0);
            }
        }
        __syncwarp();
        if (lane == 0)
            mbar_arrive(bar(c, kBarStates));
        wait(c, kBarStates, sg & 1);
        if (stop(c))
            return;
        const bool whole = s.ke - s.kb == s.tiles;
        float *part = a.parts + (2ll * cta + (s.kb == 0)) * cross_slot_floats(kRows, D);
        // eight numbers of a row per thread
        for (int i = 32 * warp + lane; i < rows * (D / 8); i += 32 * kWarps) {
            const int r = i / (D / 8), chunk = i % (D / 8);
            float m = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w)
                m = fmaxf(m, states[(w * kRows + r) * L::kStateRow + D]);
            float l = 0.f, x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                x[j] = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float *src = states + (w * kRows + r) * L::kStateRow;
                const float wt = state_weight(src[D], src[D + 1], m);
                l += src[D + 1] * wt;
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    x[j] += src[8 * chunk + j] * wt;
            }
            if (whole) {
                const float inv = l == 0.f ? 0.f : 1.f / l;
                uint16_t *dst = static_cast<uint16_t *>(a.out) +
                                (static_cast<long long>(s.q_row) + r / group) * a.out_row +
                                static_cast<long long>(s.head * group + r % group) * D + 8 * chunk;
                *reinterpret_cast<uint4 *>(dst) =
                    make_uint4(pack2<kHalf>(x[0] * inv, x[1] * inv), pack2<kHalf>(x[2] * inv, x[3] * inv),
                               pack2<kHalf>(x[4] * inv, x[5] * inv), pack2<kHalf>(x[6] * inv, x[7] * inv));
            } else {
                float4 *dst = reinterpret_cast<float4 *>(part);
                dst[(2 * chunk) * kRows + r] = make_float4(x[0], x[1], x[2], x[3]);
                dst[(2 * chunk + 1) * kRows + r] = make_float4(x[4], x[5], x[6], x[7]);
                if (chunk == 0)
                    reinterpret_cast<float2 *>(part + kRows * D)[r] = make_float2(m, l);
            }
        }
        __syncwarp();
        if (lane == 0)
            mbar_arrive(bar(c, kBarJoined));
        if (!whole && s.kb == 0 && warp == 0 && lane == 0) {
            CrossRecord rec;
            rec.row0 = s.q_row;
            rec.rows = rows;
            rec.head0 = s.head * group;
            rec.group = group;
            rec.parts = s.parts;
            a.records[cta] = rec;
        }
    }
}

template <int D, bool kHalf>
__global__ void __launch_bounds__(kThreads, cross_token_ctas(D))
attn_cross_token_kernel(const __grid_constant__ CrossArgs a)
{
    using L = Layout<D>;
    pdl_wait();
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *sbase = smem_raw + (base - raw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0 && a.records)
        a.records[blockIdx.x].parts = 0;
    Split split(a, a.heads / a.group);
    const bool work = split.find(*reinterpret_cast<Split::Scratch *>(sbase + L::kOffScratch), gridDim.x, 4);
    if (work) {
        const Ctx c{base, sbase, a, base + L::kOffBar};
        if (threadIdx.x == 0) {
            for (int st = 0; st < L::kStages; ++st) {
                mbar_init(bar(c, kBarFull + st), 1);
                mbar_init(bar(c, kBarEmpty + st), kWarps);
            }
            for (int i = 0; i < kRecs; ++i) {
                mbar_init(bar(c, kBarRecFull + i), 1);
                mbar_init(bar(c, kBarRecEmpty + i), kWarps);
            }
            mbar_init(bar(c, kBarStates), kWarps);
            mbar_init(bar(c, kBarJoined), kWarps);
            sts32(c.bars + kGaveUpInBars, 0u);
            fence_mbar_init();
        }
        __syncthreads();
        if (warp == kWarps) {
            if (lane == 0)
                producer<D>(c, split);
        } else {
            compute<D, kHalf>(c, warp, lane, blockIdx.x);
        }
        __syncwarp();
        __syncthreads();
    }
    pdl_trigger();
}

template <int D, bool kHalf>
cudaError_t launch(const CrossArgs &a, int ctas, cudaStream_t stream)
{
    static PerDeviceOnce smem_once;
    cudaError_t e = smem_opt_in(smem_once, attn_cross_token_kernel<D, kHalf>, Layout<D>::kSmemBytes);
    if (e != cudaSuccess)
        return e;
    return launch_chained(attn_cross_token_kernel<D, kHalf>, dim3(ctas), dim3(kThreads), Layout<D>::kSmemBytes,
                          stream, a);
}

}  // namespace

cudaError_t launch_cross_token(const CrossArgs &a, int dim, bool half, int ctas, cudaStream_t stream)
{
    if (dim == 64)
        return half ? launch<64, true>(a, ctas, stream) : launch<64, false>(a, ctas, stream);
    return half ? launch<128, true>(a, ctas, stream) : launch<128, false>(a, ctas, stream);
}

}  // namespace mbert
