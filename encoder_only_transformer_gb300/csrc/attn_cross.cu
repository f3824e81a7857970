// Attention of packed queries over keys and values of another length, for
// blocks of queries: a persistent, warp-specialised tcgen05 pipeline.
//
//   out_i = sum_j softmax_j(scale q_i . k_j) v_j,  j over the visible keys of
//   i's sequence; 0 where there is none
//
// Work: a unit is 256 query rows of one sequence and head (two tiles of 128;
// G = 2 below) or, in calls whose sequences have no more than 128 rows, one such
// tile (G = 1, with two CTAs an SM: a unit's start and end then lie beside the
// other one's tiles, and no softmax warps stand idle; packed calls with their
// bound given: 64 sequences of 30 queries over 600 keys each, 12 heads of 64, 45.7 ->
// 36.1 us, 100 of 20 over 250 44.4 -> 33.5; 24 of 32 over 1000, 32 heads over 8 of 128,
// 33.8 -> 30.7; but for 256 rows and more, D = 64, 200 us against 195 and 35 against
// 33, as K and V are fetched twice as often); units
// and their tiles of 128 keys (D = 128, G = 1: 64) are split among the CTAs by cost
// (cross_sched.cuh), and units cut between CTAs are joined by a second kernel
// (cross_join.cu) in a fixed order.  Query heads that share a key head share
// the blocks too: with F the largest power of two that divides their number,
// row r of a unit is query r / F, head r % F (a 3-D tensor map fetches them
// so), which leaves fewer rows empty at a sequence's end (ragged prompts of 16
// heads over 4: 179 -> 170 us) and makes few rows of many heads one unit
// instead of F.
//
// CTA (12 warps for D = 64, 16 for D = 128; for G = 1 the four of group 0, then
// those of warps 8 to 11):
//   warps 0-3    softmax group 0 (query tile 0, TMEM lanes 0..127, a thread a row)
//   warps 4-7    softmax group 1 (query tile 1)
//   warp  8      TMA producer: Q, K and V rings
//   warp  9      masks: the key bits of a tile to shared memory, and zeros over
//                the V rows that nothing may see (a weight of 0 times an
//                infinity there would be NaN)
//   warps 10,11  MMA issuers, one per query tile
//   warps 12,13  (D = 128) issuers of O += P V, one per query tile, with S = Q K^T
//                left to warps 10 and 11
// An issuer's waits and commits take 100 to 150 clocks each, completed or not.
// For D = 128, with its steps of 64 keys, they came to the whole period of the
// loop; with an issuer for each product a tile of both query tiles went from
// 3600 clocks to 2900 (the tensor cores need 2560: S of 64 keys costs them 48
// clocks per 16 of D instead of 32 for half of 128).  For D = 64, where the
// softmax bounds the loop, the larger block only takes registers from it:
// 217 us against 194 (8192 queries and keys, 12 heads).
//
// TMEM (512 columns; half for G = 1), fp32 except P (16-bit pairs):
//   D = 64:   S0 S1 (128 each), P0 P1 (64 each), O0 O1 (64 each); S of the next
//             tile is computed while the softmax works on this one
//   D = 128:  two S of 64 keys (64 each) per query tile, O0 O1 (128 each); P
//             takes the first half of its own S, and S of the next 64 keys is
//             computed into the other one meanwhile
//
// What bounds it.  D = 64: the softmax; a query tile alone takes 1750 clocks a
// key tile (TMEM load 290, maximum 280, exponentials 710, the rest hand-offs),
// two together 2100 to 2200, the tensor cores' products 1024.  8192 x 8192, 12
// heads bf16: 191 us and 5 us of joining, 1049 TFLOP/s, 0.54 of the measured
// peak.  (The compiler's layout of the loop counts: the same loop beside more or
// less code that runs once took 193 to 203 us.)  Steps of 64 keys with three S buffers, which overlap more, took 231
// us: their loads, stores and waits come twice as often.  D = 128: the tensor
// cores and the hand-offs; ragged prompts of 16 heads over 4 (fp16): 160 us and
// 10 us of joining (178 in all on another board) for 214 GFLOP, 1260 TFLOP/s, 0.65 of
// the peak.
//
// Spills: D = 64, G = 2 reloads 16 bytes, D = 128, G = 2 148 (16 warps leave 128
// registers a thread before the split), G = 1 8 bytes.
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
#include "roles.cuh"

namespace mbert {
namespace {

constexpr int kMaskSlots = 4;

// Costs, by a fit over the CTAs' times in clocks: a key tile for both query
// tiles 2200 (D = 64) and 2900 (D = 128), for one 1750 and 1850 (G = 1: beside
// another CTA's 2150, and 1450 for 64 keys of D = 128); a unit's fixed
// work (the end of the softmax, the output, the refill) 3500 and 4700.  Units
// stay whole, up to four to a CTA, where that puts no more than 30 (6 us; 72, 9
// us, for G = 1 of D = 128, where joining the parts of 304 CTAs takes longer: 24
// sequences of 32 over 1000, 43 above the share, 30 us, 36 cut) on top of a CTA's
// share.
template <int D, int G>
using Split = CrossSplit<G == 1 ? 256 : D == 64 ? 384 : 512, kBlockM * G, cross_tile_keys(D, kBlockM * G), 6,
                         G == 1 ? 6 : D == 64 ? 5 : 4, D == 128 && G == 1 ? 20 : 10,
                         kCrossBlockWholeKeys / cross_tile_keys(D, kBlockM * G), 4, D == 128 && G == 1 ? 72 : 30,
                         cross_block_ctas(kBlockM * G)>;

// G: query tiles of a unit, a softmax group for each.
template <int D, int G>
struct Layout {
    static constexpr bool kSplitIssuers = D == 128;     // S and P V issued by different warps
    static constexpr bool kPair = D == 64 && G == 2;    // the one of 12 warps
    static constexpr int kUnitRows = kBlockM * G;
    static constexpr int kCtas = cross_block_ctas(kUnitRows);
    static constexpr int kControl = 4 * G;              // first warp after the softmax groups
    static constexpr int kThreads = 32 * (kControl + (kSplitIssuers && G == 2 ? 8 : 4));
    // registers a thread: 4 x 72 + 8 x 216 = 12 x 168, 8 x 56 + 8 x 200 = 16 x 128,
    // 4 x 56 + 4 x 200 = 8 x 128
    static constexpr int kRegsSoftmax = kPair ? 216 : 200;
    static constexpr int kRegsControl = kPair ? 72 : 56;
    static constexpr int kRecReaders = (kSplitIssuers ? 6 : 5) * G + 1;   // issuers, softmax warps, the mask warp
    static constexpr int kKeys = D == 64 ? 128 : 64;    // keys of a step (an S)
    static constexpr int kTileKeys = cross_tile_keys(D, kUnitRows);
    static constexpr int kSteps = kTileKeys / kKeys;    // steps of a tile
    static constexpr int kHalves = D / 64;              // 64-column boxes of a tile
    static constexpr uint32_t kQTile = kHalves * kTileBytes;
    static constexpr uint32_t kBox = kTileKeys * 128;   // of K or V: 64 columns
    static constexpr uint32_t kTile = kHalves * kBox;
    static constexpr int kQSets = D == 64 ? 2 : 1;      // of G query tiles
    static constexpr int kStages = kPair ? 3 : 2;     // of K and of V
    static constexpr uint32_t kOffK = kQSets * G * kQTile;
    static constexpr uint32_t kOffV = kOffK + kStages * kTile;
    static constexpr uint32_t kOffOut = kOffV + kStages * kTile;    // 4 KB per softmax warp: 32 rows x 64 columns
    static constexpr uint32_t kOutRows = kCtas == 2 ? 16 : 32;   // rows that a warp stages at a time
    static constexpr uint32_t kOffBar = kOffOut + 4 * G * kOutRows * 128;
    static constexpr uint32_t kOffWords = kOffBar + 512;            // key bits, kMaskSlots x 4 words
    static constexpr uint32_t kOffRecs = kOffWords + 16 * kMaskSlots;
    static constexpr uint32_t kOffScratch = kOffRecs + 48 * 4;
    static constexpr uint32_t kSmemBytes = kOffScratch + sizeof(typename Split<D, G>::Scratch) + 1024;
    // S and P of query tile w's step (D = 128: two buffers in turn), O
    static constexpr uint32_t col_s(int w, uint32_t step) { return 128u * w + (D == 64 ? 0u : 64u * (step & 1)); }
    static constexpr uint32_t col_p(int w, uint32_t step) { return D == 64 ? 128u * G + 64u * w : col_s(w, step); }
    static constexpr uint32_t col_o(int w) { return D == 64 ? 192u * G + 64u * w : 128u * G + 128u * w; }
    static constexpr uint32_t kTmemCols = 256 * G;
};
// (1 KB of an SM's 228 is the system's for each CTA)
static_assert(Layout<64, 2>::kSmemBytes <= 232448 && Layout<128, 2>::kSmemBytes <= 232448 &&
                  Layout<64, 1>::kSmemBytes <= 115712 && Layout<128, 1>::kSmemBytes <= 115712,
              "shared memory");

// barrier slots (8 bytes each)
constexpr int kBarQFull = 0;      // + set (2)
constexpr int kBarQEmpty = 2;     // + set
constexpr int kBarKFull = 4;      // + stage (3)
constexpr int kBarKEmpty = 7;
constexpr int kBarVFull = 10;
constexpr int kBarVEmpty = 13;
constexpr int kBarSFull = 16;     // + group (2)
constexpr int kBarSEmpty = 18;    // + group: S has been read (D = 64)
constexpr int kBarSOdd = 18;      // + group: kBarSFull of the odd steps (D = 128)
constexpr int kBarPFull = 20;
constexpr int kBarODone = 22;
constexpr int kBarOFree = 24;
constexpr int kBarBitsFull = 26;  // + mask slot (4): a tile's key bits are in shared memory
constexpr int kBarBitsEmpty = 30; // + mask slot: read by every softmax thread
constexpr int kBarVClean = 34;    // + mask slot: a tile's unseen V rows are zeros
constexpr int kBarRecFull = 38;   // + record slot (4)
constexpr int kBarRecEmpty = 42;  // + record slot
constexpr int kBarPOdd = 46;      // + group: kBarPFull of the odd steps (D = 128)
constexpr int kBarOOdd = 48;      // + group: kBarODone of the odd steps (D = 128)
constexpr int kBarDrain = 50;     // + issuer (4): all of its products are done
constexpr int kNumBars = 54;
constexpr uint32_t kSlotInBars = 8 * kNumBars;                 // TMEM address
constexpr uint32_t kGaveUpInBars = kSlotInBars + 4;            // a wait has given up
static_assert(kGaveUpInBars + 4 <= 512, "barriers");

constexpr float kRescaleThreshold = 8.0f;

// kind::f16 instruction descriptor for either 16-bit type (A and B alike)
__device__ __forceinline__ constexpr uint32_t idesc(int M, int N, bool b_mn_major, bool half)
{
    const uint32_t d = make_idesc_bf16(M, N, b_mn_major);
    return half ? d & ~((7u << 7) | (7u << 10)) : d;
}

// A segment (a unit and a run of its key tiles) as the producer hands it to
// the other warps, through a ring in shared memory: finding it takes global
// loads and 64-bit divisions, 3500 clocks that stood between the segments when
// every warp did it for itself.
struct alignas(16) Rec {
    int q_row, rows, q0, k_row, k_len;  // first query, rows (queries times F), the unit's first row
    int kb, ke, tiles;      // key tiles [kb, ke) of tiles; ke = 0: no more segments
    int head, seq;          // first query head of the unit, sequence
    int parts;              // of a cut unit whose first part this is
    int k_full;             // keys before the first hidden one
};
constexpr int kRecs = 4;

struct Ctx {
    uint32_t base;          // 1024-aligned shared address
    uint32_t tmem;
    uint8_t *sbase;         // generic pointer to the same address
    const CrossArgs &a;
    uint32_t bars;
};

__device__ __forceinline__ uint32_t bar(const Ctx &c, int i) { return c.bars + 8u * i; }

// Waits for a phase of barrier i.  A role of whole warps goes on where it gives
// up, and asks (stop) where that matters.
__device__ __forceinline__ bool wait(const Ctx &c, int i, uint32_t parity)
{
    return mbar_wait_mark(bar(c, i), parity, c.a.err, c.bars + kGaveUpInBars);
}
__device__ __forceinline__ bool stop(const Ctx &c) { return any_gave_up(c.bars + kGaveUpInBars); }

// The CTA's segment sg (all lanes of a reading warp).  False: there is none.
template <int D, int G>
__device__ __forceinline__ bool read_rec(const Ctx &c, uint32_t sg, int lane, Rec &r)
{
    const int slot = sg % kRecs;
    wait(c, kBarRecFull + slot, (sg / kRecs) & 1);
    if (stop(c))
        return false;
    r = reinterpret_cast<const Rec *>(c.sbase + Layout<D, G>::kOffRecs)[slot];
    __syncwarp();
    if (lane == 0)
        mbar_arrive(bar(c, kBarRecEmpty + slot));
    return r.ke > 0;
}

// A tile whose keys are not all known to be visible, and one of a sequence with
// hidden keys among the visible ones, which needs their bits.
template <int kTileKeys>
__device__ __forceinline__ bool needs_mask(const Rec &s, int k) { return s.k_full - k * kTileKeys < kTileKeys; }
__device__ __forceinline__ bool needs_bits(const Rec &s) { return s.k_full < s.k_len; }

// The unit's second query tile holds rows.
__device__ __forceinline__ bool second_tile(const Rec &s) { return s.rows - s.q0 > kBlockM; }

// Steps of a segment: a last tile of at most 64 keys takes one step of 64.
template <int D, int G>
__device__ __forceinline__ int seg_steps(const Rec &s)
{
    const int n = (s.ke - s.kb) * Layout<D, G>::kSteps;
    return n - (Layout<D, G>::kSteps == 2 && s.k_len - (s.ke - 1) * kBlockN <= 64);
}

// ---------------------------------------------------------------- producer
// What the producer has issued so far.
struct Issued {
    uint32_t q = 0, k = 0, v = 0;   // segments' queries, key tiles of K and of V
};

template <int D, int G>
__device__ void produce(const Ctx &c, const Split<D, G> &split, Issued &n)
{
    using L = Layout<D, G>;
    auto it = split.begin();
    typename Split<D, G>::Seg seg;
    for (uint32_t sg = 0;; ++sg) {
        Rec s{};
        if (split.next(it, seg)) {
            s.q_row = seg.s.q_row;
            s.rows = seg.s.rows;
            s.q0 = seg.q0;
            s.k_row = seg.s.k_row;
            s.k_len = seg.s.k_len;
            s.k_full = seg.s.k_full;
            s.kb = seg.kb;
            s.ke = seg.ke;
            s.tiles = seg.s.tiles;
            s.head = seg.head << c.a.fold_log2;
            s.seq = seg.seq;
            s.parts = seg.kb == 0 && seg.ke < seg.s.tiles ? split.parts(seg) : 0;
        }
        const int slot = sg % kRecs;
        if (sg >= kRecs && !wait(c, kBarRecEmpty + slot, (sg / kRecs - 1) & 1))
            return;
        reinterpret_cast<Rec *>(c.sbase + L::kOffRecs)[slot] = s;
        mbar_arrive(bar(c, kBarRecFull + slot));
        if (s.ke == 0)
            return;
        const int qs = sg % L::kQSets;
        const bool two = G == 2 && second_tile(s);
        if (sg >= L::kQSets && !wait(c, kBarQEmpty + qs, (sg / L::kQSets - 1) & 1))
            return;
        const int col_k = s.head / c.a.group * D;
        const int fold = c.a.fold_log2, qrow = s.q_row + (s.q0 >> fold);
        const uint32_t qdst = c.base + qs * G * L::kQTile;
        mbar_arrive_expect_tx(bar(c, kBarQFull + qs), (two ? 2 : 1) * L::kQTile);
        ++n.q;
        for (int w = 0; w < (two ? 2 : 1); ++w)
            for (int h = 0; h < L::kHalves; ++h)
                tma_load_3d(qdst + w * L::kQTile + h * kTileBytes, &c.a.tm_q, 64 * h, s.head,
                            qrow + w * (kBlockM >> fold), bar(c, kBarQFull + qs));
        for (int k = s.kb; k < s.ke; ++k) {
            const int st = n.k % L::kStages;
            const uint32_t u = n.k / L::kStages;
            const int krow = s.k_row + k * L::kTileKeys;
            if (u > 0 && !wait(c, kBarKEmpty + st, (u - 1) & 1))
                return;
            mbar_arrive_expect_tx(bar(c, kBarKFull + st), L::kTile);
            for (int h = 0; h < L::kHalves; ++h)
                tma_load_2d(c.base + L::kOffK + st * L::kTile + h * L::kBox, &c.a.tm_k, col_k + 64 * h, krow,
                            bar(c, kBarKFull + st));
            ++n.k;
            if (u > 0 && !wait(c, kBarVEmpty + st, (u - 1) & 1))
                return;
            mbar_arrive_expect_tx(bar(c, kBarVFull + st), L::kTile);
            for (int h = 0; h < L::kHalves; ++h)
                tma_load_2d(c.base + L::kOffV + st * L::kTile + h * L::kBox, &c.a.tm_v, col_k + 64 * h, krow,
                            bar(c, kBarVFull + st));
            ++n.v;
        }
    }
}

// Every copy has landed before the CTA can exit, wherever the producer stopped.
template <int D, int G>
__device__ void producer(const Ctx &c, const Split<D, G> &split)
{
    using L = Layout<D, G>;
    Issued n;
    produce<D, G>(c, split, n);
    ring_drain(bar(c, kBarQFull), n.q, L::kQSets);
    ring_drain(bar(c, kBarKFull), n.k, L::kStages);
    ring_drain(bar(c, kBarVFull), n.v, L::kStages);
}

// ---------------------------------------------------------------- MMA issuers
// S of 64 (D = 128) or 128 keys from key `key0` of the stage.
template <int D, int G, bool kHalf>
__device__ __forceinline__ void issue_s(const Ctx &c, int w, int qs, int st, int key0, uint32_t step)
{
    using L = Layout<D, G>;
    constexpr uint32_t kIdesc = idesc(128, L::kKeys, false, kHalf);
    const uint32_t q = c.base + (qs * G + w) * L::kQTile;
    const uint32_t k = c.base + L::kOffK + st * L::kTile + 128 * key0;
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t q_off = (kk / 4) * kTileBytes + 32 * (kk % 4), k_off = (kk / 4) * L::kBox + 32 * (kk % 4);
        mma_bf16_ss_warp(c.tmem + L::col_s(w, step), make_sdesc_sw128(q + q_off, 16, 1024),
                         make_sdesc_sw128(k + k_off, 16, 1024), kIdesc, kk > 0);
    }
}

// O += P V over the step's keys, all D columns per instruction.  V is the
// MN-major operand: 64 columns (128 bytes) x 8 keys are one swizzle atom; atoms
// follow each other by 1024 bytes along the keys (stride offset) and by a
// 64-column box along the columns (leading offset).
template <int D, int G, bool kHalf>
__device__ __forceinline__ void issue_o(const Ctx &c, int w, int st, int key0, uint32_t step, bool accumulate)
{
    using L = Layout<D, G>;
    constexpr uint32_t kIdesc = idesc(128, D, true, kHalf);
    const uint32_t v = c.base + L::kOffV + st * L::kTile + 128 * key0;
#pragma unroll
    for (int kk = 0; kk < L::kKeys / 16; ++kk)
        mma_bf16_ts_warp(c.tmem + L::col_o(w), c.tmem + L::col_p(w, step) + 8 * kk,
                         make_sdesc_sw128(v + 2048 * kk, L::kBox, 1024), kIdesc,
                         (accumulate || kk > 0) ? 1u : 0u);
}

// D = 64: the issuer of query tile w, S of a key tile and then P V of the one
// before, while the softmax works on the former's predecessor.  `gw` counts the
// steps of this query tile (its S, P and O barriers), `g` all tiles of the CTA
// (the rings).  In a segment whose second query tile is empty, issuer 1 only
// hands the ring slots back as they fill (each phase only once it has begun).
template <int G, bool kHalf>
__device__ void so_issuer(const Ctx &c, int w, int lane)
{
    constexpr int D = 64;
    using L = Layout<D, G>;
    Rec s;
    uint32_t g0 = 0, gw0 = 0, sw = 0, masked = 0;
    for (uint32_t sg = 0; read_rec<D, G>(c, sg, lane, s); ++sg) {
        const int qs = sg % L::kQSets;
        const int n = s.ke - s.kb;
        const bool mine = w == 0 || second_tile(s);
        wait(c, kBarQFull + qs, (sg / L::kQSets) & 1);
        for (int t = 0; t <= n; ++t) {
            if (t < n) {
                const uint32_t g = g0 + t, gw = gw0 + t;
                const int st = g % L::kStages;
                wait(c, kBarKFull + st, (g / L::kStages) & 1);
                if (mine) {
                    if (gw > 0)
                        wait(c, kBarSEmpty + w, (gw - 1) & 1);
                    __syncwarp();
                    tc_fence_after();
                    issue_s<D, G, kHalf>(c, w, qs, st, 0, gw);
                    mma_commit_warp(bar(c, kBarSFull + w));
                    mma_commit_warp(bar(c, kBarKEmpty + st));
                    if (t == n - 1)
                        mma_commit_warp(bar(c, kBarQEmpty + qs));
                } else if (lane == 0) {
                    mbar_arrive(bar(c, kBarKEmpty + st));
                    if (t == n - 1)
                        mbar_arrive(bar(c, kBarQEmpty + qs));
                }
                __syncwarp();
            }
            if (t > 0) {
                const uint32_t g = g0 + t - 1, gw = gw0 + t - 1;
                const int st = g % L::kStages;
                wait(c, kBarVFull + st, (g / L::kStages) & 1);
                if (needs_mask<L::kTileKeys>(s, s.kb + t - 1)) {
                    if (mine)
                        wait(c, kBarVClean + masked % kMaskSlots, (masked / kMaskSlots) & 1);
                    ++masked;
                }
                if (mine) {
                    wait(c, kBarPFull + w, gw & 1);
                    if (t == 1 && sw > 0)
                        wait(c, kBarOFree + w, (sw - 1) & 1);
                    __syncwarp();
                    tc_fence_after();
                    issue_o<D, G, kHalf>(c, w, st, 0, gw, t > 1);
                    mma_commit_warp(bar(c, kBarODone + w));
                    mma_commit_warp(bar(c, kBarVEmpty + st));
                } else if (lane == 0) {
                    mbar_arrive(bar(c, kBarVEmpty + st));
                }
                __syncwarp();
            }
        }
        g0 += n;
        if (mine) {
            gw0 += n;
            ++sw;
        }
    }
}

// D = 128: issuer of query tile w's S.
template <int D, int G, bool kHalf>
__device__ void s_issuer(const Ctx &c, int w, int lane)
{
    using L = Layout<D, G>;
    Rec s;
    uint32_t g = 0, gw = 0;
    for (uint32_t sg = 0; read_rec<D, G>(c, sg, lane, s); ++sg) {
        const int qs = sg % L::kQSets;
        const int n = seg_steps<D, G>(s);
        const bool mine = w == 0 || second_tile(s);
        wait(c, kBarQFull + qs, (sg / L::kQSets) & 1);
        for (int j = 0; j < n; ++j) {
            const int st = g % L::kStages, sub = j % L::kSteps;
            const bool last_sub = sub == L::kSteps - 1 || j == n - 1;
            if (sub == 0)
                wait(c, kBarKFull + st, (g / L::kStages) & 1);
            g += last_sub;
            if (!mine) {
                if (lane == 0 && last_sub)
                    mbar_arrive(bar(c, kBarKEmpty + st));
                __syncwarp();
                continue;
            }
            // this buffer's last P has been multiplied
            if (gw > 1)
                wait(c, (gw & 1 ? kBarOOdd : kBarODone) + w, ((gw >> 1) - 1) & 1);
            __syncwarp();
            tc_fence_after();
            issue_s<D, G, kHalf>(c, w, qs, st, sub * L::kKeys, gw);
            mma_commit_warp(bar(c, (gw & 1 ? kBarSOdd : kBarSFull) + w));
            if (last_sub)
                mma_commit_warp(bar(c, kBarKEmpty + st));
            if (j == n - 1)
                mma_commit_warp(bar(c, kBarQEmpty + qs));
            ++gw;
        }
        if (!mine) {
            if (lane == 0)
                mbar_arrive(bar(c, kBarQEmpty + qs));
            __syncwarp();
        }
    }
}

// D = 128: issuer of query tile w's O += P V.
template <int D, int G, bool kHalf>
__device__ void o_issuer(const Ctx &c, int w, int lane)
{
    using L = Layout<D, G>;
    Rec s;
    uint32_t g = 0, gw = 0, sw = 0, masked = 0;
    for (uint32_t sg = 0; read_rec<D, G>(c, sg, lane, s); ++sg) {
        const int n = seg_steps<D, G>(s);
        const bool mine = w == 0 || second_tile(s);
        for (int j = 0; j < n; ++j) {
            const int st = g % L::kStages, sub = j % L::kSteps;
            const bool last_sub = sub == L::kSteps - 1 || j == n - 1;
            if (sub == 0) {
                wait(c, kBarVFull + st, (g / L::kStages) & 1);
                if (needs_mask<L::kTileKeys>(s, s.kb + j / L::kSteps)) {
                    if (mine)
                        wait(c, kBarVClean + masked % kMaskSlots, (masked / kMaskSlots) & 1);
                    ++masked;
                }
            }
            g += last_sub;
            if (!mine) {
                if (lane == 0 && last_sub)
                    mbar_arrive(bar(c, kBarVEmpty + st));
                __syncwarp();
                continue;
            }
            // one barrier per P buffer: the softmax may finish two steps, whose S
            // are both there, before this wait
            wait(c, (gw & 1 ? kBarPOdd : kBarPFull) + w, gw >> 1 & 1);
            if (j == 0 && sw > 0)
                wait(c, kBarOFree + w, (sw - 1) & 1);
            __syncwarp();
            tc_fence_after();
            issue_o<D, G, kHalf>(c, w, st, sub * L::kKeys, gw, j > 0);
            mma_commit_warp(bar(c, (gw & 1 ? kBarOOdd : kBarODone) + w));
            if (last_sub)
                mma_commit_warp(bar(c, kBarVEmpty + st));
            ++gw;
        }
        sw += mine;
    }
}

// ---------------------------------------------------------------- masks
// The visible keys of tile k as words.
template <int kTileKeys>
__device__ __forceinline__ uint32_t tile_word(const Ctx &c, const Rec &s, int k, int i)
{
    const int left = s.k_len - k * kTileKeys - 32 * i;
    uint32_t w = left >= 32 ? 0xffffffffu : left > 0 ? (1u << left) - 1u : 0u;
    if (w && needs_bits(s))
        w &= __ldg(c.a.key_bits + key_bit_word(s.k_row, s.seq) + kTileKeys / 32 * k + i);
    return w;
}

template <int D, int G>
__device__ void mask_stager(const Ctx &c, int lane)
{
    using L = Layout<D, G>;
    constexpr int kWords = L::kTileKeys / 32;
    Rec s;
    uint32_t g = 0, masked = 0, with_bits = 0;
    for (uint32_t sg = 0; read_rec<D, G>(c, sg, lane, s); ++sg) {
        for (int k = s.kb; k < s.ke; ++k, ++g) {
            const int st = g % L::kStages;
            // every tile is waited for and handed back, seen or not, so that
            // this warp neither runs ahead of the ring nor falls behind it
            if (!needs_mask<L::kTileKeys>(s, k)) {
                wait(c, kBarVFull + st, (g / L::kStages) & 1);
                if (lane == 0)
                    mbar_arrive(bar(c, kBarVEmpty + st));
                __syncwarp();
                continue;
            }
            const uint32_t clean = masked % kMaskSlots;
            ++masked;
            const uint32_t mine = lane < kWords ? tile_word<L::kTileKeys>(c, s, k, lane) : 0u;
            if (needs_bits(s)) {
                const uint32_t slot = with_bits % kMaskSlots, u = with_bits / kMaskSlots;
                ++with_bits;
                if (u > 0)
                    wait(c, kBarBitsEmpty + slot, (u - 1) & 1);
                if (lane < kWords)
                    reinterpret_cast<uint32_t *>(c.sbase + L::kOffWords)[4 * slot + lane] = mine;
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(bar(c, kBarBitsFull + slot));
            }
            wait(c, kBarVFull + st, (g / L::kStages) & 1);
            __syncwarp();
#pragma unroll 1
            for (int i = 0; i < kWords; ++i) {
                const uint32_t word = __shfl_sync(0xffffffffu, mine, i);
                if (word == 0xffffffffu)
                    continue;
                // 16 bytes of each of 32 rows per step (rows' order does not
                // matter for zeros: a row is 128 contiguous bytes per half)
                uint8_t *v = c.sbase + L::kOffV + st * L::kTile + 32 * i * 128;
                for (int j = lane; j < 32 * 8 * L::kHalves; j += 32) {
                    const int row = j / 8 % 32, part = j % 8, half = j / 256;
                    if (!(word >> row & 1))
                        *reinterpret_cast<uint4 *>(v + half * L::kBox + row * 128 + part * 16) =
                            make_uint4(0u, 0u, 0u, 0u);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(bar(c, kBarVClean + clean));
                mbar_arrive(bar(c, kBarVEmpty + st));
            }
            __syncwarp();
        }
    }
}

// ---------------------------------------------------------------- softmax
// Two weights 2^(x scale - m): added to a packed row sum, packed to 16 bits.
template <bool kHalf>
__device__ __forceinline__ uint32_t weights(float x0, float x1, uint64_t sc2, uint64_t nm2, uint64_t &acc)
{
    uint32_t pk;
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
            : "=r"(pk), "+l"(acc)
            : "f"(x0), "f"(x1), "l"(sc2), "l"(nm2));
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
            : "=r"(pk), "+l"(acc)
            : "f"(x0), "f"(x1), "l"(sc2), "l"(nm2));
    return pk;
}

template <int D, int G, bool kHalf>
__device__ void softmax_group(const Ctx &c, int w, int warp_in_group, int lane, int cta)
{
    using L = Layout<D, G>;
    constexpr int kKeys = L::kKeys;
    constexpr float kLift = kHalf ? 7.f : 0.f;        // weights times 2^7 in fp16
    const uint32_t lane_off = static_cast<uint32_t>(32 * warp_in_group) << 16;
    const uint32_t tO = c.tmem + L::col_o(w) + lane_off;
    const int rr = kBlockM * w + 32 * warp_in_group + lane;      // row within the unit
    const float scale = c.a.scale_log2;
    // step's P V has completed.  (D = 128: S of a step stands for the P V two
    // steps before, that is for the last phase of the same barrier.)
    auto wait_o = [&](uint32_t step) {
        if constexpr (D == 64)
            wait(c, kBarODone + w, step & 1);
        else
            wait(c, step & 1 ? kBarOOdd + w : kBarODone + w, step >> 1 & 1);
        __syncwarp();
    };
    Rec s;
    uint32_t gw = 0, with_bits = 0;
    for (uint32_t sg = 0; read_rec<D, G>(c, sg, lane, s); ++sg) {
        const int n = seg_steps<D, G>(s);
        if (w == 1 && !second_tile(s)) {
            // nothing to do but hand the key bits on
            for (int k = s.kb; k < s.ke && needs_bits(s); ++k) {
                if (!needs_mask<L::kTileKeys>(s, k))
                    continue;
                const uint32_t slot = with_bits % kMaskSlots;
                wait(c, kBarBitsFull + slot, (with_bits / kMaskSlots) & 1);
                mbar_arrive(bar(c, kBarBitsEmpty + slot));
                ++with_bits;
            }
            continue;
        }
        float m = -INFINITY;    // reference (scaled, base 2)
        float l = 0.f;          // sum of exp2(score - m + kLift)
        uint32_t bits[4] = {0u, 0u, 0u, 0u};   // the tile's key bits
        for (int j = 0; j < n; ++j, ++gw) {
            const int sub = j % L::kSteps;
            if constexpr (D == 64)
                wait(c, kBarSFull + w, gw & 1);
            else
                wait(c, gw & 1 ? kBarSOdd + w : kBarSFull + w, gw >> 1 & 1);
            __syncwarp();
            tc_fence_after();
            float sc[kKeys];
            {
                const uint32_t tS = c.tmem + L::col_s(w, gw) + lane_off;
                uint32_t r[kKeys / 32][32];
#pragma unroll
                for (int q = 0; q < kKeys / 32; ++q)
                    tmem_ld32(tS + 32 * q, r[q]);
                tmem_wait_ld();
#pragma unroll
                for (int q = 0; q < kKeys / 32; ++q)
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        sc[32 * q + i] = __uint_as_float(r[q][i]);
            }
            tc_fence_before();
            if constexpr (D == 64)
                mbar_arrive(bar(c, kBarSEmpty + w));   // S may be overwritten now

            const int kt = s.kb + j / L::kSteps;
            if (needs_mask<L::kTileKeys>(s, kt)) {
                if (needs_bits(s)) {
                    if (sub == 0) {
                        const uint32_t slot = with_bits % kMaskSlots;
                        wait(c, kBarBitsFull + slot, (with_bits / kMaskSlots) & 1);
                        ++with_bits;
                        const uint4 b = reinterpret_cast<const uint4 *>(c.sbase + L::kOffWords)[slot];
                        bits[0] = b.x, bits[1] = b.y, bits[2] = b.z, bits[3] = b.w;
                        mbar_arrive(bar(c, kBarBitsEmpty + slot));
                    }
                    uint32_t all = 0xffffffffu;
                    uint32_t mine[kKeys / 32];
#pragma unroll
                    for (int q = 0; q < kKeys / 32; ++q) {
                        mine[q] = L::kSteps == 2 && sub ? bits[q + 2] : bits[q];
                        all &= mine[q];
                    }
                    if (all != 0xffffffffu) {
#pragma unroll
                        for (int q = 0; q < kKeys / 32; ++q)
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (!(mine[q] >> i & 1))
                                    sc[32 * q + i] = -INFINITY;
                    }
                } else {
                    const int kvalid = s.k_len - kt * L::kTileKeys - sub * kKeys;
                    if (kvalid < kKeys) {
#pragma unroll
                        for (int i = 0; i < kKeys; ++i)
                            if (i >= kvalid)
                                sc[i] = -INFINITY;
                    }
                }
            }
            // row maximum: 8 independent chains
            float mp[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
                mp[k] = fmaxf(sc[k], sc[8 + k]);
#pragma unroll
            for (int i = 16; i < kKeys; i += 16)
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
            uint32_t pk[kKeys / 2];
            uint64_t acc2[4] = {0ull, 0ull, 0ull, 0ull};
            const uint64_t sc2 = f2(scale, scale), nm2 = f2(neg, neg);
#pragma unroll
            for (int i = 0; i < kKeys / 2; ++i)
                pk[i] = weights<kHalf>(sc[2 * i], sc[2 * i + 1], sc2, nm2, acc2[i & 3]);
            uint64_t accs = acc2[0];
            asm("add.f32x2 %0, %0, %1;" : "+l"(accs) : "l"(acc2[1]));
            asm("add.f32x2 %0, %0, %1;" : "+l"(accs) : "l"(acc2[2]));
            asm("add.f32x2 %0, %0, %1;" : "+l"(accs) : "l"(acc2[3]));
            float acc0, acc1;
            f2_split(accs, acc0, acc1);

            if (j > 0) {
                // O under the new reference, once the last P V has completed
                // (D = 64: which also frees P)
                const bool any = __any_sync(0xffffffffu, need);
                if (D == 64 || any) {
                    wait_o(gw - 1);
                    tc_fence_after();
                }
                if (any) {
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
            const uint32_t tP = c.tmem + L::col_p(w, gw) + lane_off;
            if constexpr (D == 64)
                tmem_st64(tP, pk);
            else
                tmem_st32(tP, pk);
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(bar(c, D == 128 && gw & 1 ? kBarPOdd + w : kBarPFull + w));
        }

        // ---- end of the segment: O / l to the output, or the state to this
        // CTA's part slot
        wait_o(gw - 1);
        if (stop(c))
            return;
        tc_fence_after();
        const bool whole = s.ke - s.kb == s.tiles;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        float *part = c.a.parts + (2ll * cta + (s.kb == 0)) * cross_slot_floats(L::kUnitRows, D);
        // this warp's rows of the output, those that the sequence has
        const int warp_row = kBlockM * w + 32 * warp_in_group;
        const int warp_rows = min(32, s.rows - s.q0 - warp_row);
        const int fold = c.a.fold_log2;
        uint16_t *out = static_cast<uint16_t *>(c.a.out) + static_cast<long long>(s.q_row) * c.a.out_row +
                        static_cast<long long>(s.head) * D;
        uint8_t *stage = c.sbase + L::kOffOut + (4 * w + warp_in_group) * (L::kOutRows * 128);
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
                // through shared memory, so that a store instruction writes
                // whole lines of 4 rows and not 16 bytes of 32 (chunk j of row
                // r at j ^ (r & 7): no bank conflicts either way)
#pragma unroll
                for (int r0 = 0; r0 < 32; r0 += L::kOutRows) {
                    if (L::kOutRows == 32 || lane / L::kOutRows == r0 / L::kOutRows) {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            *reinterpret_cast<uint4 *>(stage + 128 * (lane % L::kOutRows) + 16 * (i ^ (lane & 7))) =
                                make_uint4(pack2<kHalf>(o[8 * i] * inv, o[8 * i + 1] * inv),
                                           pack2<kHalf>(o[8 * i + 2] * inv, o[8 * i + 3] * inv),
                                           pack2<kHalf>(o[8 * i + 4] * inv, o[8 * i + 5] * inv),
                                           pack2<kHalf>(o[8 * i + 6] * inv, o[8 * i + 7] * inv));
                    }
                    __syncwarp();
#pragma unroll 2
                    for (int i = 0; i < L::kOutRows / 4; ++i) {
                        const int row = 4 * i + lane / 8, part = lane % 8;
                        const int at = s.q0 + warp_row + r0 + row;       // row of the sequence
                        if (r0 + row < warp_rows)
                            *reinterpret_cast<uint4 *>(out + (at >> fold) * c.a.out_row +
                                                       (at & ((1 << fold) - 1)) * D + 64 * h + 8 * part) =
                                *reinterpret_cast<const uint4 *>(stage + 128 * row + 16 * (part ^ (row & 7)));
                    }
                    __syncwarp();
                }
            } else {
                // [D/4][256 rows] float4: neighbouring rows side by side
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    reinterpret_cast<float4 *>(part)[(16 * h + i) * L::kUnitRows + rr] =
                        make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
            }
        }
        if (!whole)
            reinterpret_cast<float2 *>(part + L::kUnitRows * D)[rr] = make_float2(m, l);
        if (!whole && s.kb == 0 && rr == 0) {
            CrossRecord rec;
            rec.row0 = static_cast<long long>(s.q_row) + (s.q0 >> fold);
            rec.rows = min(L::kUnitRows, s.rows - s.q0);
            rec.head0 = s.head;
            rec.group = 1 << fold;
            rec.parts = s.parts;
            c.a.records[cta] = rec;
        }
    }
}

// The products that an issuer has issued are done before the CTA can exit and
// give its TMEM back.
__device__ __forceinline__ void drain_products(const Ctx &c, int issuer)
{
    mma_commit_warp(bar(c, kBarDrain + issuer));
    drain_wait(bar(c, kBarDrain + issuer), 0);
}

template <int D, int G, bool kHalf>
__global__ void __launch_bounds__(Layout<D, G>::kThreads, Layout<D, G>::kCtas)
attn_cross_kernel(const __grid_constant__ CrossArgs a)
{
    using L = Layout<D, G>;
    pdl_wait();
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *sbase = smem_raw + (base - raw);
    uint32_t *slot = reinterpret_cast<uint32_t *>(sbase + L::kOffBar + kSlotInBars);
    const int cta = blockIdx.x;

    // TMEM first, as the next CTA of this SM only starts once this one has given
    // up its right to allocate.  (The 12 warps of D = 64, alone on their SM, take
    // it after the search: 193 us against 197 for 8192 x 8192; the 16 of D = 128
    // lose 1 % so.)
    if constexpr (!L::kPair) {
        if (threadIdx.x < 32) {
            tmem_alloc(smem_u32(slot), L::kTmemCols);
            tmem_relinquish();
        }
    }
    if (threadIdx.x == 0 && a.records)
        a.records[cta].parts = 0;
    static_assert(sizeof(typename Split<D, G>::Deal) <= 4 * G * L::kOutRows * 128, "dealing");
    Split<D, G> split(a, a.heads >> a.fold_log2);
    // two tiles and a unit's fixed work per CTA at least
    constexpr int kLeast = 2 * Split<D, G>::kFull + Split<D, G>::kAlpha;
    const bool work = split.find(*reinterpret_cast<typename Split<D, G>::Scratch *>(sbase + L::kOffScratch), gridDim.x, kLeast,
                                 reinterpret_cast<typename Split<D, G>::Deal *>(sbase + L::kOffOut));
    if (work) {
        Ctx c{base, 0u, sbase, a, base + L::kOffBar};
        const int warp = threadIdx.x >> 5;
        const int lane = threadIdx.x & 31;
        if (threadIdx.x == 0) {
            tma_prefetch_desc(&a.tm_q);
            tma_prefetch_desc(&a.tm_k);
            tma_prefetch_desc(&a.tm_v);
            for (int q = 0; q < L::kQSets; ++q) {
                mbar_init(bar(c, kBarQFull + q), 1);
                mbar_init(bar(c, kBarQEmpty + q), G);   // one commit per issuer
            }
            for (int st = 0; st < L::kStages; ++st) {
                mbar_init(bar(c, kBarKFull + st), 1);
                mbar_init(bar(c, kBarKEmpty + st), G);
                mbar_init(bar(c, kBarVFull + st), 1);
                mbar_init(bar(c, kBarVEmpty + st), G + 1);  // and the mask warp
            }
            for (int w = 0; w < 2; ++w) {
                mbar_init(bar(c, kBarSFull + w), 1);
                mbar_init(bar(c, kBarSEmpty + w), D == 64 ? kBlockM : 1);   // (kBarSOdd: one commit)
                mbar_init(bar(c, kBarPFull + w), kBlockM);
                mbar_init(bar(c, kBarPOdd + w), kBlockM);
                mbar_init(bar(c, kBarODone + w), 1);
                mbar_init(bar(c, kBarOOdd + w), 1);
                mbar_init(bar(c, kBarOFree + w), kBlockM);
            }
            for (int i = 0; i < kRecs; ++i) {
                mbar_init(bar(c, kBarRecFull + i), 1);
                mbar_init(bar(c, kBarRecEmpty + i), L::kRecReaders);
            }
            for (int i = 0; i < kMaskSlots; ++i) {
                mbar_init(bar(c, kBarBitsFull + i), 1);
                mbar_init(bar(c, kBarBitsEmpty + i), L::kUnitRows);
                mbar_init(bar(c, kBarVClean + i), 1);
            }
            for (int i = 0; i < 4; ++i)
                mbar_init(bar(c, kBarDrain + i), 1);
            sts32(c.bars + kGaveUpInBars, 0u);
            fence_mbar_init();
        }
        if constexpr (L::kPair) {
            if (warp == 0) {
                tmem_alloc(smem_u32(slot), L::kTmemCols);
                tmem_relinquish();
            }
        }
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        c.tmem = *slot;

        if (warp >= L::kControl) {
            asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(L::kRegsControl));
            if (warp == L::kControl) {
                if (lane == 0)
                    producer<D, G>(c, split);
            } else if (warp == L::kControl + 1) {
                mask_stager<D, G>(c, lane);
            } else if (warp < L::kControl + 2 + G) {
                if constexpr (L::kSplitIssuers)
                    s_issuer<D, G, kHalf>(c, warp - L::kControl - 2, lane);
                else
                    so_issuer<G, kHalf>(c, warp - L::kControl - 2, lane);
                drain_products(c, warp - L::kControl - 2);
            } else if (warp < L::kControl + 2 + 2 * G) {
                if constexpr (L::kSplitIssuers) {
                    o_issuer<D, G, kHalf>(c, warp - L::kControl - 2 - G, lane);
                    drain_products(c, warp - L::kControl - 2);
                }
            }
            __syncwarp();
        } else {
            asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(L::kRegsSoftmax));
            softmax_group<D, G, kHalf>(c, warp >> 2, warp & 3, lane, cta);
            __syncwarp();
        }
        if constexpr (L::kPair) {
            tc_fence_before();
            __syncthreads();
            if (warp == 0) {
                tc_fence_after();
                tmem_dealloc(c.tmem, L::kTmemCols);
            }
        }
    }
    if constexpr (!L::kPair) {
        tc_fence_before();
        __syncthreads();
        if (threadIdx.x < 32) {
            tc_fence_after();
            tmem_dealloc(*slot, L::kTmemCols);
        }
    }
    pdl_trigger();
}

template <int D, int G, bool kHalf>
cudaError_t launch(const CrossArgs &a, int ctas, cudaStream_t stream)
{
    static PerDeviceOnce smem_once;
    cudaError_t e = smem_opt_in(smem_once, attn_cross_kernel<D, G, kHalf>, Layout<D, G>::kSmemBytes);
    if (e != cudaSuccess)
        return e;
    return launch_chained(attn_cross_kernel<D, G, kHalf>, dim3(ctas), dim3(Layout<D, G>::kThreads), Layout<D, G>::kSmemBytes, stream, a);
}

}  // namespace

cudaError_t launch_cross_blocks(const CrossArgs &a, int dim, bool half, int unit_rows, int ctas, cudaStream_t stream)
{
    if (dim == 64 && unit_rows == kCrossSmallRows)
        return half ? launch<64, 1, true>(a, ctas, stream) : launch<64, 1, false>(a, ctas, stream);
    if (dim == 64)
        return half ? launch<64, 2, true>(a, ctas, stream) : launch<64, 2, false>(a, ctas, stream);
    if (unit_rows == kCrossSmallRows)
        return half ? launch<128, 1, true>(a, ctas, stream) : launch<128, 1, false>(a, ctas, stream);
    return half ? launch<128, 2, true>(a, ctas, stream) : launch<128, 2, false>(a, ctas, stream);
}

}  // namespace mbert
