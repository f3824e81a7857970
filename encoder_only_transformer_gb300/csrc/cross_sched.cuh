// The split of cross attention among CTAs, shared by its kernels.
//
// A unit is one (sequence, head, block of query rows); it takes tiles(s) key
// tiles.  All units stand one after the other on a line of costs, in order of
// sequence, head, block: a unit takes kFull for each tile (kHalf where only
// half of its block holds rows: the last block of a sequence) and kAlpha for
// its fixed work (the query load, the end of its softmax, its output).  CTA c
// of n owns the tiles that begin in [c X / n, (c + 1) X / n), X the line's
// length; so every CTA gets the same cost whatever the lengths of the
// sequences, and a long unit among few is cut between many CTAs.  A border
// that falls into a unit of kSnap tiles or fewer (into any, where the call has
// no records of cut units) moves to that unit's start: joining its parts would
// cost more than it evens out.
//
// No list of the work is made: each CTA sums the sequences' costs and finds
// its own range, one thread per sequence.
//
// Where the units are few (kRounds to a CTA at most), they are first dealt out
// whole, the longest first, in rounds that run forth and back over the CTAs;
// if the CTA with the most gets no more than the line's share and kJoin, what
// cutting and joining costs, they stay so.  12 sequences of 250 queries over
// 1000 keys, 12 heads of 64: 21.0 us, 25.5 cut; 24 of 256 over 600 to 1000 evenly: 29.9,
// 33.6 cut; 9 of 250 over 1000, 32 heads over 8 of 128: 41.6, 50.4 cut; 64 of 30 over
// 600, 12 heads of 64: 36.1, 42.4 cut.  What it loses is its search, where no unit is
// long enough to be cut: 100 of 20 over 250: 33.5, 30.9 without.  With the longest
// unit 34 above the share (16 sequences of 118 to 1946 keys) both took 32.5 to
// 33.  Divisions stay the compiler's 64-bit ones: 32-bit ones where the costs
// allow, a branch at each, made 8192 x 8192 1 % slower.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace mbert {

// kBlockQ: query rows of a unit (0: all of a sequence's), each the rows of
// 2^fold_log2 heads, side by side; kTile: keys of a tile; kRounds 0: units are
// never dealt out whole; kPerSm: CTAs of an SM.
template <int kThreads, int kBlockQ_, int kTile_, int kFull_, int kHalf_, int kAlpha_, int kSnap_, int kRounds = 0,
          int kJoin = 0, int kPerSm = 1>
struct CrossSplit {
    static constexpr int kBlockQ = kBlockQ_, kTile = kTile_, kSnap = kSnap_;
    static constexpr int kFull = kFull_, kHalf = kHalf_, kAlpha = kAlpha_;
    static constexpr int kWarps = kThreads / 32;
    // Sequences whose units are dealt out, at most: two threads rank each, and the
    // lists must fit the output's staging place.  One more costs what dealing gains
    // (20 queries over 550 keys, 6 heads of 64: 128 sequences 36.3 us, 129 42.5).
    static constexpr int kDealSeqs = 128;
    static_assert(kRounds == 0 || 2 * kDealSeqs <= kThreads, "two threads per sequence");

    struct Scratch {
        long long warp[kWarps];
        long long base[2];
        int seq[2];
        int units[kWarps], most[kWarps], least[kWarps];
        int deal_seq[kRounds + 1], deal_unit[kRounds + 1];      // this CTA's whole units
    };
    // What dealing takes besides, while find() runs.
    struct Deal {
        int2 need[kDealSeqs];           // cost of a whole block, units
        int2 tail[kDealSeqs];           // cost of the last block, blocks
        int2 order[kDealSeqs];          // by length: first unit, sequence
    };

    // What a sequence needs: rows, tiles, blocks of query rows.
    struct Seq {
        int q_row, q_len, k_row, k_all, tiles;
        int rows;               // q_len times the heads that share a block
        int k_len, k_full;      // up to the last visible key, before the first hidden one
        int whole;              // blocks of cost kFull a tile
        int half;               // 1: the last block costs kHalf a tile
        // costs of a whole block, of one head, of the sequence
        __device__ __forceinline__ long long block() const { return static_cast<long long>(tiles) * kFull + kAlpha; }
        __device__ __forceinline__ long long head() const
        {
            return whole * block() + half * (static_cast<long long>(tiles) * kHalf + kAlpha);
        }
    };

    // Where a place x of a sequence lies: its unit, and that unit's start.
    struct Place {
        int head, b;            // head, block
        int per;                // cost of a tile
        long long xa, end;      // the unit's start and the next one's
    };
    __device__ __forceinline__ Place place(const Seq &q, long long base, long long x) const
    {
        const long long ch = q.head(), cb = q.block();
        Place p;
        p.head = static_cast<int>((x - base) / ch);
        const long long h0 = base + p.head * ch;
        const long long b = (x - h0) / cb;
        p.b = b < q.whole ? static_cast<int>(b) : q.whole;
        p.per = p.b < q.whole ? kFull : kHalf;
        p.xa = h0 + p.b * cb;
        p.end = p.b < q.whole ? p.xa + cb : h0 + ch;
        return p;
    }

    const CrossArgs &a;
    int unit_heads;         // heads that units are made for
    int ctas;
    long long total;        // X
    long long lo, hi;       // this CTA's range
    int seq0;               // the sequence that holds lo, and where it starts
    long long base0;
    const Scratch *dealt = nullptr;     // whole units, dealt out

    __device__ explicit CrossSplit(const CrossArgs &args, int heads) : a(args), unit_heads(heads) {}

    __device__ __forceinline__ Seq load(int s) const
    {
        Seq q;
        if (a.cu_q) {
            q.q_row = __ldg(a.cu_q + s);
            q.q_len = __ldg(a.cu_q + s + 1) - q.q_row;
        } else {
            q.q_row = s * a.len_q;
            q.q_len = a.len_q;
        }
        if (a.cu_k) {
            q.k_row = __ldg(a.cu_k + s);
            q.k_all = __ldg(a.cu_k + s + 1) - q.k_row;
        } else {
            q.k_row = s * a.len_k;
            q.k_all = a.len_k;
        }
        q.k_len = q.k_full = q.k_all;
        if (a.key_len) {
            const int2 v = __ldg(a.key_len + s);
            q.k_len = min(q.k_all, v.x);
            q.k_full = min(q.k_len, v.y);
        }
        q.tiles = max(1, (q.k_len + kTile - 1) / kTile);
        if constexpr (kBlockQ > 0) {
            q.rows = q.q_len << a.fold_log2;
            const int rest = q.rows % kBlockQ;
            q.half = kHalf != kFull && rest > 0 && rest <= kBlockQ / 2;
            q.whole = q.rows / kBlockQ + (rest > 0 && !q.half);
        } else {
            q.rows = q.q_len;
            q.half = 0;
            q.whole = q.q_len > 0;
        }
        return q;
    }

    __device__ __forceinline__ long long cost(const Seq &q) const { return unit_heads * q.head(); }

    __device__ __forceinline__ long long border(int c) const
    {
        return c * total / ctas;
    }

    // The CTA whose range holds x (borders inside long units do not move).
    __device__ __forceinline__ int cta_of(long long x) const
    {
        return static_cast<int>(((x + 1) * ctas - 1) / total);
    }

    // Every thread of the block.  min_cost: of a CTA, at least kFull, so that
    // every CTA inside a unit's tiles has one.  False: nothing to do for this
    // CTA (or the offsets are bad, then *a.err says so and no CTA does anything).
    // work: memory for dealing, free again afterwards (kRounds > 0).
    __device__ bool find(Scratch &sm, int max_ctas, int min_cost, Deal *work = nullptr)
    {
        const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
        long long sum = 0;
        int bad = 0, units = 0, most = 0, least = INT32_MAX;    // most, least: cost of a unit
        for (int s = tid; s < a.n_seqs; s += kThreads) {
            const Seq q = load(s);
            if (q.q_len < 0 || q.k_all < 0 || q.q_row < 0 || q.k_row < 0 ||
                static_cast<long long>(q.q_row) + q.q_len > a.rows_q ||
                static_cast<long long>(q.k_row) + q.k_all > a.rows_k)
                bad |= kErrBadCu;
            else if (q.q_len > a.max_q)
                bad |= kErrTooLong;
            else {
                sum += cost(q);
                // (only compared with few)
                units = static_cast<int>(min(1ll << 20, units + static_cast<long long>(unit_heads) * (q.whole + q.half)));
                if (q.whole + q.half > 0) {
                    const int unit = q.tiles * (q.whole ? kFull : kHalf) + kAlpha;
                    most = max(most, unit);
                    least = min(least, unit);
                }
            }
        }
        if (tid == 0 && ((a.cu_q && a.cu_q[0] != 0) || (a.cu_k && a.cu_k[0] != 0)))
            bad |= kErrBadCu;
#pragma unroll
        for (int d = 16; d; d >>= 1)
            sum += __shfl_xor_sync(0xffffffffu, sum, d);
        if constexpr (kRounds > 0) {
            units = __reduce_add_sync(0xffffffffu, units);
            most = __reduce_max_sync(0xffffffffu, most);
            least = __reduce_min_sync(0xffffffffu, least);
        }
        if (lane == 0) {
            sm.warp[warp] = sum;
            sm.units[warp] = units;
            sm.most[warp] = most;
            sm.least[warp] = least;
        }
        if (tid < 2)
            sm.seq[tid] = -1;
        const int any = __syncthreads_or(bad);
        if (any) {
            if (bad && blockIdx.x == 0)
                atomicOr(a.err, bad);
            return false;
        }
        total = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
            total += sm.warp[w];
        if (total == 0)
            return false;
        const long long want = total / min_cost;
        ctas = want < 1 ? 1 : want < max_ctas ? static_cast<int>(want) : max_ctas;
        if constexpr (kRounds > 0) {
            int all = 0, longest = 0, shortest = INT32_MAX;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                all += sm.units[w];
                longest = max(longest, sm.most[w]);
                shortest = min(shortest, sm.least[w]);
            }
            // an SM gets its second unit when every one has a first (152 units over
            // 512 keys: 14.1 -> 10.8 us)
            if (kPerSm == 2 && all <= max_ctas / 2 && !a.records)
                ctas = min(ctas, max_ctas / 2);
            const long long share = total / ctas;
            const long long limit = a.records ? share + kJoin : INT64_MAX;
            // (not worth dealing where one unit, or the shortest in every round, is
            // above the limit)
            const int rounds = (all + max_ctas - 1) / max_ctas;
            if (a.n_seqs <= kDealSeqs && rounds <= kRounds && longest <= limit &&
                static_cast<long long>(rounds) * shortest <= limit && deal(sm, *work, max_ctas, all, limit)) {
                dealt = &sm;
                return sm.deal_seq[0] >= 0;
            }
        }
        if (static_cast<int>(blockIdx.x) >= ctas)
            return false;
        lo = border(blockIdx.x);
        hi = border(blockIdx.x + 1);
        // the sequences that hold lo and hi
        long long carry = 0;
        for (int s0 = 0; s0 < a.n_seqs; s0 += kThreads) {
            const int s = s0 + tid;
            const long long v = s < a.n_seqs ? cost(load(s)) : 0;
            long long incl = v;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const long long o = __shfl_up_sync(0xffffffffu, incl, d);
                if (lane >= d)
                    incl += o;
            }
            __syncthreads();            // the sums of the last round are read
            if (lane == 31)
                sm.warp[warp] = incl;
            __syncthreads();
            long long before = carry, all = carry;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                before += w < warp ? sm.warp[w] : 0;
                all += sm.warp[w];
            }
            const long long start = before + incl - v;
            if (start <= lo && lo < start + v) {
                sm.seq[0] = s;
                sm.base[0] = start;
            }
            if (start <= hi && hi < start + v) {
                sm.seq[1] = s;
                sm.base[1] = start;
            }
            carry = all;
            if (carry > hi)
                break;
        }
        __syncthreads();
        seq0 = sm.seq[0];
        base0 = sm.base[0];
        lo = snap(lo, seq0, base0);
        hi = snap(hi, sm.seq[1], sm.base[1]);   // none for hi = total: stays
        return lo < hi;
    }

    // Deals the units out whole: true if no CTA gets more than `limit`.
    __device__ bool deal(Scratch &sm, Deal &d, int n, int all, long long limit)
    {
        const int tid = threadIdx.x;
        constexpr int kStep = 8;
        if (tid < a.n_seqs) {
            const Seq q = load(tid);
            const int full = q.tiles * kFull + kAlpha, half = q.tiles * kHalf + kAlpha;
            d.need[tid] = make_int2(q.whole ? full : half, unit_heads * (q.whole + q.half));
            d.tail[tid] = make_int2(q.half ? half : full, q.whole + q.half);
        } else if (tid < kDealSeqs) {
            d.need[tid] = make_int2(-1, 0);             // shorter than any
            d.order[tid] = make_int2(INT32_MAX, 0);     // behind all
        }
        if (tid <= kRounds)
            sm.deal_seq[tid] = -1;
        __syncthreads();
        // two threads per sequence: the units of the longer ones come first
        {
            const int s = tid / 2, mine = s < a.n_seqs ? d.need[s].x : 0;
            int rank = 0, start = 0;
            for (int o = tid % 2 * kStep; o < a.n_seqs; o += 2 * kStep) {
                int2 x[kStep];
#pragma unroll
                for (int i = 0; i < kStep; ++i)
                    x[i] = d.need[o + i];
#pragma unroll
                for (int i = 0; i < kStep; ++i) {
                    const bool before = x[i].x > mine || (x[i].x == mine && o + i < s);
                    rank += before;
                    start += before ? x[i].y : 0;
                }
            }
            rank += __shfl_xor_sync(0xffffffffu, rank, 1);
            start += __shfl_xor_sync(0xffffffffu, start, 1);
            if (s < a.n_seqs && tid % 2 == 0)
                d.order[rank] = make_int2(start, s);
        }
        __syncthreads();
        // a thread per CTA: its units, one of each round, of the last sequence
        // that starts at them or before (the rounds' searches side by side)
        int top = 1;
        while (2 * top < a.n_seqs)
            top *= 2;
        bool over = false;
        for (int c = tid; c < n; c += kThreads) {
            int at[kRounds], lo[kRounds];
#pragma unroll
            for (int r = 0; r < kRounds; ++r) {
                at[r] = r * n + (r & 1 ? n - 1 - c : c);
                lo[r] = 0;
            }
            for (int step = top; step > 0; step /= 2)
#pragma unroll
                for (int r = 0; r < kRounds; ++r)
                    if (d.order[lo[r] + step].x <= at[r])
                        lo[r] += step;
            long long sum = 0;
#pragma unroll
            for (int r = 0; r < kRounds; ++r)
                if (at[r] < all) {
                    const int2 x = d.order[lo[r]], tail = d.tail[x.y];
                    const int unit = at[r] - x.x;
                    sum += unit % tail.y == tail.y - 1 ? tail.x : d.need[x.y].x;
                    if (c == static_cast<int>(blockIdx.x)) {
                        sm.deal_seq[r] = x.y;
                        sm.deal_unit[r] = unit;
                    }
                }
            over |= sum > limit;
        }
        return !__syncthreads_or(over);
    }

    __device__ __forceinline__ long long snap(long long x, int s, long long base) const
    {
        if (s < 0)
            return x;
        const Seq q = load(s);
        if (a.records && q.tiles > kSnap)
            return x;
        return place(q, base, x).xa;
    }

    // A run of key tiles [kb, ke) of one unit.
    struct Seg {
        Seq s;
        int seq, head, q0;
        int kb, ke;
        int per;            // cost of a tile
        long long xa;       // place of the unit's first tile
    };

    // Walks this CTA's segments in order.
    struct Iter {
        int seq = -1;           // (dealt units: the round)
        long long base = 0, x = 0;
        Seq s;
    };

    __device__ __forceinline__ Iter begin() const
    {
        Iter it;
        if (kRounds > 0 && dealt) {
            it.seq = 0;
            return it;
        }
        it.seq = seq0;
        it.base = base0;
        it.x = lo;
        it.s = load(seq0);
        return it;
    }

    __device__ bool next(Iter &it, Seg &g) const
    {
        if constexpr (kRounds > 0) {
            if (dealt) {
                g.seq = dealt->deal_seq[it.seq];
                if (g.seq < 0)
                    return false;
                const int unit = dealt->deal_unit[it.seq++];
                g.s = load(g.seq);
                const int blocks = g.s.whole + g.s.half;
                g.head = unit / blocks;
                g.q0 = unit % blocks * kBlockQ;
                g.kb = 0;
                g.ke = g.s.tiles;
                return true;
            }
        }
        while (it.x < hi) {
            if (it.x - it.base >= cost(it.s)) {
                it.base += cost(it.s);
                if (++it.seq >= a.n_seqs)
                    return false;
                it.s = load(it.seq);
                continue;
            }
            const Place p = place(it.s, it.base, it.x);
            const int kb = static_cast<int>((it.x - p.xa + p.per - 1) / p.per);
            const long long cut = (hi - p.xa + p.per - 1) / p.per;
            g.ke = cut < it.s.tiles ? static_cast<int>(cut) : it.s.tiles;
            it.x = p.end;
            if (kb >= g.ke)
                continue;       // x lies behind the unit's tiles, or hi before the next one
            g.s = it.s;
            g.seq = it.seq;
            g.head = p.head;
            g.q0 = p.b * kBlockQ;
            g.kb = kb;
            g.xa = p.xa;
            g.per = p.per;
            return true;
        }
        return false;
    }

    // Parts that a cut unit has.
    __device__ __forceinline__ int parts(const Seg &g) const
    {
        return cta_of(g.xa + static_cast<long long>(g.s.tiles - 1) * g.per) - cta_of(g.xa) + 1;
    }
};

}  // namespace mbert
