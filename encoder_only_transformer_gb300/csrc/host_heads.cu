// Host side of the calls beside the attention block: argument checks of the
// rotary, norm and cross-attention calls, the rotation's frequencies, the
// choice of the cross-attention kernel.
#include <algorithm>
#include <cmath>

#include "mbert_attn.h"
#include "common.cuh"
#include "handle.h"
#include "internal.h"

#define MBERT_API extern "C" __attribute__((visibility("default")))

using namespace mbert;

namespace {

constexpr double kTwoPi = 6.283185307179586476925;

// The extent in bytes of elements (t, h, d): t * row + h * head + d.
struct Extent {
    uintptr_t lo, hi;
};

Extent extent(const void *p, long long tokens, long long row, int heads, long long head, int dim, int es)
{
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return {lo, lo + static_cast<uintptr_t>(((tokens - 1) * row + (heads - 1) * head + dim) * es)};
}

// May some element of a (written) be an element of b?  Exact where both have
// the same row stride and each row's heads lie within it (column blocks of
// the same rows); else by extent.
bool may_overlap(Extent a, long long arow, long long awidth, Extent b, long long brow, long long bwidth, int es)
{
    if (a.hi <= b.lo || b.hi <= a.lo)
        return false;
    if (arow != brow || arow <= 0 || awidth > arow || bwidth > arow)
        return true;
    const uintptr_t pitch = static_cast<uintptr_t>(arow) * es;
    const uintptr_t d = b.lo >= a.lo ? (b.lo - a.lo) % pitch : (pitch - (a.lo - b.lo) % pitch) % pitch;
    return !(d >= static_cast<uintptr_t>(awidth) * es && d + static_cast<uintptr_t>(bwidth) * es <= pitch);
}

constexpr long long kMaxStride = 1ll << 40;
// Elements from a tensor's first to its last, at most: beyond any device's
// memory, and far from where extents in bytes would overflow.
constexpr long long kMaxSpan = 1ll << 48;

// (rows - 1) * pitch stays within kMaxSpan
bool span_ok(long long rows, long long pitch) { return rows <= 1 || pitch <= kMaxSpan / (rows - 1); }

// Rows of a packed tensor, at most: places up to a tile behind the last row
// (and a block's stride behind that) still fit 32 bits.
constexpr long long kMaxRows = INT32_MAX - 1024;

int check_heads(const mbert_attn_heads &x, long long T, int dim, int es, bool weight)
{
    if (!x.src || !x.dst || (weight && !x.weight) || x.heads < 1 || x.heads > 65536)
        return MBERT_ERR_BAD_ARG;
    for (const void *p : {x.src, static_cast<const void *>(x.dst), weight ? x.weight : x.src})
        if (reinterpret_cast<uintptr_t>(p) % es)
            return MBERT_ERR_BAD_ARG;
    for (int64_t s : {x.src_row, x.src_head, x.dst_row, x.dst_head})
        if (s < 0 || s > kMaxStride)
            return MBERT_ERR_BAD_ARG;
    if (!span_ok(T, x.src_row) || !span_ok(T, x.dst_row) || !span_ok(x.heads, x.src_head) ||
        !span_ok(x.heads, x.dst_head))
        return MBERT_ERR_BAD_ARG;
    // the elements of dst are distinct: heads within rows, or rows within heads
    const bool heads_apart = x.heads == 1 || x.dst_head >= dim;
    const bool rows_apart = T == 1 || x.dst_row >= dim;
    const long long hw = (x.heads - 1) * x.dst_head + dim, rw = (T - 1) * x.dst_row + dim;
    if (!heads_apart || !rows_apart ||
        (T > 1 && x.heads > 1 && x.dst_row < hw && x.dst_head < rw))
        return MBERT_ERR_BAD_ARG;
    return MBERT_OK;
}

// The written rows of `w` against what the call reads (or writes) of `r`.
bool clash(const mbert_attn_heads &w, const void *p, long long prow, long long phead, int pheads,
           bool in_place_ok, long long T, int dim, int es)
{
    if (in_place_ok && p == w.dst && (T == 1 || prow == w.dst_row) && (pheads == 1 || phead == w.dst_head))
        return false;
    return may_overlap(extent(w.dst, T, w.dst_row, w.heads, w.dst_head, dim, es), w.dst_row,
                       (w.heads - 1) * w.dst_head + dim, extent(p, T, prow, pheads, phead, dim, es), prow,
                       (pheads - 1) * phead + dim, es);
}

int rotary_impl(mbert_attn *h, const mbert_attn_heads *const (&xs)[2], int64_t tokens, int head_dim, int dtype,
                int norm, float eps, const mbert_attn_rotary_spec *rope, const void *positions,
                int position_bits, const int32_t *cu, int n_seqs, int inverse, void *stream)
{
    if (!h || (!xs[0] && !xs[1]) || tokens < 0 || tokens > INT32_MAX || head_dim < 2 || head_dim > 256 ||
        (head_dim & 1) || dtype < MBERT_BF16 || dtype > MBERT_F32 || !(eps >= 0.f) || eps > 1.f)
        return MBERT_ERR_BAD_ARG;
    RotaryArgs a;
    a.dim = head_dim;
    a.rot = rope ? rope->dim : 0;
    if (a.rot < 0 || a.rot > head_dim || (a.rot & 1))
        return MBERT_ERR_BAD_ARG;
    if (a.rot > 0) {
        if ((rope->layout != MBERT_ROTARY_HALF && rope->layout != MBERT_ROTARY_INTERLEAVED) ||
            !std::isfinite(static_cast<float>(rope->amplitude)))    // (fp32 in the kernel)
            return MBERT_ERR_BAD_ARG;
        for (int m = 0; m < a.rot / 2; ++m) {
            if (!(rope->freq[m] >= 0.0) || !std::isfinite(rope->freq[m]))
                return MBERT_ERR_BAD_ARG;
            // turns per position modulo 1 as a 64-bit binary fraction
            double t = rope->freq[m] / kTwoPi;
            t -= std::floor(t);
            const double t32 = t * 0x1p32, hi = std::floor(t32);
            a.turns[m] = (static_cast<uint64_t>(hi) << 32) + static_cast<uint64_t>((t32 - hi) * 0x1p32);
        }
        // exactly one source of positions
        if (positions) {
            if ((position_bits != 32 && position_bits != 64) || cu ||
                reinterpret_cast<uintptr_t>(positions) % (position_bits / 8))
                return MBERT_ERR_BAD_ARG;
            if (position_bits == 32)
                a.pos32 = static_cast<const int32_t *>(positions);
            else
                a.pos64 = static_cast<const int64_t *>(positions);
        } else if (tokens > 0) {
            if (!cu || n_seqs < 1 || (reinterpret_cast<uintptr_t>(cu) & 3))
                return MBERT_ERR_BAD_ARG;
            a.cu = cu;
            a.n_seqs = n_seqs;
        }
    } else if (positions || cu) {
        return MBERT_ERR_BAD_ARG;   // nothing to turn by them
    }
    if (tokens == 0)
        return MBERT_OK;
    const int es = dtype == MBERT_F32 ? 4 : 2;
    for (int t = 0; t < 2; ++t) {
        if (!xs[t])
            continue;
        const mbert_attn_heads &x = *xs[t];
        const int rc = check_heads(x, tokens, head_dim, es, norm != 0);
        if (rc != MBERT_OK)
            return rc;
        RotaryRows &r = a.x[t];
        r.src = x.src;
        r.dst = x.dst;
        r.weight = x.weight;
        r.heads = x.heads;
        r.src_row = x.src_row;
        r.src_head = x.src_head;
        r.dst_row = x.dst_row;
        r.dst_head = x.dst_head;
    }
    for (int t = 0; t < 2; ++t) {
        if (!xs[t])
            continue;
        const mbert_attn_heads &w = *xs[t];
        const Extent we = extent(w.dst, tokens, w.dst_row, w.heads, w.dst_head, head_dim, es);
        auto hits = [&](const void *p, uintptr_t bytes) {
            const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
            return p && we.lo < lo + bytes && lo < we.hi;
        };
        if (hits(positions, tokens * (position_bits / 8)) || hits(a.cu, (n_seqs + 1ull) * 4))
            return MBERT_ERR_BAD_ARG;
        for (int r = 0; r < 2; ++r) {
            if (!xs[r])
                continue;
            const mbert_attn_heads &x = *xs[r];
            if (clash(w, x.src, x.src_row, x.src_head, x.heads, r == t, tokens, head_dim, es) ||
                (r != t && clash(w, x.dst, x.dst_row, x.dst_head, x.heads, false, tokens, head_dim, es)) ||
                (norm && hits(x.weight, static_cast<uintptr_t>(head_dim) * es)))
                return MBERT_ERR_BAD_ARG;
        }
    }
    a.dtype = dtype;
    a.interleaved = a.rot > 0 && rope->layout == MBERT_ROTARY_INTERLEAVED;
    a.norm = norm;
    a.eps = eps;
    // Squares that fp32 rounds to nothing (below 2^-149, so a sum of 2^-90 of 256
    // numbers is off by 2^-51 of itself at most) only matter beside an eps below
    // 2^-40.  A scale of 2^k keeps eps 2^2k at 2^100 or less; where that holds k
    // down, eps is all that counts of the sum.
    constexpr uint32_t kBits2M90 = (127 - 90) << 23, kBits2P126 = (127 + 126) << 23;
    a.least_squares = eps >= 0x1p-40f ? 0 : kBits2M90;
    a.squares = kBits2P126 - a.least_squares;
    a.most_scale = eps > 0.f ? std::ldexp(1.f, std::min(126, (100 - std::ilogb(eps)) / 2)) : 0x1p126f;
    a.amplitude = a.rot > 0 ? static_cast<float>(rope->amplitude) : 1.f;
    a.sin_amplitude = inverse ? -a.amplitude : a.amplitude;
    a.tokens = tokens;
    a.err = h->err;
    DeviceGuard g(h->device);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = launch_rotary(a, h->num_sms, st);
    h->launches += 1;
    return e == cudaSuccess ? MBERT_OK : MBERT_ERR_CUDA;
}

}  // namespace

MBERT_API int mbert_attn_rotary_init(mbert_attn_rotary_spec *spec, int dim, int layout, double base,
                                     const mbert_attn_scaling *scaling)
{
    if (!spec || dim < 0 || dim > 2 * kMaxRotaryPairs || (dim & 1) || !(base > 1.0) || !std::isfinite(base) ||
        (layout != MBERT_ROTARY_HALF && layout != MBERT_ROTARY_INTERLEAVED))
        return MBERT_ERR_BAD_ARG;
    const int kind = scaling ? scaling->kind : MBERT_SCALING_NONE;
    const double s = kind == MBERT_SCALING_NONE ? 1.0 : scaling->factor;
    if (kind < MBERT_SCALING_NONE || kind > MBERT_SCALING_YARN || !(s > 0.0) || !std::isfinite(s) ||
        (kind >= MBERT_SCALING_NTK && s < 1.0) || (kind == MBERT_SCALING_NTK && dim <= 2))
        return MBERT_ERR_BAD_ARG;
    const bool borders = kind == MBERT_SCALING_BY_PARTS || kind == MBERT_SCALING_YARN;
    if (borders && (!(scaling->original > 0.0) || !std::isfinite(scaling->original) || !(scaling->low > 0.0) ||
                    !(scaling->high > scaling->low) || !std::isfinite(scaling->high)))
        return MBERT_ERR_BAD_ARG;
    if (kind == MBERT_SCALING_YARN && (!(scaling->amplitude >= 0.0) || !std::isfinite(scaling->amplitude)))
        return MBERT_ERR_BAD_ARG;
    spec->dim = dim;
    spec->layout = layout;
    spec->amplitude = 1.0;
    for (double &f : spec->freq)
        f = 0.0;
    if (kind == MBERT_SCALING_NTK)
        base *= std::pow(s, static_cast<double>(dim) / (dim - 2));
    double lo = 0.0, hi = 0.0;   // YARN's borders as pair numbers
    if (kind == MBERT_SCALING_YARN && dim > 0) {
        auto pair_at = [&](double turns) {
            return dim * std::log(scaling->original / (turns * kTwoPi)) / (2.0 * std::log(base));
        };
        lo = std::fmax(std::floor(pair_at(scaling->high)), 0.0);
        hi = std::fmin(std::ceil(pair_at(scaling->low)), dim - 1.0);
        spec->amplitude = scaling->amplitude > 0.0 ? scaling->amplitude : 0.1 * std::log(s) + 1.0;
    }
    for (int m = 0; m < dim / 2; ++m) {
        double f = std::pow(base, -2.0 * m / dim);
        double keep = 1.0;       // share of the unscaled frequency
        if (kind == MBERT_SCALING_LINEAR)
            keep = 0.0;
        else if (kind == MBERT_SCALING_BY_PARTS)
            keep = (scaling->original * f / kTwoPi - scaling->low) / (scaling->high - scaling->low);
        else if (kind == MBERT_SCALING_YARN)
            keep = 1.0 - (m - lo) / std::fmax(hi - lo, 1e-3);
        keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
        spec->freq[m] = kind == MBERT_SCALING_NTK ? f : f * keep + f / s * (1.0 - keep);
    }
    return MBERT_OK;
}

MBERT_API int mbert_attn_rotary(mbert_attn *h, const mbert_attn_heads *x, int64_t tokens, int head_dim,
                                int dtype, const mbert_attn_rotary_spec *rope, const void *positions,
                                int position_bits, const int32_t *cu_seqlens, int n_seqs, int inverse,
                                void *stream)
{
    if (!rope || !x)
        return MBERT_ERR_BAD_ARG;
    const mbert_attn_heads *const xs[2] = {x, nullptr};
    return rotary_impl(h, xs, tokens, head_dim, dtype, 0, 0.f, rope, positions, position_bits, cu_seqlens,
                       n_seqs, inverse, stream);
}

MBERT_API int mbert_attn_qk_norm_rotary(mbert_attn *h, const mbert_attn_heads *q, const mbert_attn_heads *k,
                                        int64_t tokens, int head_dim, int dtype, int norm, float eps,
                                        const mbert_attn_rotary_spec *rope, const void *positions,
                                        int position_bits, const int32_t *cu_seqlens, int n_seqs,
                                        void *stream)
{
    if (norm != MBERT_NORM_RMS && norm != MBERT_NORM_LAYER)
        return MBERT_ERR_BAD_ARG;
    const mbert_attn_heads *const xs[2] = {q, k};
    return rotary_impl(h, xs, tokens, head_dim, dtype, norm, eps, rope, positions, position_bits, cu_seqlens,
                       n_seqs, 0, stream);
}

namespace {

// How a cross-attention call runs: the kernel, its CTAs and the workspace.
struct CrossPlan {
    bool token;             // few rows per sequence and key head
    bool join;              // a sequence may be long enough to be cut
    int group, max_q, ctas, unit_rows;
    int fold_log2;          // blocks: query heads that share a block's rows
    int64_t records, parts, lens, bits, bytes;      // offsets and the total
};

int64_t align256(int64_t x) { return (x + 255) & ~static_cast<int64_t>(255); }

// Checks everything but the device pointers' contents.
int cross_plan(const mbert_attn *h, const mbert_attn_cross_args *c, CrossPlan *p)
{
    if (!h || !c)
        return MBERT_ERR_BAD_ARG;
    if ((c->head_dim != 64 && c->head_dim != 128) || (c->dtype != MBERT_BF16 && c->dtype != MBERT_F16))
        return MBERT_ERR_UNSUPPORTED;
    if (c->heads < 1 || c->heads > 65536 || c->kv_heads < 1 || c->heads % c->kv_heads ||
        c->rows_q < 0 || c->rows_q > kMaxRows || c->rows_k < 0 || c->rows_k > kMaxRows || c->n_seqs < 0 ||
        c->max_seqlen_q < 0 || !(c->scale >= 0.f) || !std::isfinite(c->scale * 1.5f))
        return MBERT_ERR_BAD_ARG;
    if (c->n_seqs == 0 && (c->rows_q > 0 || c->rows_k > 0))
        return MBERT_ERR_BAD_ARG;
    if (c->n_seqs > 0 && ((!c->cu_q && c->rows_q % c->n_seqs) || (!c->cu_k && c->rows_k % c->n_seqs)))
        return MBERT_ERR_BAD_ARG;
    p->group = c->heads / c->kv_heads;
    int64_t most = c->cu_q || c->n_seqs == 0 ? c->rows_q : c->rows_q / c->n_seqs;
    if (c->max_seqlen_q > 0 && c->max_seqlen_q < most) {
        if (!c->cu_q)
            return MBERT_ERR_SEQ_TOO_LONG;
        most = c->max_seqlen_q;
    }
    p->max_q = static_cast<int>(most);
    // up to 16 rows per (sequence, key head): the kernel that reads K and V
    // once for all of them
    p->token = most * p->group <= kCrossTokenRows;
    p->fold_log2 = 0;
    while (!p->token && p->fold_log2 < 7 && (p->group >> p->fold_log2) % 2 == 0)
        ++p->fold_log2;
    if (most << p->fold_log2 > INT32_MAX)
        return MBERT_ERR_BAD_ARG;   // (more than any device holds)
    const bool small = most << p->fold_log2 <= kCrossSmallRows &&
                       (c->head_dim == 64 || c->rows_k <= kCrossSmallKeys * static_cast<int64_t>(c->n_seqs));
    p->unit_rows = p->token ? kCrossTokenRows : small ? kCrossSmallRows : kCrossBlockRows;
    p->ctas = h->num_sms * (p->token ? cross_token_ctas(c->head_dim) : cross_block_ctas(p->unit_rows));
    const int64_t longest = c->cu_k || c->n_seqs == 0 ? c->rows_k : c->rows_k / c->n_seqs;
    p->join = longest > (p->token ? kCrossTokenWholeRows : kCrossBlockWholeRows);
    p->records = 0;
    p->parts = p->join ? align256(static_cast<int64_t>(sizeof(CrossRecord)) * p->ctas) : 0;
    p->lens = p->join ? align256(p->parts + 2 * p->ctas * cross_slot_floats(p->unit_rows, c->head_dim) * 4) : 0;
    p->bits = c->key_mask ? align256(p->lens + 8ll * c->n_seqs) : p->lens;
    p->bytes = c->key_mask ? align256(p->bits + 4 * (key_bit_word(c->rows_k, c->n_seqs) + 1)) : p->lens;
    return MBERT_OK;
}

}  // namespace

MBERT_API int mbert_attn_cross_workspace(mbert_attn *h, const mbert_attn_cross_args *args, int64_t *bytes)
{
    CrossPlan p;
    if (!bytes)
        return MBERT_ERR_BAD_ARG;
    const int rc = cross_plan(h, args, &p);
    if (rc == MBERT_OK)
        *bytes = p.bytes;
    return rc;
}

MBERT_API int mbert_attn_cross(mbert_attn *h, const mbert_attn_cross_args *args, void *workspace,
                               int64_t workspace_bytes, void *stream)
{
    CrossPlan p;
    int rc = cross_plan(h, args, &p);
    if (rc != MBERT_OK)
        return rc;
    const mbert_attn_cross_args &c = *args;
    if (c.rows_q == 0)
        return MBERT_OK;
    const bool keys = c.rows_k > 0;
    if (!c.q || !c.out || (p.bytes > 0 && !workspace) || workspace_bytes < p.bytes || (keys && (!c.k || !c.v)))
        return MBERT_ERR_BAD_ARG;
    for (const void *ptr : {c.q, c.k, c.v, static_cast<const void *>(c.out), static_cast<const void *>(workspace)})
        if (reinterpret_cast<uintptr_t>(ptr) & 15)
            return MBERT_ERR_BAD_ARG;
    for (const void *ptr : {static_cast<const void *>(c.cu_q), static_cast<const void *>(c.cu_k),
                            static_cast<const void *>(c.key_mask)})
        if (reinterpret_cast<uintptr_t>(ptr) & 3)
            return MBERT_ERR_BAD_ARG;
    const int D = c.head_dim;
    const int64_t qw = static_cast<int64_t>(c.heads) * D, kw = static_cast<int64_t>(c.kv_heads) * D;
    // rows of whole 16-byte vectors that do not run into each other
    auto row_ok = [](int64_t pitch, int64_t width, int64_t n) {
        return pitch >= width && pitch % 8 == 0 && pitch < (1ll << 38) && span_ok(n, pitch);
    };
    if (!row_ok(c.q_row, qw, c.rows_q) || !row_ok(c.out_row, qw, c.rows_q) ||
        (keys && (!row_ok(c.k_row, kw, c.rows_k) || !row_ok(c.v_row, kw, c.rows_k))))
        return MBERT_ERR_BAD_ARG;
    auto rows = [&](const void *ptr, int64_t n, int64_t pitch, int64_t width) {
        const uintptr_t lo = reinterpret_cast<uintptr_t>(ptr);
        return Extent{lo, lo + static_cast<uintptr_t>(((n - 1) * pitch + width) * 2)};
    };
    auto flat = [&](const void *ptr, int64_t bytes) {
        const uintptr_t lo = reinterpret_cast<uintptr_t>(ptr);
        return Extent{lo, lo + static_cast<uintptr_t>(bytes)};
    };
    const Extent oe = rows(c.out, c.rows_q, c.out_row, qw);
    const Extent we = p.bytes > 0 ? flat(workspace, p.bytes) : Extent{0, 0};
    auto meet = [](Extent x, Extent y) { return x.lo < y.hi && y.lo < x.hi; };
    if (may_overlap(oe, c.out_row, qw, rows(c.q, c.rows_q, c.q_row, qw), c.q_row, qw, 2) || meet(oe, we) ||
        meet(we, rows(c.q, c.rows_q, c.q_row, qw)))
        return MBERT_ERR_BAD_ARG;
    if (keys) {
        const Extent ke = rows(c.k, c.rows_k, c.k_row, kw), ve = rows(c.v, c.rows_k, c.v_row, kw);
        if (may_overlap(oe, c.out_row, qw, ke, c.k_row, kw, 2) || may_overlap(oe, c.out_row, qw, ve, c.v_row, kw, 2) ||
            meet(we, ke) || meet(we, ve))
            return MBERT_ERR_BAD_ARG;
    }
    for (const Extent x : {flat(c.cu_q, c.cu_q ? 4ll * (c.n_seqs + 1) : 0), flat(c.cu_k, c.cu_k ? 4ll * (c.n_seqs + 1) : 0),
                           flat(c.key_mask, c.key_mask ? 4 * c.rows_k : 0)})
        if (x.hi > x.lo && (meet(oe, x) || meet(we, x)))
            return MBERT_ERR_BAD_ARG;

    DeviceGuard g(h->device);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    CrossArgs a;
    const int kbox = p.token ? 64 : cross_tile_keys(D, p.unit_rows);
    // A head's part of a row is what a CTA reads of it: 128 bytes for D = 64.
    // Fetching 256 brought the next head's in too, for nobody on a long cache
    // (672 MB from DRAM for 488 MB of keys and values).
    const int l2 = 2 * D;
    // without any key row the maps stand over q: all of it is masked
    if ((!p.token &&
         encode_heads(h, &a.tm_q, c.q, D, c.heads, c.rows_q, c.q_row, 1 << p.fold_log2) != MBERT_OK) ||
        encode_rows(h, &a.tm_k, keys ? c.k : c.q, keys ? kw : qw, keys ? c.rows_k : c.rows_q,
                    keys ? c.k_row : c.q_row, kbox, l2) != MBERT_OK ||
        encode_rows(h, &a.tm_v, keys ? c.v : c.q, keys ? kw : qw, keys ? c.rows_k : c.rows_q,
                    keys ? c.v_row : c.q_row, kbox, l2) != MBERT_OK)
        return MBERT_ERR_CUDA;
    a.q = c.q;
    a.out = c.out;
    a.q_row = c.q_row;
    a.out_row = c.out_row;
    a.cu_q = c.cu_q;
    a.cu_k = c.cu_k;
    a.n_seqs = c.n_seqs;
    a.len_q = c.cu_q ? 0 : static_cast<int>(c.rows_q / c.n_seqs);
    a.len_k = c.cu_k ? 0 : static_cast<int>(c.rows_k / c.n_seqs);
    a.rows_q = c.rows_q;
    a.rows_k = c.rows_k;
    a.max_q = p.max_q;
    a.heads = c.heads;
    a.group = p.group;
    a.fold_log2 = p.fold_log2;
    a.scale_log2 = static_cast<float>((c.scale > 0.f ? c.scale : 1.0 / std::sqrt(static_cast<double>(D))) *
                                      1.4426950408889634);
    a.err = h->err;
    char *ws = static_cast<char *>(workspace);
    if (p.join) {
        a.records = reinterpret_cast<CrossRecord *>(ws + p.records);
        a.parts = reinterpret_cast<float *>(ws + p.parts);
    }
    const bool half = c.dtype == MBERT_F16;
    cudaError_t e = cudaSuccess;
    if (c.key_mask && keys) {
        int2 *lens = reinterpret_cast<int2 *>(ws + p.lens);
        uint32_t *bits = reinterpret_cast<uint32_t *>(ws + p.bits);
        e = launch_key_bits(a, c.key_mask, bits, lens, st);
        a.key_len = lens;
        a.key_bits = bits;
        h->launches += 1;
    }
    if (e == cudaSuccess)
        e = p.token ? launch_cross_token(a, D, half, p.ctas, st) : launch_cross_blocks(a, D, half, p.unit_rows, p.ctas, st);
    h->launches += 1;
    if (e == cudaSuccess && p.join) {
        e = launch_cross_join(a, D, half, p.token ? p.max_q * p.group : p.unit_rows, p.ctas, st);
        h->launches += 1;
    }
    return e == cudaSuccess ? MBERT_OK : MBERT_ERR_CUDA;
}
