// Host side of the calls beside the attention block: argument checks of the
// rotary and norm calls, the rotation's frequencies.
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
            !std::isfinite(rope->amplitude))
            return MBERT_ERR_BAD_ARG;
        for (int m = 0; m < a.rot / 2; ++m) {
            if (!(rope->freq[m] >= 0.0) || !std::isfinite(rope->freq[m]))
                return MBERT_ERR_BAD_ARG;
            // turns per position modulo 1 as a 64-bit binary fraction
            double t = rope->freq[m] / kTwoPi;
            t -= std::floor(t);
            const double t32 = std::ldexp(t, 32), hi = std::floor(t32);
            a.turns[m] = (static_cast<uint64_t>(hi) << 32) +
                         static_cast<uint64_t>(std::floor(std::ldexp(t32 - hi, 32)));
        }
        // exactly one source of positions
        if (positions) {
            if ((position_bits != 32 && position_bits != 64) || cu ||
                reinterpret_cast<uintptr_t>(positions) % (position_bits / 8))
                return MBERT_ERR_BAD_ARG;
            (position_bits == 32 ? reinterpret_cast<const void *&>(a.pos32)
                                 : reinterpret_cast<const void *&>(a.pos64)) = positions;
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
    a.amplitude = a.rot > 0 ? static_cast<float>(rope->amplitude) : 1.f;
    a.sin_amplitude = inverse ? -a.amplitude : a.amplitude;
    a.tokens = tokens;
    a.err = h->err;
    DeviceGuard g(h->device);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = launch_rotary(a, h->num_sms, st);
    h->launches += 1;
    h->last_stream = st;
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
