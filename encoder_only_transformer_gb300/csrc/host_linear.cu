// Host side of the products of any width and of the norms around a block: argument
// checks, tensor maps, the choice of the kernel.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "mbert_attn.h"
#include "common.cuh"
#include "handle.h"
#include "internal.h"
#include "linear.h"
#include "residual_norm.h"

#define MBERT_API extern "C" __attribute__((visibility("default")))

using namespace mbert;

namespace {

constexpr int64_t kMaxRows = INT32_MAX - 1024;
constexpr int kMaxWidth = 1 << 24;
// Elements from a tensor's first to its last, at most: beyond any device's memory,
// and far from where extents in bytes would overflow.
constexpr int64_t kMaxSpan = 1ll << 48;
constexpr int64_t kMaxPitch = 1ll << 38;    // what a tensor map can hold

// Rows of `width` elements, `pitch` elements apart.
struct Rows {
    const void *p;
    int64_t rows, pitch, width;
    int es;

    bool ok() const
    {
        return p && reinterpret_cast<uintptr_t>(p) % es == 0 &&
               (rows <= 1 || (pitch >= width && pitch <= kMaxPitch && pitch <= kMaxSpan / rows)) && width <= kMaxSpan;
    }
    uintptr_t lo() const { return reinterpret_cast<uintptr_t>(p); }
    uintptr_t hi() const { return lo() + static_cast<uintptr_t>(((rows - 1) * pitch + width) * es); }
    bool aligned(int bytes) const { return lo() % bytes == 0 && (rows <= 1 || pitch * es % bytes == 0); }
    bool none() const { return !p || rows <= 0 || width <= 0; }
};

Rows flat(const void *p, int64_t n, int es) { return {p, 1, n, n, es}; }

// May some element of a be an element of b?  Exact where both have the same pitch
// (column blocks of the same rows); else by extent.
bool meet(const Rows &a, const Rows &b)
{
    if (a.none() || b.none() || a.hi() <= b.lo() || b.hi() <= a.lo())
        return false;
    if (a.rows <= 1 || b.rows <= 1 || a.pitch != b.pitch || a.es != b.es)
        return true;
    const uintptr_t pitch = static_cast<uintptr_t>(a.pitch) * a.es;
    const uintptr_t d = b.lo() >= a.lo() ? (b.lo() - a.lo()) % pitch : (pitch - (a.lo() - b.lo()) % pitch) % pitch;
    return !(d >= static_cast<uintptr_t>(a.width) * a.es && d + static_cast<uintptr_t>(b.width) * b.es <= pitch);
}

// `a` may also be `b` itself, element for element.
bool meet_unless_same(const Rows &a, const Rows &b)
{
    return !(a.p == b.p && (a.rows <= 1 || a.pitch == b.pitch)) && meet(a, b);
}

// 3-D map of 16-bit elements over [groups][rows][inner], box 64 x `box` x 1, 128-byte
// swizzle, out-of-range reads give 0.
int encode_groups(const mbert_attn *h, CUtensorMap *tm, const void *p, int64_t inner, int64_t rows, int64_t groups,
                  int64_t pitch, int64_t group_pitch, int box)
{
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(rows),
                                static_cast<cuuint64_t>(groups)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(pitch) * 2, static_cast<cuuint64_t>(group_pitch) * 2};
    const cuuint32_t boxes[3] = {64, static_cast<cuuint32_t>(box), 1};
    const cuuint32_t ones[3] = {1, 1, 1};
    const CUresult r = h->encode(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(p), dims, strides, boxes,
                                 ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                 CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? MBERT_OK : MBERT_ERR_CUDA;
}

// 2-D map of 16-bit elements over [rows][width] for the staging buffers of linear.cu:
// box 64 x 32 with the 128-byte swizzle or 32 x 32 with the 64-byte one.
int encode_chunks(const mbert_attn *h, CUtensorMap *tm, const void *p, int64_t width, int64_t rows, int64_t pitch,
                  int chunk)
{
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(width), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(pitch) * 2};
    const cuuint32_t boxes[2] = {static_cast<cuuint32_t>(chunk), 32};
    const cuuint32_t ones[2] = {1, 1};
    const CUresult r = h->encode(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(p), dims, strides, boxes,
                                 ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                                 chunk == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                                 CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? MBERT_OK : MBERT_ERR_CUDA;
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Blocks of `rows` rows over all groups, at most.
int64_t block_bound(const mbert_attn_linear_args &c, int rows)
{
    if (c.experts == 0)
        return ceil_div(c.rows, rows);
    return std::min<int64_t>(c.rows, c.rows / rows + c.experts);
}

// What a product takes, in clocks of an SM: estimates from measured calls (a few rows to
// 2048 by 768 to 8192, 8 to 64 experts), good for the choice between kernels and
// tiles and no more: over the first 120 products that perf/more_operators.py draws from
// random.Random(2026) the chosen form took 6 % longer than the best of both widths of unit
// and four tiles in the geometric mean, 1.56 times as long at worst (88 x 1128 -> 32, 10.9 us
// against 7), and as much for even groups as for ragged ones.  (Kernel for few rows against that for many, us: 128 x 4096 -> 512 9.2 / 19.0, 300 x
// 768 -> 2304 8.9 / 9.7, 1024 x 1024 -> 8192 26.8 / 20.5; 500 rows of 16 experts, 768 -> 2304,
// 15.8 / 26.3, 2000 rows of 16, 1024 -> 8192, 65 / 70; tiles of 64 against 128 rows, 500 rows of
// 16 experts, 4096 -> 2 x 512, 48 / 32.)
struct Cost {
    double clocks;
    LinearPlan plan;
};

// Does the activation go without exponentials?
bool plain(const mbert_attn_linear_args &c)
{
    return c.activation == MBERT_ACT_NONE || c.activation == MBERT_ACT_RELU;
}

// The row tiles that groups of about the same size make.
int64_t tile_estimate(const mbert_attn_linear_args &c, int rows)
{
    if (c.experts == 0)
        return ceil_div(c.rows, rows);
    const int64_t groups = std::min<int64_t>(c.experts, c.rows);
    return std::max(groups, c.rows / rows + groups / 2);
}

// The kernel for few rows with tiles of `tile`, its best pieces and split: a step takes
// what its bytes take at 60 a clock, its MMAs (which read 4 KB of weights and the rows
// each), or what a warp needs from step to step, 330; 32 rows of an epilogue 1300, 2300 with
// exponentials; a cluster's exchange of sums 2000 and its bytes at 8 a clock.
Cost rows_cost(const mbert_attn *h, const mbert_attn_linear_args &c, int tile)
{
    Cost best{1e300, {}};
    const bool gated = c.gated;
    const int64_t bound = block_bound(c, tile), tiles = tile_estimate(c, tile);
    const int64_t granules = ceil_div(c.outer, kLinearGranule), steps = ceil_div(c.inner, 64);
    const int64_t places = static_cast<int64_t>(h->num_sms) * linear_rows_ctas(tile, gated);
    const double sides = gated ? 2 : 1, mma = 4 * sides * (32 + tile / 4.0);
    const double epilogue = (plain(c) ? 1300.0 : 2300.0) * (gated ? 1.3 : 1.0) * ceil_div(tile, 32);
    // every row tile reads its group's weights, from memory or from L2, at 2850 a clock
    const double traffic = static_cast<double>(tiles) * c.outer * sides * c.inner * 2 / 2850;
    auto consider = [&](int m, int split) {
        const int64_t pieces = ceil_div(granules, m), ctas = split > 1 ? bound * pieces : std::min(places, bound * pieces);
        // clusters fit where their SMs lie together, which leaves some idle
        if (split > 1 && (10 * ctas * split > 8 * places || linear_rows_stages(tile, gated, m, split) < 3))
            return;
        const int64_t runs = split > 1 ? 1 : ceil_div(tiles * pieces, ctas);     // pieces of a CTA
        const int64_t share = std::max<int64_t>(1, ceil_div(std::min(ctas, tiles * pieces) * split, h->num_sms));
        const double step = std::max(330.0, share * std::max(mma, (tile * 128 + sides * m * 4096) / 60.0));
        const double work = runs * std::max(ceil_div(steps, split) * step, epilogue) + epilogue;
        const double clocks = 9500 + std::max(traffic, work) + 0.3 * std::min(traffic, work) +
                              (split > 1 ? 2000 + linear_rows_parts(tile, gated, m, split) / 8.0 : 0.0);
        if (clocks < best.clocks) {
            best.clocks = clocks;
            best.plan.few = true;
            best.plan.rows = {tile, m, split, ctas};
            best.plan.units = bound * granules;
        }
    };
    for (int m = 1; m <= kLinearGranules; ++m)
        for (int split = 1; split <= 8 && split <= steps; split *= 2)
            consider(m, split);
    return best;
}

// The kernel for many rows: a step of 256 x 256 takes 600 clocks, one of 256 x 128 450; an
// epilogue 5000 (gated 3700, for half the columns), an activation that computes
// exponentials 3700 (2100) more, ragged groups 1000; 256 x 128 a little over half of it.
Cost pair_cost(const mbert_attn *h, const mbert_attn_linear_args &c, int columns)
{
    Cost p{};
    const int64_t across = ceil_div(c.outer, c.gated ? columns / 2 : columns);
    const int64_t waves = ceil_div(tile_estimate(c, kLinearRows) * across, h->num_sms / 2);
    const double epilogue = (columns == 256 ? 1.0 : 0.56) *
        ((c.gated ? 3700 : 5000) + (plain(c) ? 0 : c.gated ? 2100 : 3700) + (c.experts > 0 ? 1000 : 0));
    // weights that few rows meet come at 1750 a clock
    const double fetch = static_cast<double>(std::max<int64_t>(1, std::min<int64_t>(c.experts, c.rows))) * c.outer *
                         (c.gated ? 2 : 1) * c.inner * 2 / 1750;
    p.clocks = 9900 + std::max(fetch, waves * std::max<double>(ceil_div(c.inner, 64) * (columns == 256 ? 600 : 450), epilogue)) +
               epilogue;
    p.plan.columns = columns;
    p.plan.units = block_bound(c, kLinearRows) * across;
    return p;
}

LinearPlan make_plan(const mbert_attn *h, const mbert_attn_linear_args &c)
{
    Cost best = pair_cost(h, c, 256);
    auto consider = [&](const Cost &o) {
        if (o.clocks < best.clocks)
            best = o;
    };
    consider(pair_cost(h, c, 128));
    const int64_t mean = ceil_div(c.rows, std::max(c.experts, 1));
    if (mean <= 2048) {
        // tiles that a group of the mean size fills, smaller and larger ones
        int tile = 16;
        while (tile < 128 && tile < mean)
            tile *= 2;
        consider(rows_cost(h, c, tile));
        if (tile < 128)
            consider(rows_cost(h, c, 2 * tile));
        if (tile > 16)
            consider(rows_cost(h, c, tile / 2));
    }
    return best.plan;
}

// The plan of a call; that of one like an earlier one is found again (weighing takes
// microseconds, as long as a short kernel).  Under a lock: a plan that two threads had
// written together would be none.
LinearPlan linear_plan(mbert_attn *h, const mbert_attn_linear_args &c)
{
    const int64_t key[4] = {c.rows, static_cast<int64_t>(c.inner) << 32 | c.outer, c.experts,
                            c.activation * 2 + c.gated};
    uint64_t x = 0;
    for (const int64_t k : key)
        x = (x ^ static_cast<uint64_t>(k)) * 0x9E3779B97F4A7C15ull;
    const std::lock_guard<std::mutex> lock(h->plan_lock);
    mbert::PlanEntry &e = h->plans[x >> 58];
    if (!e.known || std::memcmp(e.key, key, sizeof key) != 0) {
        e.plan = make_plan(h, c);
        std::memcpy(e.key, key, sizeof key);
        e.known = true;
    }
    return e.plan;
}

bool sizes_ok(const mbert_attn_linear_args &c)
{
    return c.rows >= 0 && c.rows <= kMaxRows && c.inner >= 1 && c.inner <= kMaxWidth && c.outer >= 1 && c.outer <= kMaxWidth &&
           c.activation >= MBERT_ACT_NONE && c.activation <= MBERT_ACT_RELU && (c.gated == 0 || c.gated == 1) &&
           c.experts >= 0 && c.experts <= 65536;
}

}  // namespace

MBERT_API int mbert_attn_linear_plan(mbert_attn *h, const mbert_attn_linear_args *args, int32_t plan[4])
{
    if (!h || !args || !plan || !sizes_ok(*args) || args->rows == 0)
        return MBERT_ERR_BAD_ARG;
    const LinearPlan p = linear_plan(h, *args);
    plan[0] = p.few;
    plan[1] = p.few ? p.rows.tile : p.columns;
    plan[2] = p.few ? p.rows.granules : 0;
    plan[3] = p.few ? p.rows.split : 0;
    return MBERT_OK;
}

MBERT_API int mbert_attn_linear(mbert_attn *h, const mbert_attn_linear_args *args, void *stream)
{
    if (!h || !args)
        return MBERT_ERR_BAD_ARG;
    const mbert_attn_linear_args &c = *args;
    if (c.dtype != MBERT_BF16 && c.dtype != MBERT_F16)
        return MBERT_ERR_UNSUPPORTED;
    if (!sizes_ok(c))
        return MBERT_ERR_BAD_ARG;
    // the router's weights go with experts, a residual with the plain product
    if (c.experts > 0 ? c.residual != nullptr : c.cu_experts || c.row_scale)
        return MBERT_ERR_BAD_ARG;
    if (c.rows == 0)
        return MBERT_OK;
    if (c.experts > 0 && (!c.cu_experts || reinterpret_cast<uintptr_t>(c.cu_experts) % 4))
        return MBERT_ERR_BAD_ARG;
    const int64_t groups = std::max(c.experts, 1), width = static_cast<int64_t>(c.gated ? 2 : 1) * c.outer;
    const Rows x{c.x, c.rows, c.x_row, c.inner, 2}, out{c.out, c.rows, c.out_row, c.outer, 2};
    const Rows weight{c.weight, width, c.weight_row, c.inner, 2};
    const Rows residual{c.residual, c.rows, c.residual_row, c.outer, 2};
    if (!x.ok() || !out.ok() || !weight.ok() || (c.residual && !residual.ok()))
        return MBERT_ERR_BAD_ARG;
    // what TMA can fetch: 16-byte aligned rows
    const int64_t matrix = (width - 1) * c.weight_row + c.inner;
    if (!x.aligned(16) || !weight.aligned(16) ||
        (groups > 1 && (c.weight_expert < matrix || c.weight_expert % 8 || c.weight_expert > kMaxPitch ||
                        c.weight_expert > kMaxSpan / groups)))
        return MBERT_ERR_BAD_ARG;
    const Rows bias = flat(c.bias, groups * width, 2), scale = flat(c.row_scale, c.rows, 4);
    const Rows weights = flat(c.weight, (groups - 1) * c.weight_expert + matrix, 2);
    const Rows cu = flat(c.cu_experts, groups + 1, 4);
    if ((c.bias && !bias.ok()) || (c.row_scale && !scale.ok()) || meet(out, x) || meet(out, weights) ||
        meet(out, bias) || meet(out, scale) || meet(out, cu) || meet_unless_same(out, residual))
        return MBERT_ERR_BAD_ARG;

    const LinearPlan p = linear_plan(h, c);
    if (p.units > INT32_MAX / 4)
        return MBERT_ERR_BAD_ARG;       // (more than any device holds)
    DeviceGuard g(h->device);
    LinearArgs a;
    // a dimension of one element has no stride that matters; a map wants one all the same
    auto pitch = [](int64_t rows, int64_t given, int64_t w) { return rows > 1 ? given : (w + 7) / 8 * 8; };
    const int64_t wrow = pitch(width, c.weight_row, c.inner);
    const int xbox = p.few ? p.rows.tile : kLinearRows / 2, wbox = p.few ? kLinearGranule * p.rows.granules : p.columns / 2;
    if (encode_rows(h, &a.tm_x, c.x, c.inner, c.rows, pitch(c.rows, c.x_row, c.inner), xbox, 256) != MBERT_OK ||
        encode_groups(h, &a.tm_w, c.weight, c.inner, width, groups, wrow, groups > 1 ? c.weight_expert : width * wrow,
                      wbox) != MBERT_OK)
        return MBERT_ERR_CUDA;
    a.out_vectors = out.aligned(16);
    a.out_bytes = out.aligned(8) ? 8 : out.aligned(4) ? 4 : 2;
    a.residual_bytes = residual.aligned(8) ? 8 : residual.aligned(4) ? 4 : 2;
    a.residual_vectors = c.residual && residual.aligned(16);
    const int chunk = linear_chunk(c.gated);
    if ((a.out_vectors && !p.few && encode_chunks(h, &a.tm_out, c.out, c.outer, c.rows, pitch(c.rows, c.out_row, c.outer), chunk) !=
                          MBERT_OK) ||
        (a.residual_vectors && !p.few && encode_chunks(h, &a.tm_residual, c.residual, c.outer, c.rows,
                                         pitch(c.rows, c.residual_row, c.outer), chunk) != MBERT_OK))
        return MBERT_ERR_CUDA;
    a.bias = c.bias;
    a.residual = c.residual;
    a.row_scale = c.row_scale;
    a.out = c.out;
    a.residual_row = c.residual_row;
    a.out_row = c.out_row;
    a.cu = c.cu_experts;
    a.groups = static_cast<int>(groups);
    a.rows = c.rows;
    a.inner = c.inner;
    a.outer = c.outer;
    a.activation = c.activation;
    a.err = h->err;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool half = c.dtype == MBERT_F16;
    const cudaError_t e = p.few ? launch_linear_rows(a, p.rows, c.gated, half, st)
                                : launch_linear(a, p.columns, c.gated, half, p.units, h->num_sms, st);
    h->launches += 1;
    return e == cudaSuccess ? MBERT_OK : MBERT_ERR_CUDA;
}

MBERT_API int mbert_attn_residual_norm(mbert_attn *h, const mbert_attn_residual_norm_args *args, void *stream)
{
    if (!h || !args)
        return MBERT_ERR_BAD_ARG;
    const mbert_attn_residual_norm_args &c = *args;
    if (c.dtype < MBERT_BF16 || c.dtype > MBERT_F32 || c.rows < 0 || c.rows > kMaxRows || c.width < 1 ||
        c.width > kResidualNormMaxWidth || (c.norm != MBERT_NORM_RMS && c.norm != MBERT_NORM_LAYER) ||
        !(c.eps >= 0.f) || c.eps > 1.f || !std::isfinite(c.residual_scale))
        return MBERT_ERR_BAD_ARG;
    // a norm's bias with its weight; without a branch nothing is scaled or gated, and
    // the call is y's norm alone
    if ((c.bias && !c.weight) || (c.branch_bias && !c.branch_weight) || (c.cu_seqlens && !c.gate) ||
        (!c.branch && (c.branch_weight || c.gate || c.h || c.residual_scale != 1.f || !c.weight)) ||
        c.gate_kind < MBERT_GATE_NONE || c.gate_kind > MBERT_GATE_SEQUENCES ||
        (c.gate != nullptr) != (c.gate_kind != MBERT_GATE_NONE) ||
        (c.cu_seqlens != nullptr) != (c.gate_kind == MBERT_GATE_SEQUENCES) || (c.cu_seqlens && (c.n_seqs < 1 || c.n_seqs > kMaxRows)) ||
        reinterpret_cast<uintptr_t>(c.cu_seqlens) % 4)
        return MBERT_ERR_BAD_ARG;
    if (c.rows == 0)
        return MBERT_OK;
    const int es = c.dtype == MBERT_F32 ? 4 : 2;
    const int64_t gates = c.gate_kind == MBERT_GATE_ROWS ? c.rows : c.gate_kind == MBERT_GATE_SEQUENCES ? c.n_seqs : 1;
    const Rows x{c.x, c.rows, c.x_row, c.width, es}, branch{c.branch, c.rows, c.branch_row, c.width, es};
    const Rows gate{c.gate, gates, c.gate_row, c.width, es};
    const Rows hr{c.h, c.rows, c.h_row, c.width, es}, y{c.y, c.rows, c.y_row, c.width, es};
    if (!x.ok() || (c.branch && (!branch.ok() || !hr.ok())) || (c.gate && !gate.ok()) || (c.weight && !y.ok()))
        return MBERT_ERR_BAD_ARG;
    const Rows cu = flat(c.cu_seqlens, static_cast<int64_t>(c.n_seqs) + 1, 4);
    const void *const params[4] = {c.weight, c.bias, c.branch_weight, c.branch_bias};
    bool vectors = c.width * es % 16 == 0;
    for (const Rows *r : {&x, &branch, &gate, &hr, &y})
        vectors = vectors && (r->none() || r->aligned(16));
    for (const void *p : params) {
        const Rows r = flat(p, c.width, es);
        if (p && (!r.ok() || (c.branch && meet(hr, r)) || (c.weight && meet(y, r))))
            return MBERT_ERR_BAD_ARG;
        vectors = vectors && reinterpret_cast<uintptr_t>(p) % 16 == 0;
    }
    // h may be x or the branch, and so may y; no two results share elements
    for (const Rows *r : {&hr, &y}) {
        if (r == &hr ? !c.branch : !c.weight)
            continue;
        if (meet_unless_same(*r, x) || meet_unless_same(*r, branch) || meet(*r, gate) || meet(*r, cu))
            return MBERT_ERR_BAD_ARG;
    }
    if (c.branch && c.weight && meet(hr, y))
        return MBERT_ERR_BAD_ARG;

    ResidualNormArgs a;
    a.x = c.x;
    a.branch = c.branch;
    a.gate = c.gate;
    a.weight = c.weight;
    a.bias = c.bias;
    a.after_weight = c.branch_weight;
    a.after_bias = c.branch_bias;
    a.h = c.h;
    a.y = c.y;
    a.x_row = c.x_row;
    a.branch_row = c.branch_row;
    a.gate_row = c.gate_row;
    a.gate_channels = c.gate_kind == MBERT_GATE_CHANNELS;
    a.h_row = c.h_row;
    a.y_row = c.y_row;
    a.cu = c.cu_seqlens;
    a.n_seqs = c.n_seqs;
    a.rows = c.rows;
    a.width = c.width;
    a.vectors = vectors;
    a.residual_scale = c.residual_scale;
    a.eps = c.eps;
    int k = 0;
    while ((1 << k) < c.width)
        ++k;
    a.sum_scale = std::ldexp(1.f, -k);
    a.half_mean_scale = static_cast<float>(std::ldexp(0.5, k) / c.width);
    a.inv_width = static_cast<float>(1.0 / c.width);
    a.least_squares = c.eps >= 0x1p-40f ? 0.f : 0x1p-90f;
    a.most_scale = c.eps > 0.f ? std::min(126, (100 - std::ilogb(c.eps)) / 2) : 126;
    a.err = h->err;
    DeviceGuard g(h->device);
    const cudaError_t e = launch_residual_norm(a, c.dtype, c.norm == MBERT_NORM_LAYER, h->num_sms,
                                               static_cast<cudaStream_t>(stream));
    h->launches += 1;
    return e == cudaSuccess ? MBERT_OK : MBERT_ERR_CUDA;
}
