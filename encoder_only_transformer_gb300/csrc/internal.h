// Launch interface between the host library (host.cu) and the kernel
// translation units.  Not part of the public C ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <stdint.h>

#include <atomic>
#include <mutex>

namespace mbert {

constexpr int kMaxDevices = 64;

// Per-device set-up of one kernel that must happen once in each device
// context before its first launch there (a shared-memory opt-in, an
// occupancy query).  Safe to use from several host threads: the first
// caller on a device runs the set-up under the lock, later callers read the
// published value without locking.
struct PerDeviceOnce {
    std::mutex mu;
    std::atomic<int> value[kMaxDevices] = {};   // 0: not set up yet
};

// Returns in *value the set-up result for the current device (a positive
// int), running `setup(&v)` on the first call there.
template <typename Setup>
cudaError_t per_device_once(PerDeviceOnce &once, int *value, Setup setup)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev < 0 || dev >= kMaxDevices)
        return cudaErrorInvalidDevice;
    int v = once.value[dev].load(std::memory_order_acquire);
    if (v == 0) {
        std::lock_guard<std::mutex> lock(once.mu);
        v = once.value[dev].load(std::memory_order_relaxed);
        if (v == 0) {
            e = setup(&v);
            if (e != cudaSuccess)
                return e;
            once.value[dev].store(v, std::memory_order_release);
        }
    }
    *value = v;
    return cudaSuccess;
}

// Raise `kernel`'s dynamic shared-memory limit to `bytes` on the current
// device (once per device).
template <typename Kernel>
cudaError_t smem_opt_in(PerDeviceOnce &once, Kernel kernel, size_t bytes)
{
    int v = 0;
    return per_device_once(once, &v, [&](int *out) {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(bytes));
        *out = 1;
        return e;
    });
}

// Launch `kernel` on `stream` with programmatic stream serialization: its
// launch may overlap the tail of the previous kernel in the stream, which
// it waits for in-kernel (pdl_wait) before touching memory.
template <typename... KArgs, typename... Args>
cudaError_t launch_chained(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                           cudaStream_t stream, Args &&...args)
{
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

constexpr int kPairsConst = 32;

// Work list written by the plan kernel: one entry per (sequence, 128-query
// block), longest sequences first; the attention grid covers entries x heads.
struct Plan {
    int block = 128;        // query rows per work entry (128 or 256)
    const int32_t *cu;      // device [n_seqs + 1]
    int n_seqs;
    int64_t T;
    int max_seqlen;         // longest sequence accepted by the device check
    int2 *work;             // device [entry_bound]
    int32_t *work_count;    // device scalar: entries written (0 if the checks failed)
    int entry_bound;        // host-side upper bound on the entry count
    int32_t *err;           // device error word (sticky, bit mask)
    bool cu_short_ok = false;   // accept cu[n] <= T: rows past cu[n] belong to no sequence
    // Optional (global layers): tile_start[e] = sum over entries before e of
    // heads * ceil(L/128) (the entry's first iteration in the split of all
    // (entry, head, key tile) iterations among persistent CTAs), with
    // tile_start[count] = the total; unit_cnt[entry * heads + head] zeroed.
    int32_t *tile_start = nullptr;   // device [entry_bound + 1]
    int32_t *unit_cnt = nullptr;     // device [entry_bound * heads]
};

cudaError_t launch_plan(const Plan &p, cudaStream_t stream);

// The plan and, in the same launch, the RoPE of Q and K of every row (all
// heads) into rot[T][1536] bf16.  With norms set (global layers), also the
// Euclidean norm of every rotated row and head: Q head h in norms[h][row]
// (fp32), K head h in knorm[h][row] (fp16 bits, rounded up), rows
// `norm_pitch` apart (a multiple of 8).
cudaError_t launch_plan_rope(const Plan &p, const __nv_bfloat16 *qkv, const float2 *table,
                             int table_rows, __nv_bfloat16 *rot, float *norms, uint16_t *knorm,
                             long long norm_pitch, cudaStream_t stream);

// Admitted-key count per query row, from the attention kernels' tile
// schedule and mask.
cudaError_t launch_key_count(const Plan &p, int half_window, int32_t *counts,
                             cudaStream_t stream);

struct AttnArgs {
    CUtensorMap tm_rot;     // rotated Q/K [T][1536], box 64 x 128, 128B swizzle
    CUtensorMap tm_qkv;     // qkv [T][2304], box 64 x 128, 128B swizzle
    const int32_t *cu;
    const int2 *work;
    const int32_t *work_count;
    int entry_bound;
    int half_window;        // < 0: global layer
    __nv_bfloat16 *out;     // [T][768]
    int32_t *err;
    // global layers: persistent CTAs and the split of iterations
    int num_ctas = 0;
    const int32_t *tile_start = nullptr;
    int32_t *unit_cnt = nullptr;
    float *partials = nullptr;   // [2 * num_ctas][kPartialFloats]
    const float *norms = nullptr;     // [12][norm_pitch]: rotated Q row norms per head
    const uint16_t *knorm = nullptr;  // [12][norm_pitch]: rotated K row norms, fp16 rounded up
    long long norm_pitch = 0;         // a multiple of 8
    long long rows = 0;               // rows of qkv
};

// One partial state of a query block split across CTAs: O (unnormalised,
// fp32) for 256 rows x 64, then (m, l) for the 256 rows.
constexpr int kPartialRows = 256;
constexpr int kPartialFloats = kPartialRows * 64 + kPartialRows * 2;

// RoPE constants for computing cos/sin in the local kernel: for pair m the
// frequency in turns per position as a 64-bit binary fraction (frac_hi holds
// 2^-1 .. 2^-32, frac_lo 2^-33 .. 2^-64), so that the turns of any position
// are exact modulo 1 in integer arithmetic, and the rotation by 128
// positions (cos, sin of 128 w, fp64 values rounded to fp32).
struct RopeConsts {
    uint32_t frac_hi[kPairsConst];
    uint32_t frac_lo[kPairsConst];
    float cos128[kPairsConst];
    float sin128[kPairsConst];
};

struct LocalArgs {
    RopeConsts rope;
    CUtensorMap tm_qkv;          // qkv [T][2304], box 64 x 128, 128B swizzle
    CUtensorMap tm_out;          // out [T][768], box 64 x 128, 128B swizzle
    const int32_t *cu;
    int n_seqs;
    long long T;
    int max_seqlen;
    const int2 *work;            // null: each CTA finds its block from cu_seqlens
    const int32_t *work_count;
    int half_window;             // <= kBandReach
    int block_bound;             // upper bound on 128-query blocks over all sequences
    int num_ctas;                // persistent CTAs (one per SM)
    __nv_bfloat16 *out;
    int32_t *err;
};

// Local-layer attention with RoPE in the prologue: persistent CTAs, each
// walking a contiguous range of (128-query block, head) units, two band
// tiles of keys per unit.
cudaError_t launch_attn_local(const LocalArgs &a, cudaStream_t stream);

// Output projection with the residual add, y = x + a Wo^T: persistent pairs
// of CTAs over 256 x 256 output blocks.
struct OutProjArgs {
    CUtensorMap tm_a;            // a  [T][768], box 64 x 128, 128B swizzle
    CUtensorMap tm_w;            // Wo [768][768] ([out][in]), box 64 x 128, 128B swizzle
    CUtensorMap tm_x;            // x  [T][768], box 64 x 128, 128B swizzle
    CUtensorMap tm_y;            // y  [T][768] (may be x), box 64 x 128, 128B swizzle
    const __nv_bfloat16 *x;      // x itself, for L2 prefetches
    long long T;
    int num_ctas;                // SMs: the launch sizes its pairs by occupancy
    int32_t *err;
};

cudaError_t launch_out_proj(const OutProjArgs &a, cudaStream_t stream);

// The fused Wqkv projection, qkv = h Wqkv^T: the same paired GEMM over
// 256 x 256 output blocks, 2304 output columns, no residual.
struct QkvProjArgs {
    CUtensorMap tm_a;            // h    [T][768], box 64 x 128, 128B swizzle
    CUtensorMap tm_w;            // Wqkv [2304][768] ([out][in]), box 64 x 128, 128B swizzle
    CUtensorMap tm_y;            // qkv  [T][2304], box 64 x 128, 128B swizzle
    long long T;
    int num_ctas;
    int32_t *err;
};

cudaError_t launch_qkv_proj(const QkvProjArgs &a, cudaStream_t stream);

// The GeGLU MLP's two GEMMs, on the same paired body: m = GELU(g) * u from
// h [T][768] and Wi [2304][768] into m [T][1152] (tm_a over h with width
// 768, tm_w over Wi, tm_y over m), then y = x + m Wo^T with Wo [768][1152]
// (tm_a over m and tm_w over Wo, both width 1152).
cudaError_t launch_mlp_up(const QkvProjArgs &a, cudaStream_t stream);
cudaError_t launch_mlp_down(const OutProjArgs &a, cudaStream_t stream);

// Bias-free LayerNorm of each row of x [T][768] (bf16) with weight w [768]
// into h [T][768] (bf16): one warp per row, fp32 statistics.
cudaError_t launch_layernorm(const __nv_bfloat16 *x, const __nv_bfloat16 *w, long long T,
                             float eps, __nv_bfloat16 *h, int num_sms, cudaStream_t stream);

// The padded-batch form [B][S] with a 0/1 attention mask, to and from the
// packed form: mask_scan writes, per row b, each real token's rank among the
// row's real tokens (-1 for a pad) and the row's count, then the exclusive
// prefix sum of the counts as cu_seqlens[0..B]; gather copies every real
// token's qkv row to packed row cu[b] + rank; scatter writes every padded
// row of out from its packed row, zeros for pads.
cudaError_t launch_mask_scan(const int32_t *mask, int B, int S, int32_t *rank, int32_t *len,
                             int32_t *cu, cudaStream_t stream);
cudaError_t launch_gather_rows(const __nv_bfloat16 *src, const int32_t *rank, const int32_t *cu,
                               int B, int S, int width, __nv_bfloat16 *dst, int num_sms,
                               cudaStream_t stream);
cudaError_t launch_scatter_rows(const __nv_bfloat16 *src, const int32_t *rank, const int32_t *cu,
                                int B, int S, int width, __nv_bfloat16 *dst, int num_sms,
                                cudaStream_t stream);

// Rotary positions on rows of heads, alone or after a norm of every head
// (rotary.cu): up to two tensors (queries and keys) of the same rows.
struct RotaryRows {
    const void *src = nullptr;
    void *dst = nullptr;             // may be src
    const void *weight = nullptr;    // [dim], with a norm
    int heads = 0;                   // 0: no such tensor
    long long src_row = 0, src_head = 0, dst_row = 0, dst_head = 0;   // strides in elements
};

constexpr int kMaxRotaryPairs = 128;

struct RotaryArgs {
    RotaryRows x[2];
    int dtype = 0;                   // MBERT_BF16, MBERT_F16 or MBERT_F32
    int dim = 0, rot = 0;            // head size, turned part (both even)
    int interleaved = 0;
    int norm = 0;                    // MBERT_NORM_*
    float eps = 0.f;
    // a head's squares add up to one of the `squares` floats from the one with these
    // bits on, or it is scaled first, by most_scale at most
    uint32_t least_squares = 0, squares = 0;
    float most_scale = 1.f;
    float amplitude = 1.f, sin_amplitude = 1.f;   // sin_amplitude < 0: the inverse rotation
    long long tokens = 0;
    // positions: 32 or 64 bits per row, or from cu_seqlens; none for rot = 0
    const int32_t *pos32 = nullptr;
    const int64_t *pos64 = nullptr;
    const int32_t *cu = nullptr;
    int n_seqs = 0;
    int32_t *err = nullptr;
    // set by the launcher: lanes of a head; a block's heads, rows, and the
    // rows it takes side by side
    int lanes_log2 = 0, block_heads = 1, block_rows = 1, teams = 1, table_offset = 0;
    uint64_t turns[kMaxRotaryPairs] = {};   // turns per position, 64-bit binary fractions
};

cudaError_t launch_rotary(RotaryArgs &a, int num_sms, cudaStream_t stream);

// Cross attention: packed queries over keys and values of another length
// (attn_cross.cu: blocks of queries; attn_cross_token.cu: few rows a
// sequence; cross_join.cu: what goes before and after).
struct CrossArgs {
    CUtensorMap tm_q;                   // [rows][heads][D], box 64 columns x 2^fold_log2 heads (blocks)
    CUtensorMap tm_k, tm_v;             // [rows][heads * D], box 64 columns
    const void *q = nullptr;
    void *out = nullptr;
    long long q_row = 0, out_row = 0;   // row strides in elements
    const int32_t *cu_q = nullptr, *cu_k = nullptr;   // null: sequences of len_q / len_k rows
    int n_seqs = 0, len_q = 0, len_k = 0;
    long long rows_q = 0, rows_k = 0;
    int max_q = 0;                      // longest query sequence accepted
    int heads = 0, group = 1;           // query heads, query heads per key head
    int fold_log2 = 0;                  // query heads that share a block's rows (blocks)
    float scale_log2 = 0.f;             // softmax scale in base 2
    // with a key mask: per sequence the visible keys as bits (sequence s from
    // word key_bit_word(s) on), the place after the last visible one, and the
    // number of visible keys before the first hidden one
    const uint32_t *key_bits = nullptr;
    const int2 *key_len = nullptr;
    int32_t *err = nullptr;
    // units cut between CTAs: a record and two part slots per CTA (null where
    // no sequence can be long enough)
    struct CrossRecord *records = nullptr;
    float *parts = nullptr;
};

// What the joining kernel needs of a unit whose first part CTA c holds.
struct CrossRecord {
    long long row0;     // first query row
    int rows;           // rows of the unit (row r: query row0 + r / group, head head0 + r % group)
    int head0, group;
    int parts;          // 0: CTA c holds no first part
};

// Rows of a unit of attn_cross.cu: two query tiles, or one in calls whose
// sequences have no more (both measured there).
constexpr int kCrossBlockRows = 256;
constexpr int kCrossSmallRows = 128;
// For head size 128 only up to this many keys a sequence, in the mean: its CTAs
// have half the bytes in flight.  One query tile against two, us: 24 sequences of 32,
// 32 heads over 8: 800 keys 26.6 / 33.1, 1500 38.9 / 42.2, 2000 52.9 / 49.9, 3000 72.6 /
// 69.1; 100 of 100, 8 heads: 1200 94 / 106, 1600 116 / 128, 2000 156 / 153; 40 of 16, 16
// over 2: 1600 25.9 / 27.0, 2000 29.4 / 29.4.
constexpr int kCrossSmallKeys = 1536;
// Keys of a tile of its K and V: 64 where two CTAs of head size 128 share an SM.
constexpr int cross_tile_keys(int dim, int unit_rows) { return dim == 128 && unit_rows == kCrossSmallRows ? 64 : 128; }
constexpr int kCrossTokenRows = 16;     // rows of a unit of attn_cross_token.cu

// Units of at most this many keys are not cut between CTAs (blocks of queries,
// single tokens): up to there joining parts costs more than it evens out
// (ragged blocks over 300 to 700 keys 24.8 us against 27.6 with 512; tokens over
// four times 1000 keys 10.3 us against 15.0 with 1024).
constexpr int kCrossBlockWholeKeys = 256;
constexpr int kCrossTokenWholeKeys = 512;
// In a call whose sequences can have no more keys than this none is cut, which
// saves the joining kernel and the workspace (tokens over four times 200 keys 6.7 us
// against 9.7).
constexpr int kCrossBlockWholeRows = 512;
constexpr int kCrossTokenWholeRows = 1024;

// First word of sequence s's key bits: every sequence starts a new word.
__host__ __device__ inline long long key_bit_word(long long k_row, int s) { return k_row / 32 + s; }

constexpr long long cross_slot_floats(int rows, int dim) { return static_cast<long long>(rows) * (dim + 2); }

// CTAs of the token kernel on one SM (by shared memory and registers).
constexpr int cross_token_ctas(int dim) { return dim == 64 ? 3 : 2; }

// CTAs of the kernel for blocks of queries on one SM.
constexpr int cross_block_ctas(int unit_rows) { return unit_rows == kCrossSmallRows ? 2 : 1; }

// key_mask [rows_k] (non-zero: visible) to bits and lengths per sequence.
cudaError_t launch_key_bits(const CrossArgs &a, const int32_t *key_mask, uint32_t *bits, int2 *len,
                            cudaStream_t stream);
cudaError_t launch_cross_blocks(const CrossArgs &a, int dim, bool half, int unit_rows, int ctas, cudaStream_t stream);
cudaError_t launch_cross_token(const CrossArgs &a, int dim, bool half, int ctas, cudaStream_t stream);
// Joins the parts of cut units; rows: those of a unit (kCrossBlockRows or
// kCrossSmallRows after the first kernel, at most kCrossTokenRows after the second).
cudaError_t launch_cross_join(const CrossArgs &a, int dim, bool half, int rows, int ctas, cudaStream_t stream);

// Number of sequences up to which the local kernel finds its blocks itself
// (above it the plan kernel writes a work list first).
constexpr int kLocalSelfScheduleMaxSeqs = 256;

// Moves the error word to *taken (device) and clears it, in one step.
cudaError_t launch_take_error(int32_t *err, int32_t *taken, cudaStream_t stream);

// One bounded mbarrier wait that nothing completes (exercises kErrTimeout).
cudaError_t launch_wait_timeout_selftest(int32_t *err, unsigned long long limit_ns,
                                         cudaStream_t stream);

// Generic flash attention over pre-rotated Q/K: one CTA per (entry, head),
// entries of 128 query rows.
cudaError_t launch_attn_generic(const AttnArgs &a, cudaStream_t stream);

// Global-layer attention over pre-rotated Q/K: one CTA per (entry, head),
// entries of 256 query rows, warp-specialised tcgen05 pipeline.
cudaError_t launch_attn_global(const AttnArgs &a, cudaStream_t stream);

}  // namespace mbert
