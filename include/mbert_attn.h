/*
 * mbert_attn: the bidirectional self-attention block of ModernBERT-base as a
 * C-ABI library for NVIDIA GB300 (sm_103a).
 *
 * What one call computes (page title, section):
 *  - Input: the fused Wqkv output, one row of 2304 bf16 numbers per token,
 *    cut as (3, 12, 64): columns 0..767 are Q, 768..1535 K, 1536..2303 V,
 *    head h at columns h*64 .. h*64+63 of each block ("ModernBERT-base
 *    Architecture Teardown", "How Does ModernBERT Make Q, K and V?";
 *    "ModernBERT" (candding), "The tensors").
 *  - RoPE, rotate-half over the full 64-wide head, on Q and K only; pair m
 *    turns by pos * base^(-2m/64); base 160000 on global layers, 10000 on
 *    local layers (teardown, "How Does RoPE Work With Two Bases?"; candding,
 *    "The two rope tables").  Positions restart at 0 in every sequence.
 *  - Scores q.k / sqrt(64), softmax along the keys, weighted blend of V, no
 *    causal mask (teardown, "How Does Self-Attention Work?").
 *  - Local layers keep key j for query i when |i - j| <= 64; global layers
 *    keep every key of the sequence (teardown, "What Are Local and Global
 *    Attention?"; candding, "The alternating attention").
 *  - Sequences are unpadded and packed back to back; cu_seqlens holds their
 *    offsets.  A query never sees keys of another sequence, which is what a
 *    padding mask achieves for a padded batch ("Encoder-only models"
 *    (rayaq), padding mask; teardown, "What Is ModernBERT-base?", unpadding).
 *  - Output: out[t, h*64 + d], 768 bf16 per token, heads in input order,
 *    ready for Wo (teardown, "How Does ModernBERT Make Q, K and V?").
 *
 * Conventions for every entry point:
 *  - Status: 0 on success, a negative MBERT_ERR_* code otherwise.  Host-side
 *    argument checks are synchronous and enqueue nothing when they fail.
 *    Checks that need device data (cu_seqlens contents) run on the GPU and
 *    are reported later by mbert_attn_get_error().
 *  - Pointers marked "device" must be CUDA device (or managed) memory on the
 *    handle's device; "host" pointers are ordinary host memory.
 *  - `stream` is a cudaStream_t passed as void* (NULL = legacy default
 *    stream).  All device work is enqueued asynchronously on it; the caller
 *    keeps ownership of the stream and of every buffer it passes.
 *  - A handle may be used from one host thread at a time.  Only
 *    mbert_attn_linear and mbert_attn_residual_norm may be called on it by any
 *    number of threads at once, and beside one thread's other calls.
 */
#ifndef MBERT_ATTN_H
#define MBERT_ATTN_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Opaque handle: owns the two RoPE cos/sin tables, the device work-list
 * workspace, the rotated-operand scratch (with the rotated rows' norms that
 * global layers use to bound their scores) and the device error word. */
typedef struct mbert_attn mbert_attn;

/* Layer kinds.  Layer i of the 22-layer stack is global iff i % 3 == 0
 * (teardown, "What Are Local and Global Attention?"). */
enum {
    MBERT_GLOBAL = 0,
    MBERT_LOCAL = 1
};

/* Status codes. */
enum {
    MBERT_OK = 0,
    MBERT_ERR_BAD_ARG = -1,        /* null/misaligned/aliased pointer, bad size or kind */
    MBERT_ERR_UNSUPPORTED = -2,    /* config other than 12 heads x 64, or no sm_103 device */
    MBERT_ERR_SEQ_TOO_LONG = -3,   /* a sequence longer than the handle's max_seqlen */
    MBERT_ERR_BAD_CU_SEQLENS = -4, /* cu_seqlens[0] != 0, decreasing, or cu[n] != T (device-detected) */
    MBERT_ERR_TIMEOUT = -5,        /* a kernel's bounded wait ran out; results are invalid */
    MBERT_ERR_CUDA = -6,           /* a CUDA runtime call failed */
    MBERT_ERR_OOM = -7             /* device allocation failed */
};

/* Create-time configuration. */
typedef struct {
    int heads;            /* must be 12 */
    int head_dim;         /* must be 64 */
    int half_window;      /* local band half-width, |i - j| <= half_window (64), 0..128 */
    int max_seqlen;       /* longest sequence accepted; sizes the RoPE tables (8192) */
    double theta_global;  /* RoPE base of global layers (160000) */
    double theta_local;   /* RoPE base of local layers (10000) */
} mbert_attn_config;

/* Fill *cfg with ModernBERT-base's values: 12, 64, 64, 8192, 160000, 10000. */
int mbert_attn_default_config(mbert_attn_config *cfg);

/* Create a handle on CUDA device `device` (host pointer out, host pointer
 * cfg; cfg == NULL means the defaults).  Allocates the RoPE tables
 * (2 x max_seqlen x 32 x (cos, sin) fp32, computed in fp64 on the host) and a
 * small workspace.  Synchronous.  On failure *out is NULL. */
int mbert_attn_create(mbert_attn **out, const mbert_attn_config *cfg, int device);

/* Grow the workspace so that later forward calls with up to `max_tokens`
 * packed tokens in up to `max_seqs` sequences allocate nothing.  Optional:
 * mbert_attn_forward grows it on demand (a synchronous cudaMalloc). */
int mbert_attn_reserve(mbert_attn *h, int64_t max_tokens, int64_t max_seqs);

/* The attention block for one layer.
 *   qkv          device, bf16 [total_tokens][2304] row-major, 16-byte aligned.
 *   cu_seqlens   device, int32 [n_seqs + 1]; cu[0] = 0, non-decreasing,
 *                cu[n_seqs] = total_tokens.  Empty sequences are allowed.
 *   n_seqs       >= 0; total_tokens >= 0 (0 enqueues nothing).
 *   max_seqlen   caller's bound on the longest sequence (<= the handle's
 *                max_seqlen, else MBERT_ERR_SEQ_TOO_LONG); a longer sequence
 *                found on the device sets MBERT_ERR_SEQ_TOO_LONG.
 *   layer_kind   MBERT_GLOBAL or MBERT_LOCAL.
 *   out          device, bf16 [total_tokens][768], 16-byte aligned, must not
 *                overlap qkv.  Every row of every sequence is written.
 * Enqueues a few kernels on `stream`; when the device-side checks fail the
 * attention kernels write nothing and the error is reported by
 * mbert_attn_get_error(). */
int mbert_attn_forward(mbert_attn *h, const void *qkv, const int32_t *cu_seqlens,
                       int n_seqs, int64_t total_tokens, int max_seqlen,
                       int layer_kind, void *out, void *stream);

/* The attention block for a padded batch: B rows of S tokens with an
 * attention mask of 1 for a real token and 0 for a pad ("ModernBERT-base
 * Architecture Teardown", the tokenizer with padding=True: the 0s of the
 * mask become a mask inside attention, so no real token takes information
 * from a pad; "Encoder-only models", "Padding and the key padding mask").
 * Each row's real tokens, in order, are one sequence: a real token's
 * position is its rank among its row's real tokens (its index for a
 * right-padded row), and only real tokens of the same row are keys.
 *   qkv             device bf16 [batch][seq_len][2304], 16-byte aligned.
 *   attention_mask  device int32 [batch][seq_len]: non-zero = real token.
 *   seq_len         <= the handle's max_seqlen (else MBERT_ERR_SEQ_TOO_LONG);
 *                   batch * seq_len < 2^31.
 *   out             device bf16 [batch][seq_len][768], 16-byte aligned, must
 *                   not overlap qkv or the mask.  Every row is written: a
 *                   real token's attention output, zeros for a pad.
 * The call packs the real rows into handle-owned buffers (grown with
 * cudaMalloc when needed), runs mbert_attn_forward's kernels on them and
 * unpacks the result, all on `stream`; calls sharing a handle must not
 * overlap on the GPU.  Returns as mbert_attn_forward. */
int mbert_attn_forward_padded(mbert_attn *h, const void *qkv, const int32_t *attention_mask,
                              int batch, int seq_len, int layer_kind, void *out, void *stream);

/* Debug/verification entry: for every packed row, the number of keys the
 * attention kernel's tile schedule and mask admit for that query (the size
 * of its admitted set), computed by the same device code the forward pass
 * uses to choose and mask key tiles.  counts: device int32 [total_tokens].
 * Other arguments as for mbert_attn_forward. */
int mbert_attn_key_counts(mbert_attn *h, const int32_t *cu_seqlens, int n_seqs,
                          int64_t total_tokens, int max_seqlen, int layer_kind,
                          int32_t *counts, void *stream);

/* The step before the attention block: its input qkv from the residual
 * stream x, qkv = LayerNorm(x) Wqkv^T.  The LayerNorm is bias-free: each
 * row minus its mean, divided by sqrt(population variance + eps), times the
 * weight ("ModernBERT-base Architecture Teardown", "What Does LayerNorm
 * Do?"); layer 0 has no norm before attention ("ModernBERT" (candding), "The
 * pre-norm layer and the final norm").  Wqkv turns 768 numbers into 2304 =
 * (3, 12, 64), Q, K, V head by head (teardown, "How Does ModernBERT Make Q,
 * K and V?"), the layout mbert_attn_forward reads.
 *   x       device bf16 [total_tokens][768], row-major.
 *   norm_w  device bf16 [768], the norm's weight; NULL for no norm
 *           (layer 0: qkv = x Wqkv^T).
 *   wqkv    device bf16 [2304][768], row-major, [out][in].
 *   eps     added to the variance under the square root (1e-5 in
 *           ModernBERT-base); 0 <= eps <= 1.
 *   qkv     device bf16 [total_tokens][2304], row-major: written; must not
 *           overlap x, norm_w or wqkv.
 * The norm runs in fp32 and its output is rounded to bf16 (the GEMM's
 * operand) in a handle-owned buffer of total_tokens x 768 (grown with
 * cudaMalloc when a call needs more; mbert_attn_reserve does not size it);
 * the products accumulate in fp32 and qkv is rounded to bf16 once.  All
 * pointers 16-byte aligned; the caller owns every buffer.  Returns MBERT_OK;
 * MBERT_ERR_BAD_ARG for a null handle or buffer, a misaligned or overlapping
 * buffer, a bad eps or total_tokens outside [0, 2^31); MBERT_ERR_OOM if the
 * buffer cannot grow; MBERT_ERR_CUDA on a launch failure.  Calls that share
 * a handle must not overlap on the GPU (they share the buffer).  Device
 * timeouts are reported by mbert_attn_get_error(). */
int mbert_attn_ln_qkv(mbert_attn *h, const void *x, const void *norm_w, const void *wqkv,
                      int64_t total_tokens, float eps, void *qkv, void *stream);

/* The layer's second block, the GeGLU MLP with its pre-norm and residual:
 * y = x + (GELU(g) * u) Wo^T with g, u the first and second halves of
 * LayerNorm(x) Wi^T ("ModernBERT-base Architecture Teardown", "What Does
 * the GeGLU MLP Do?": Wi makes two vectors of 1152, the first goes through
 * GELU and the second multiplies it, Wo brings 1152 back to 768;
 * "modernbert-base" (nest.franknoh), "The fused projections": the first
 * half of Wi's output is the GELU branch).  GELU is the exact erf form
 * ("ModernBERT" (candding), "The feed-forward halves"); the LayerNorm is as
 * in mbert_attn_ln_qkv.
 *   x       device bf16 [total_tokens][768]: the residual stream.
 *   norm_w  device bf16 [768]: the MLP norm's weight (not NULL).
 *   wi      device bf16 [2304][768], [out][in].
 *   wo      device bf16 [768][1152], [out][in].
 *   eps     as in mbert_attn_ln_qkv.
 *   y       device bf16 [total_tokens][768]: written.  y may be x itself
 *           (in-place update); it must not overlap the weights, and must
 *           overlap x either exactly or not at all.
 * Three kernels: the norm (fp32, bf16 result), Wi with the GeGLU in its
 * epilogue (fp32 accumulation, GELU(g) * u rounded to bf16), Wo with the
 * residual (fp32, y rounded to bf16 once).  The norm's output and the
 * [total_tokens][1152] intermediate live in handle-owned buffers (grown
 * with cudaMalloc when needed); calls sharing a handle must not overlap on
 * the GPU.  All pointers 16-byte aligned.  Returns as mbert_attn_ln_qkv. */
int mbert_attn_mlp(mbert_attn *h, const void *x, const void *norm_w, const void *wi,
                   const void *wo, int64_t total_tokens, float eps, void *y, void *stream);

/* The step after the attention block: the output projection with the
 * residual add, y = x + a Wo^T ("ModernBERT-base Architecture Teardown",
 * "How Does ModernBERT Make Q, K and V?": Wo maps the joined heads back from
 * 768 to 768, stored [out, in]; "ModernBertModel", "Implementing it":
 * x = x + a Wo^T).
 *   a   device bf16 [total_tokens][768], row-major: the attention block's out.
 *   wo  device bf16 [768][768], row-major, [out][in].
 *   x   device bf16 [total_tokens][768], row-major: the residual stream.
 *   y   device bf16 [total_tokens][768], row-major: written.  y may be x
 *       itself (in-place update); it must not overlap a or wo, and must
 *       overlap x either exactly or not at all.
 * Products accumulate in fp32; y is rounded to bf16 (nearest even) once.
 * All pointers 16-byte aligned; the caller owns every buffer.  Returns
 * MBERT_OK; MBERT_ERR_BAD_ARG for a null handle or buffer, a misaligned or
 * overlapping buffer, or total_tokens outside [0, 2^31); MBERT_ERR_CUDA on a
 * launch failure.  Device timeouts are reported by mbert_attn_get_error(). */
int mbert_attn_out_proj(mbert_attn *h, const void *a, const void *wo, const void *x,
                        int64_t total_tokens, void *y, void *stream);

/* ------------------------------------------------------------------------
 * Beside the block: rotary positions and per-head norms on any rows of heads,
 * and attention over keys and values of another length.  For callers whose
 * heads are turned or normed in another way than ModernBERT-base's, and for
 * decoders and pooling heads that read the encoder's states.  These calls
 * keep nothing in the handle but the error word, so calls on different
 * streams may overlap on the GPU; mbert_attn_get_error() waits for all of them.
 * ------------------------------------------------------------------------ */

/* Element types of the calls below. */
enum {
    MBERT_BF16 = 0,
    MBERT_F16 = 1,
    MBERT_F32 = 2     /* rotary and qk_norm_rotary only */
};

/* Which numbers of a head form pair m (of the first dim numbers). */
enum {
    MBERT_ROTARY_HALF = 0,          /* x[m], x[m + dim/2] */
    MBERT_ROTARY_INTERLEAVED = 1    /* x[2m], x[2m + 1] */
};

/* How the frequencies are scaled for contexts longer than the trained one. */
enum {
    MBERT_SCALING_NONE = 0,
    MBERT_SCALING_LINEAR = 1,    /* f / factor */
    MBERT_SCALING_NTK = 2,       /* base * factor^(dim / (dim - 2)); dim > 2 */
    MBERT_SCALING_BY_PARTS = 3,  /* by the turns r = original f / (2 pi) over the original
                                  * context: f where r >= high, f / factor where r <= low,
                                  * linear in r between */
    MBERT_SCALING_YARN = 4       /* the same two borders as pair numbers,
                                  * dim ln(original / (2 pi turns)) / (2 ln base), rounded
                                  * down (high) and up (low), kept within 0 .. dim - 1, and a
                                  * ramp linear in the pair number between them; amplitude
                                  * 0.1 ln(factor) + 1 unless given */
};

typedef struct {
    int kind;           /* MBERT_SCALING_* */
    double factor;      /* > 0; >= 1 for NTK, BY_PARTS and YARN */
    double original;    /* trained context length (BY_PARTS, YARN), > 0 */
    double low, high;   /* borders in turns (BY_PARTS, YARN), 0 < low < high */
    double amplitude;   /* YARN: > 0, or 0 for 0.1 ln(factor) + 1 */
} mbert_attn_scaling;

/* The rotation of a head: its first `dim` numbers, pair m by
 * position * freq[m] radians, both results times `amplitude`. */
typedef struct {
    int dim;            /* even, 0 .. 256 (0: no rotation) */
    int layout;         /* MBERT_ROTARY_* */
    double amplitude;   /* within fp32's range */
    double freq[128];   /* dim / 2 of them, radians per position, finite, >= 0 */
} mbert_attn_rotary_spec;

/* Fill *spec: freq[m] = base^(-2m/dim), scaled (scaling == NULL: not at all).
 * Host only.  base > 1, or MBERT_ERR_BAD_ARG. */
int mbert_attn_rotary_init(mbert_attn_rotary_spec *spec, int dim, int layout, double base,
                           const mbert_attn_scaling *scaling);

/* One tensor of heads: element (t, h, d) at t * row + h * head + d, strides in
 * elements.  src strides may be 0 (broadcast); the elements of dst must be
 * distinct.  dst may be src itself with the same strides (in place); else the
 * two must not overlap (interleaved column blocks of the same rows may). */
typedef struct {
    const void *src;
    void *dst;
    const void *weight;             /* [head_dim], same type: the norm's weight */
    int heads;
    int64_t src_row, src_head, dst_row, dst_head;
} mbert_attn_heads;

/* Rotary positions: dst(t, h) = src(t, h) turned by the position of row t.
 *   tokens         rows, 0 <= tokens < 2^31 (0 enqueues nothing).
 *   head_dim       even, 2 .. 256, >= rope->dim; numbers past rope->dim are copied.
 *   dtype          MBERT_BF16, MBERT_F16 or MBERT_F32; fp32 arithmetic, one rounding.
 *   positions      device, int32 or int64 [tokens] (position_bits 32 or 64), any value; or
 *                  NULL, and then
 *   cu_seqlens     device int32 [n_seqs + 1], cu[0] = 0, non-decreasing, cu[n] <= tokens: a
 *                  row's position is its place in its sequence; rows from cu[n] on are left
 *                  as they were.  A bad cu_seqlens sets MBERT_ERR_BAD_CU_SEQLENS for
 *                  mbert_attn_get_error(), and the results are then unspecified.
 *   inverse        non-zero: by the negative angle (with the same amplitude: the transpose,
 *                  which also is the gradient with respect to src).
 * Any alignment of the element size; 16-byte aligned addresses, strides and parts (head_dim and
 * rope->dim multiples of 16, of 8 for fp32) are read in 16-byte vectors.  One kernel. */
int mbert_attn_rotary(mbert_attn *h, const mbert_attn_heads *x, int64_t tokens, int head_dim,
                      int dtype, const mbert_attn_rotary_spec *rope, const void *positions,
                      int position_bits, const int32_t *cu_seqlens, int n_seqs, int inverse,
                      void *stream);

/* Norms of one head's numbers. */
enum {
    MBERT_NORM_RMS = 1,     /* x / sqrt(mean(x^2) + eps) * weight */
    MBERT_NORM_LAYER = 2    /* (x - mean) / sqrt(population variance + eps) * weight */
};

/* Norm of every query and key head, then the rotation, in one pass and one
 * kernel.  q and k share the rows; either may be NULL (the other is then done
 * alone).  rope == NULL (or rope->dim == 0): the norm alone, without
 * positions.  0 <= eps <= 1; statistics in fp32, where heads whose squares it
 * does not hold are scaled by a power of two first, so any finite numbers do; a
 * head without spread (all zeros, for LayerNorm all equal) is 0/0 with eps = 0.
 * Else as mbert_attn_rotary. */
int mbert_attn_qk_norm_rotary(mbert_attn *h, const mbert_attn_heads *q, const mbert_attn_heads *k,
                              int64_t tokens, int head_dim, int dtype, int norm, float eps,
                              const mbert_attn_rotary_spec *rope, const void *positions,
                              int position_bits, const int32_t *cu_seqlens, int n_seqs,
                              void *stream);

/* Attention of packed queries over keys and values of another length (a
 * decoder's queries over the encoder's states, a pooling head's, or rows that
 * were turned by mbert_attn_rotary, with cu_q = cu_k):
 *   out[i, h] = sum_j softmax_j(scale q[i, h] . k[j, h / g]) v[j, h / g],
 * j over the visible keys of i's sequence, g = heads / kv_heads query heads
 * sharing a key head.  No rotation, no causal mask.  A row without a visible
 * key (or whose visible scores are all -infinity) is 0.  What invisible and
 * other sequences' rows hold, infinities and NaN included, does not matter.
 *   q, out       device [rows_q][heads][head_dim], rows q_row / out_row elements apart
 *   k, v         device [rows_k][kv_heads][head_dim], rows k_row / v_row apart
 *                (16-byte aligned, pitches multiples of 8 and at least the
 *                row's width, so views of fused rows are fine; out overlaps
 *                nothing else; k and v unused for rows_k = 0).  Fewer than
 *                2^31 - 1024 rows each.
 *   head_dim     64 or 128; dtype MBERT_BF16 or MBERT_F16, else MBERT_ERR_UNSUPPORTED.
 *   scale        > 0 and at most 2e38, or 0 for 1 / sqrt(head_dim).
 *   cu_q, cu_k   device int32 [n_seqs + 1]: cu[0] = 0, non-decreasing, cu[n] <= rows; empty
 *                sequences are allowed on either side; rows of out from cu_q[n] on are left
 *                as they were.  NULL: n_seqs sequences of rows / n_seqs each (a padded batch).
 *   max_seqlen_q the caller's bound on the longest query sequence, 0 for none.  Up to
 *                16 / g a kernel for single tokens runs, which reads k and v once, up to 128 / f
 *                (f the largest power of two that divides g) one for short blocks; a longer
 *                sequence found on the device sets MBERT_ERR_SEQ_TOO_LONG.
 *   key_mask     device int32 [rows_k], non-zero = visible, or NULL for all.
 * Scores, weights' sums and products in fp32; weights are rounded to dtype for the second
 * product (off by 2^-8 of themselves at most in bf16, 2^-11 in fp16), out once. */
typedef struct {
    const void *q, *k, *v;
    void *out;
    int64_t q_row, k_row, v_row, out_row;
    int64_t rows_q, rows_k;
    int heads, kv_heads, head_dim, dtype;
    float scale;
    int n_seqs;
    const int32_t *cu_q, *cu_k;
    int max_seqlen_q;
    const int32_t *key_mask;
} mbert_attn_cross_args;

/* Bytes of device workspace that mbert_attn_cross needs for these arguments
 * (pointers need only be NULL or not).  Host only. */
int mbert_attn_cross_workspace(mbert_attn *h, const mbert_attn_cross_args *args, int64_t *bytes);

/* Enqueue the call.  workspace: device memory of that size (NULL for 0),
 * 16-byte aligned, contents irrelevant; it may be used again once the call's work is done, so
 * calls that may overlap on the GPU need one each.  When the device-side
 * checks of cu_q and cu_k fail nothing is written and the error is reported by
 * mbert_attn_get_error().  Results do not depend on timing: the parts of a
 * sequence that several CTAs share are joined in a fixed order. */
int mbert_attn_cross(mbert_attn *h, const mbert_attn_cross_args *args, void *workspace,
                     int64_t workspace_bytes, void *stream);

/* ------------------------------------------------------------------------
 * Layers of any width: matrix products with their epilogue, plain and grouped by
 * expert, and the norms around a block.  For encoders of other sizes, a model's
 * heads, decoders beside the cross attention, and mixtures of experts.  Nothing of a
 * call's data stays in the handle but the error word, so calls on different streams may
 * overlap on the GPU; on the host it keeps how calls of the same sizes run (the plans of
 * 64 of them, under a lock) and the count of launches.
 * ------------------------------------------------------------------------ */

/* Activations, of z in fp32. */
enum {
    MBERT_ACT_NONE = 0,
    MBERT_ACT_GELU = 1,         /* z Phi(z), Phi the normal distribution (the erf form) */
    MBERT_ACT_GELU_TANH = 2,    /* z (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3))) / 2 */
    MBERT_ACT_SILU = 3,         /* z / (1 + e^-z) */
    MBERT_ACT_RELU = 4          /* max(z, 0) */
};

/* A matrix product with bias, activation and residual:
 *   z = x weight^T + bias,  out = residual + act(z);
 * gated, with weight and bias of 2 outer rows, z_g the first and z_u the other half of z:
 *   out = residual + act(z_g) z_u.
 * With experts > 0 the rows are grouped: rows cu_experts[e] .. cu_experts[e+1] take
 * weight and bias e, and row t's result is multiplied by row_scale[t] (a router's weight).
 *   x, out, residual  device [rows][inner] / [rows][outer], rows x_row / out_row /
 *                residual_row elements apart (at least the width).  residual NULL: 0, and
 *                always with experts.  out may be residual itself with the same pitch; else it
 *                overlaps nothing.  x 16-byte aligned with x_row a multiple of 8; out, residual
 *                and bias of any alignment (16-byte aligned rows are faster).
 *   weight       device [max(experts, 1)][outer or 2 outer][inner], rows weight_row and experts
 *                weight_expert elements apart (at least a row's and an expert's extent), multiples
 *                of 8, 16-byte aligned.  ([out][in].)
 *   bias         device [max(experts, 1)][outer or 2 outer], contiguous, or NULL.
 *   rows         0 <= rows < 2^31 - 1024 (0 enqueues nothing); inner, outer 1 .. 2^24.
 *   dtype        MBERT_BF16 or MBERT_F16, of all of these, else MBERT_ERR_UNSUPPORTED.
 *   cu_experts   device int32 [experts + 1] (experts at most 65536): cu[0] = 0, non-decreasing,
 *                cu[experts] <= rows; empty experts are allowed; rows of out from cu[experts] on
 *                are left as they were.  A bad list sets MBERT_ERR_BAD_CU_SEQLENS for
 *                mbert_attn_get_error(), and nothing is written.
 *   row_scale    device fp32 [rows], with experts only, or NULL for 1.
 * Products, sums and the epilogue in fp32, out rounded once.  One kernel, no workspace; results
 * do not depend on timing, but the order of sums may go by all sizes of the call, rows and experts
 * among them. */
typedef struct {
    const void *x, *weight, *bias, *residual;
    void *out;
    int64_t x_row, weight_row, weight_expert, residual_row, out_row;
    int64_t rows;
    int inner, outer, dtype, activation, gated;
    int experts;
    const int32_t *cu_experts;
    const float *row_scale;
} mbert_attn_linear_args;

int mbert_attn_linear(mbert_attn *h, const mbert_attn_linear_args *args, void *stream);

/* How mbert_attn_linear runs a call of these sizes, type aside (pointers and strides are not
 * looked at; host only), for profiles and tests:
 *   plan[0]   0: the kernel for many rows, units of 256 rows x plan[1] columns (of both halves
 *             together where gated);
 *             1: that for few rows, tiles of plan[1] rows x pieces of plan[2] times 32 output
 *             columns, the inner dimension shared by plan[3] CTAs.
 * Its choice goes by rows, experts, inner, outer, activation, gated and the device's SMs. */
int mbert_attn_linear_plan(mbert_attn *h, const mbert_attn_linear_args *args, int32_t plan[4]);

/* Whose gate a row takes. */
enum {
    MBERT_GATE_NONE = 0,
    MBERT_GATE_CHANNELS = 1,    /* gate [width], of every row */
    MBERT_GATE_ROWS = 2,        /* gate [rows][width] */
    MBERT_GATE_SEQUENCES = 3    /* gate [n_seqs][width], of the row's sequence */
};

/* The norms after one block and before the next, with the gate and the residual between:
 *   h = residual_scale x + gate P(branch),  y = N(h),
 * P the norm with branch_weight and branch_bias (branch_weight NULL: none), N the one with
 * weight and bias (weight NULL: no y), both of kind `norm` (MBERT_NORM_*; a bias is added last
 * and may be NULL) over rows of `width`.  branch NULL: y = N(x) alone (no gate, no h,
 * residual_scale 1).
 *   x, branch, h, y   device [rows][width], rows x_row, ... elements apart (at least the width).
 *                h and y may each be x or branch itself with the same pitch; else they overlap
 *                nothing.
 *   width        1 .. 16384; rows as in mbert_attn_linear; dtype MBERT_BF16, _F16 or _F32, of all.
 *   gate         rows of width, gate_row elements apart, as gate_kind says.
 *   cu_seqlens   with MBERT_GATE_SEQUENCES: device int32 [n_seqs + 1] (n_seqs as rows), cu[0] = 0,
 *                non-decreasing, cu[n] <= rows; rows of h and y from cu[n] on are left as they were.  A bad list
 *                sets MBERT_ERR_BAD_CU_SEQLENS, and nothing is written.
 *   eps          0 <= eps <= 1.
 * All in fp32, h and y rounded once; y is of the h that has not been rounded.  Rows whose squares
 * fp32 does not hold are scaled by a power of two first, so any rows of normal numbers do; a row
 * without spread (all zeros, for LayerNorm all equal) is 0/0 with eps = 0.  Any alignment of the element
 * size; rows of whole, 16-byte aligned vectors are read in these.  Of other rows the bytes beside them,
 * within 16-byte boundaries, may be read too, but never those before a tensor's first number or behind
 * its last one; what they hold does not count.  One kernel; the order of a row's sums goes by its width,
 * type and alignment alone, so its results do not depend on the other rows or on how many there are. */
typedef struct {
    const void *x, *branch, *gate;
    const void *weight, *bias, *branch_weight, *branch_bias;
    void *h, *y;
    int64_t x_row, branch_row, gate_row, h_row, y_row;
    int64_t rows;
    int width, dtype, norm, gate_kind;
    const int32_t *cu_seqlens;
    int n_seqs;
    float residual_scale, eps;
} mbert_attn_residual_norm_args;

int mbert_attn_residual_norm(mbert_attn *h, const mbert_attn_residual_norm_args *args, void *stream);

/* Wait for the device's work so far (every stream the handle was used on, and
 * replayed graphs), then return and clear, in one step, the device error word
 * as a status: MBERT_OK, MBERT_ERR_BAD_CU_SEQLENS, MBERT_ERR_SEQ_TOO_LONG or
 * MBERT_ERR_TIMEOUT; MBERT_ERR_CUDA if the wait itself fails.  The word holds
 * what calls on all streams have set since it was last asked for; it does not
 * say which call. */
int mbert_attn_get_error(mbert_attn *h);

/* Diagnostic: enqueue one kernel whose bounded wait on a barrier that
 * nothing completes gives up after limit_us microseconds (1 .. 2000000),
 * exactly as the attention kernels' waits do if a transfer or an MMA never
 * completes.  Afterwards mbert_attn_get_error() returns MBERT_ERR_TIMEOUT.
 * Nothing faults or traps; the context stays usable. */
int mbert_attn_selftest_timeout(mbert_attn *h, int64_t limit_us, void *stream);

/* Largest batch the allocation-free entry point below accepts: total
 * tokens, and also sequences, per call. */
#define MBERT_NOALLOC_MAX_TOKENS 8192

/* The attention block without any device allocation.  The pages have no
 * counterpart: this exists for callers that cannot call cudaMalloc -- a
 * plugin inside a framework that owns all device memory through its own
 * pool, a service whose memory is reserved once at start-up, or a loop that
 * cannot take the device-wide synchronisation cudaMalloc/cudaFree may
 * cause.  Such callers cannot create a handle, so this call needs none.
 *   Arguments as for mbert_attn_forward, on the current CUDA device, with
 *   the ModernBERT-base defaults (half window 64, bases 160000 / 10000).
 *   device_status  device int32 or NULL: receives the device-side error bits
 *                  of this call (0 = ok, 1 = bad cu_seqlens, 2 = a sequence
 *                  longer than max_seqlen, 4 = a bounded wait timed out),
 *                  written on `stream` after the kernels.
 * Scratch memory (work list, rotated Q/K rows, RoPE tables: about 28 MiB)
 * is one static device array that every GPU that loads this part of the
 * library holds until the process exits.  total_tokens or n_seqs above
 * MBERT_NOALLOC_MAX_TOKENS, or max_seqlen above it, are rejected
 * (MBERT_ERR_BAD_ARG / MBERT_ERR_SEQ_TOO_LONG) before anything is enqueued.
 * The first call on a device does a one-time set-up (it looks up the
 * array's device address and fills the RoPE tables with blocking copies,
 * which synchronise with other work on that device); make that first call
 * before any stream capture and outside any loop that must not block.
 * Every call shares the array and overwrites what the previous call left
 * there, so two calls whose work overlaps on the GPU (e.g. on different
 * streams) race.
 * This is not the benchmarked path: for both layer kinds it runs the plan
 * and a RoPE pass into the static rotated-Q/K rows (one launch), then the generic
 * attention kernel (one CTA per 128-query block and head), not the
 * persistent kernels of mbert_attn_forward, so its speed and its fp32
 * summation order differ; its results meet the same bounds against the
 * oracle. */
int mbert_attn_forward_noalloc(const void *qkv, const int32_t *cu_seqlens, int n_seqs,
                               int64_t total_tokens, int max_seqlen, int layer_kind,
                               void *out, int32_t *device_status, void *stream);

/* Measurement.  While enabled, every mbert_attn_forward also records a
 * CUDA event pair on its stream around its attention kernel (the plan and
 * RoPE kernels before it are outside the pair), every mbert_attn_out_proj
 * one around its kernel, and every mbert_attn_ln_qkv and mbert_attn_mlp one
 * around each of their kernels.  The handle always counts the kernels it enqueues. */
int mbert_attn_profile_enable(mbert_attn *h, int enable);

/* Profile slots: the two layer kinds, the output projection, the Wqkv
 * projection, the LayerNorm (before attention or before the MLP) and the
 * MLP's two GEMMs. */
enum {
    MBERT_PROFILE_OUT_PROJ = 2,
    MBERT_PROFILE_QKV_PROJ = 3,
    MBERT_PROFILE_LAYERNORM = 4,
    MBERT_PROFILE_MLP_UP = 5,
    MBERT_PROFILE_MLP_DOWN = 6,
    MBERT_PROFILE_SLOTS = 7
};

/* Synchronise on the recorded events and return, per profile slot (index
 * MBERT_GLOBAL, MBERT_LOCAL or MBERT_PROFILE_* of the host arrays
 * kernel_ms[MBERT_PROFILE_SLOTS] and kernel_launches[MBERT_PROFILE_SLOTS]),
 * the summed kernel milliseconds and
 * the number of recorded kernels, plus the number of kernels enqueued by
 * every entry point (*total_launches).  Clears all three.  Any output
 * pointer may be NULL. */
int mbert_attn_profile_read(mbert_attn *h, double *kernel_ms, int64_t *kernel_launches,
                            int64_t *total_launches);

/* Release the handle's device memory.  NULL is allowed.  The caller must
 * make sure no enqueued work still uses the handle. */
void mbert_attn_destroy(mbert_attn *h);

/* Static, human-readable text for a status code. */
const char *mbert_attn_strerror(int status);

#ifdef __cplusplus
}
#endif

#endif /* MBERT_ATTN_H */
