// The library handle, for the host-side translation units.  Not part of the
// public C ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cuda_bf16.h>

#include <atomic>
#include <mutex>
#include <vector>

#include "mbert_attn.h"
#include "internal.h"
#include "linear.h"

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                  const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                  const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

struct mbert_attn {
    int device = 0;
    mbert::RopeConsts rope_consts[2];              // per layer kind, for in-kernel cos/sin
    int num_sms = 0;
    mbert_attn_config cfg{};
    float2 *rope[2] = {nullptr, nullptr};   // [MBERT_GLOBAL], [MBERT_LOCAL]: [max_seqlen][32]
    int32_t *err = nullptr;                 // sticky device error word, and what get_error took of it
    int32_t *work_count = nullptr;
    int2 *work = nullptr;
    int64_t work_cap = 0;                   // entries
    __nv_bfloat16 *rot = nullptr;           // rotated Q/K scratch [rows][1536]
    int64_t rot_cap = 0;                    // rows
    __nv_bfloat16 *ln = nullptr;            // normalised rows [ln_cap][768] (ln_qkv, mlp)
    int64_t ln_cap = 0;                     // rows
    __nv_bfloat16 *mid = nullptr;           // GELU(g) * u rows [mid_cap][1152] (mlp)
    int64_t mid_cap = 0;                    // rows
    // the padded-batch call: packed qkv and out, each padded token's rank
    // among its row's real tokens, the row lengths and their cu_seqlens
    __nv_bfloat16 *pad_qkv = nullptr, *pad_out = nullptr;
    int64_t pad_qkv_cap = 0, pad_out_cap = 0;
    int32_t *pad_idx = nullptr, *pad_len = nullptr, *pad_cu = nullptr;
    int64_t pad_idx_cap = 0, pad_seq_cap = 0;
    // global layers: split of the (entry, head, key tile) iterations among
    // one persistent CTA per SM
    int32_t *tile_start = nullptr;          // [entries + 1]
    int32_t *unit_cnt = nullptr;            // [entries * heads]
    int64_t sk_cap = 0;                     // entries
    float *partials = nullptr;              // [2 * num_sms][kPartialFloats]
    // global layers: norms of the rotated rows, for the score bound that
    // lets the softmax skip its row maximum: Q fp32 [12][rot_cap], then K
    // fp16 [12][rot_cap] (rot_cap a multiple of 8)
    float *norms = nullptr;
    EncodeTiledFn encode = nullptr;
    // measurement: event pairs around the attention kernel, per layer kind
    bool profiling = false;
    // start, end, start, end, ... per profile slot (global, local, projection)
    std::vector<cudaEvent_t> ev[MBERT_PROFILE_SLOTS];
    size_t ev_used[MBERT_PROFILE_SLOTS] = {};
    std::atomic<int64_t> launches{0};       // every kernel this handle enqueued (calls of several threads count)
    // recently encoded tensor maps, by (address, width, rows): encoding one
    // costs microseconds of host time, as much as a short kernel
    struct MapEntry {
        const void *ptr = nullptr;
        int width = 0;
        int64_t rows = -1;
        uint64_t used = 0;
        CUtensorMap map;
    };
    MapEntry maps[32];
    uint64_t map_clock = 0;
    mbert::PlanEntry plans[64];             // of products of any width, by their sizes
    std::mutex plan_lock;
};

namespace mbert {

// 2-D tensor map of 16-bit elements over [rows][width], rows `pitch` elements
// apart, box 64 columns x `box` rows, 128-byte swizzle, out-of-range reads
// give 0.  l2_bytes: what the L2 fetches at a time, 128 or 256.
int encode_rows(const mbert_attn *h, CUtensorMap *tm, const void *ptr, int64_t width, int64_t rows,
                int64_t pitch, int box, int l2_bytes);

// 3-D tensor map of 16-bit elements over [rows][heads][dim], box 64 columns x
// `fold` heads x 128 / fold rows (128 rows of shared memory, a row's heads side
// by side); otherwise as encode_rows.
int encode_heads(const mbert_attn *h, CUtensorMap *tm, const void *ptr, int dim, int64_t heads, int64_t rows,
                 int64_t pitch, int fold);

struct DeviceGuard {
    int prev = -1;
    bool changed = false;
    explicit DeviceGuard(int dev)
    {
        if (cudaGetDevice(&prev) == cudaSuccess && prev != dev) {
            changed = cudaSetDevice(dev) == cudaSuccess;
        }
    }
    ~DeviceGuard()
    {
        if (changed)
            cudaSetDevice(prev);
    }
};

}  // namespace mbert
