// What cross attention does before and after its attention kernels: the key
// mask as bits, and the joining of units that were cut between CTAs.
#include "common.cuh"
#include "internal.h"
#include "roles.cuh"

namespace mbert {
namespace {

constexpr int kBitThreads = 512;

// One block per sequence: key_mask [rows_k] of int32 to one bit per key, the
// place after the sequence's last visible key, and the number of visible keys
// before its first hidden one.  Reads the mask once (4 bytes a key), so that
// the attention kernels skip the tiles behind the last visible key, take those
// before the first hidden one without a mask, and read 16 bytes for each of
// the rest; a right-padded row needs no bits at all.
__global__ void __launch_bounds__(kBitThreads)
key_bits_kernel(const int32_t *__restrict__ cu_k, int len_k, long long rows_k,
                const int32_t *__restrict__ mask, uint32_t *__restrict__ bits, int2 *__restrict__ len)
{
    pdl_wait();
    __shared__ int s_last[kBitThreads / 32], s_full[kBitThreads / 32];
    const int s = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long row0 = cu_k ? cu_k[s] : static_cast<long long>(s) * len_k;
    long long end = cu_k ? cu_k[s + 1] : row0 + len_k;
    // offsets that the attention kernel will refuse must not lead outside
    // the mask (nor, as words are counted from them, outside the bits)
    const bool bad = row0 < 0 || end < row0 || end > rows_k;
    const int n = bad ? 0 : static_cast<int>(end - row0);
    int last = 0, full = n;
    for (int j0 = 32 * warp; j0 < n; j0 += kBitThreads) {
        const int j = j0 + lane;
        const uint32_t b = __ballot_sync(0xffffffffu, j < n && mask[row0 + j] != 0);
        if (lane == 0)
            bits[key_bit_word(row0, s) + j0 / 32] = b;
        if (b)
            last = j0 + 32 - __clz(b);
        if (b != 0xffffffffu)
            full = min(full, j0 + __ffs(~b) - 1);
    }
    if (lane == 0) {
        s_last[warp] = last;
        s_full[warp] = full;
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        const bool mine = lane < kBitThreads / 32;
        const int v = __reduce_max_sync(0xffffffffu, mine ? s_last[lane] : 0);
        const int f = __reduce_min_sync(0xffffffffu, mine ? s_full[lane] : n);
        if (lane == 0)
            len[s] = make_int2(v, f);
    }
    pdl_trigger();
}

// The parts of a unit are states over disjoint keys, (O_p, m_p, l_p) with
// O_p = sum 2^(s - m_p) v and l_p = sum 2^(s - m_p).  With m = max m_p,
//   out = sum_p O_p 2^(m_p - m) / sum_p l_p 2^(m_p - m),
// 0 where no part saw a visible key.  Always in the order of the parts, so a
// call's result does not depend on which CTA ran first.  Block (c, y) joins
// rows of the unit whose first part CTA c holds: kRows rows side by side, D/8
// threads a row, kGroups groups of threads that share a row's parts (for few
// rows cut into many parts).  Bound: latency; the parts lie in L2.
template <int D, bool kHalf, int kUnitRows, int kRows, int kGroups>
__global__ void __launch_bounds__(kRows * kGroups * (D / 8))
cross_join_kernel(const CrossRecord *__restrict__ records, const float *__restrict__ parts_base,
                  void *__restrict__ out, long long out_row)
{
    pdl_wait();
    constexpr int kChunks = D / 8;
    constexpr long long kSlot = cross_slot_floats(kUnitRows, D);
    const CrossRecord rec = records[blockIdx.x];
    const int tid = threadIdx.x;
    const int r = blockIdx.y * kRows + tid % kRows;
    const int chunk = tid / kRows % kChunks, group = tid / (kRows * kChunks);
    const bool mine = rec.parts > 0 && r < rec.rows;
    float o[8], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        o[i] = 0.f;
    if (mine) {
        // part 0 lies in CTA c's slot 1, part p > 0 in CTA c + p's slot 0
        auto slot = [&](int p) {
            return parts_base + (2ll * (blockIdx.x + p) + (p == 0)) * kSlot;
        };
#pragma unroll 4
        for (int p = group; p < rec.parts; p += kGroups) {
            const float *src = slot(p);
            const float2 ml = __ldcg(reinterpret_cast<const float2 *>(src + kUnitRows * D) + r);
            const float4 a = __ldcg(reinterpret_cast<const float4 *>(src) + (2 * chunk) * kUnitRows + r);
            const float4 b = __ldcg(reinterpret_cast<const float4 *>(src) + (2 * chunk + 1) * kUnitRows + r);
            const float mn = fmaxf(m, ml.x);
            // a part without a visible key has m = -inf and l = 0
            const float wa = m == -INFINITY ? 0.f : ex2_approx(m - mn);
            const float wb = ml.x == -INFINITY ? (ml.y == 0.f ? 0.f : 1.f) : ex2_approx(ml.x - mn);
            o[0] = o[0] * wa + a.x * wb;
            o[1] = o[1] * wa + a.y * wb;
            o[2] = o[2] * wa + a.z * wb;
            o[3] = o[3] * wa + a.w * wb;
            o[4] = o[4] * wa + b.x * wb;
            o[5] = o[5] * wa + b.y * wb;
            o[6] = o[6] * wa + b.z * wb;
            o[7] = o[7] * wa + b.w * wb;
            l = l * wa + ml.y * wb;
            m = mn;
        }
    }
    if constexpr (kGroups > 1) {
        // the groups' states, in order of the groups
        __shared__ float s_state[kGroups][kChunks][kRows][10];
        float *mine_s = s_state[group][chunk][tid % kRows];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            mine_s[i] = o[i];
        mine_s[8] = m;
        mine_s[9] = l;
        __syncthreads();
        if (group == 0) {
            for (int g = 1; g < kGroups; ++g) {
                const float *x = s_state[g][chunk][tid % kRows];
                const float mn = fmaxf(m, x[8]);
                const float wa = m == -INFINITY ? (l == 0.f ? 0.f : 1.f) : ex2_approx(m - mn);
                const float wb = x[8] == -INFINITY ? (x[9] == 0.f ? 0.f : 1.f) : ex2_approx(x[8] - mn);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    o[i] = o[i] * wa + x[i] * wb;
                l = l * wa + x[9] * wb;
                m = mn;
            }
        }
    }
    if (mine && group == 0) {
        const float inv = l == 0.f ? 0.f : 1.f / l;
        uint4 *dst = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(out) + (rec.row0 + r / rec.group) * out_row +
                                               static_cast<long long>(rec.head0 + r % rec.group) * D + 8 * chunk);
        *dst = make_uint4(pack2<kHalf>(o[0] * inv, o[1] * inv), pack2<kHalf>(o[2] * inv, o[3] * inv),
                          pack2<kHalf>(o[4] * inv, o[5] * inv), pack2<kHalf>(o[6] * inv, o[7] * inv));
    }
    pdl_trigger();
}

template <int D, bool kHalf>
cudaError_t join(const CrossArgs &a, int rows, int ctas, cudaStream_t stream)
{
    constexpr int kGroups = 128 / (D / 8);      // 128 threads for one row's parts
    if (rows == kCrossSmallRows)
        return launch_chained(cross_join_kernel<D, kHalf, kCrossSmallRows, 32, 1>,
                              dim3(ctas, kCrossSmallRows / 32), dim3(32 * (D / 8)), 0, stream, a.records,
                              a.parts, a.out, a.out_row);
    if (rows > kCrossTokenRows)
        return launch_chained(cross_join_kernel<D, kHalf, kCrossBlockRows, 32, 1>,
                              dim3(ctas, kCrossBlockRows / 32), dim3(32 * (D / 8)), 0, stream, a.records,
                              a.parts, a.out, a.out_row);
    // more than a few rows: four to a block, with a quarter of the threads each
    // (a block per row would be mostly blocks without work)
    if (rows > 4)
        return launch_chained(cross_join_kernel<D, kHalf, kCrossTokenRows, 4, kGroups / 4>,
                              dim3(ctas, (rows + 3) / 4), dim3(128), 0, stream, a.records, a.parts, a.out,
                              a.out_row);
    return launch_chained(cross_join_kernel<D, kHalf, kCrossTokenRows, 1, kGroups>,
                          dim3(ctas, rows), dim3(128), 0, stream, a.records, a.parts, a.out,
                          a.out_row);
}

}  // namespace

cudaError_t launch_key_bits(const CrossArgs &a, const int32_t *key_mask, uint32_t *bits, int2 *len,
                            cudaStream_t stream)
{
    return launch_chained(key_bits_kernel, dim3(a.n_seqs), dim3(kBitThreads), 0, stream, a.cu_k, a.len_k,
                          a.rows_k, key_mask, bits, len);
}

cudaError_t launch_cross_join(const CrossArgs &a, int dim, bool half, int rows, int ctas, cudaStream_t stream)
{
    if (dim == 64)
        return half ? join<64, true>(a, rows, ctas, stream) : join<64, false>(a, rows, ctas, stream);
    return half ? join<128, true>(a, rows, ctas, stream) : join<128, false>(a, rows, ctas, stream);
}

}  // namespace mbert
