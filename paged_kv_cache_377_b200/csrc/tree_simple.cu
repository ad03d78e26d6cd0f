// tree.cu -- attention of drafted trees over the paged cache.
//
// Sequence s brings n_s drafted tokens, the last n_s of its L_s cached ones.
// Draft i sees the committed positions 0 .. L_s - n_s - 1 and the drafts its
// mask row names: out = sum_j e^(scale q.k_j) v_j / sum_j e^(scale q.k_j) over
// what it sees, zero where it sees nothing. What it does not see is never part
// of a sum, whatever it holds.
//
// One warp per (drafted token, query head), lanes over head_dim, one position
// at a time with the running maximum and sum.
#include <cuda_bf16.h>

#include "device_utils.cuh"
#include "launch.h"

namespace pkv {
namespace {

constexpr int kTreeWarps = 4;

__device__ __forceinline__ float e4m3_value(uint8_t code) {
    const __half_raw h = __nv_cvt_fp8_to_halfraw(code, __NV_E4M3);
    return __half2float(__half(h));
}

template <int D, bool FP8>
__global__ void __launch_bounds__(kTreeWarps * 32) paged_tree_simple_kernel(const TreeArgs a) {
    constexpr int E = D / 32;
    const int s = blockIdx.y, lane = threadIdx.x & 31;
    const int q0 = a.query_start[s], n = a.query_start[s + 1] - q0, L = a.context_lens[s];
    if (q0 < 0 || n < 0 || q0 + n > a.num_tokens || n > a.max_query_len || n > L ||
        L > static_cast<int64_t>(a.max_blocks_per_seq) * a.block_size) {
        if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(a.status, PKV_STATUS_BAD_CONTEXT_LEN);
        return;
    }
    const int64_t item = static_cast<int64_t>(blockIdx.x) * kTreeWarps + (threadIdx.x >> 5);
    const int i = static_cast<int>(item / a.num_q_heads), j = static_cast<int>(item % a.num_q_heads);
    if (i >= n) return;
    const int h = j / a.group, base = L - n;
    const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(a.q) +
                             (static_cast<int64_t>(q0 + i) * a.num_q_heads + j) * D + lane * E;
    const int32_t *bits = a.tree_mask + static_cast<int64_t>(q0 + i) * a.mask_words;
    const int32_t *table = a.block_tables + static_cast<int64_t>(s) * a.max_blocks_per_seq;
    const float ks = FP8 ? a.k_scale[h] : 1.f, vs = FP8 ? a.v_scale[h] : 1.f;
    float qv[E], o[E], m = -INFINITY, l = 0.f;
    for (int e = 0; e < E; ++e) {
        qv[e] = __bfloat162float(q[e]) * a.scale_log2 * ks;
        o[e] = 0.f;
    }
    for (int t = 0; t < L; ++t) {
        if (t >= base && !((bits[(t - base) >> 5] >> ((t - base) & 31)) & 1)) continue;
        const int p = table[t / a.block_size];
        if (p < 0 || p >= a.num_blocks) {
            if (lane == 0) atomicOr(a.status, PKV_STATUS_BAD_BLOCK_ID);
            continue;
        }
        const int64_t at =
            ((static_cast<int64_t>(p) * a.block_size + t % a.block_size) * a.num_kv_heads + h) * D + lane * E;
        float x = 0.f, v[E];
        for (int e = 0; e < E; ++e) {
            float k;
            if (FP8) {
                k = e4m3_value(static_cast<const uint8_t *>(a.k_cache)[at + e]);
                v[e] = e4m3_value(static_cast<const uint8_t *>(a.v_cache)[at + e]) * vs;
            } else {
                k = __bfloat162float(static_cast<const __nv_bfloat16 *>(a.k_cache)[at + e]);
                v[e] = __bfloat162float(static_cast<const __nv_bfloat16 *>(a.v_cache)[at + e]);
            }
            x += qv[e] * k;
        }
        for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
        const float top = fmaxf(m, x);
        const float keep = m == -INFINITY ? 0.f : exp2f(m - top), w = exp2f(x - top);
        for (int e = 0; e < E; ++e) o[e] = o[e] * keep + w * v[e];
        l = l * keep + w;
        m = top;
    }
    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out) + (static_cast<int64_t>(q0 + i) * a.num_q_heads + j) * D +
                         lane * E;
    for (int e = 0; e < E; ++e) out[e] = __float2bfloat16(l == 0.f ? 0.f : o[e] / l);
}

}  // namespace

cudaError_t tree_simple_launch(bool fp8, int head_dim, const TreeArgs &a, cudaStream_t stream) {
    const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(a.max_query_len) * a.num_q_heads + kTreeWarps - 1) /
                                          kTreeWarps),
                    a.num_seqs);
    if (head_dim == 64)
        fp8 ? paged_tree_simple_kernel<64, true><<<grid, kTreeWarps * 32, 0, stream>>>(a)
            : paged_tree_simple_kernel<64, false><<<grid, kTreeWarps * 32, 0, stream>>>(a);
    else
        fp8 ? paged_tree_simple_kernel<128, true><<<grid, kTreeWarps * 32, 0, stream>>>(a)
            : paged_tree_simple_kernel<128, false><<<grid, kTreeWarps * 32, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace pkv
