// tables.cu -- the bookkeeping of a step on the GPU: block tables and slots from
// request lengths, the visibility mask of drafted trees, and the moves that
// keep an accepted path.
//
// The pages build tables on the host and send them to the GPU at every step
// ("vLLM Fundamentals: Paged Attention and Batching", section "Just a python
// process"); with these kernels a step's tables, slots and lengths follow from
// device tensors alone, so a whole step fits one captured graph.
#include <cooperative_groups.h>

#include "device_utils.cuh"
#include "launch.h"

namespace pkv {
namespace {

namespace cg = cooperative_groups;

constexpr int kTableThreads = 1024;  // = sequences scanned at a time
constexpr int kTableWarps = kTableThreads / 32;

// Exclusive prefix sums of a and b over the CTA's threads; *ta, *tb = totals.
// `tmp` holds 2 * (kTableWarps + 1) values. Two barriers.
__device__ __forceinline__ void scan2(int64_t &a, int64_t &b, int64_t *ta, int64_t *tb, int64_t *tmp) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t xa = a, xb = b;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t ya = __shfl_up_sync(0xffffffffu, xa, d), yb = __shfl_up_sync(0xffffffffu, xb, d);
        if (lane >= d) {
            xa += ya;
            xb += yb;
        }
    }
    __syncthreads();
    if (lane == 31) {
        tmp[warp] = xa;
        tmp[kTableWarps + warp] = xb;
    }
    __syncthreads();
    int64_t before_a = 0, before_b = 0, all_a = 0, all_b = 0;
    {
        int64_t wa = lane < kTableWarps ? tmp[lane] : 0, wb = lane < kTableWarps ? tmp[kTableWarps + lane] : 0;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t ya = __shfl_up_sync(0xffffffffu, wa, d), yb = __shfl_up_sync(0xffffffffu, wb, d);
            if (lane >= d) {
                wa += ya;
                wb += yb;
            }
        }
        all_a = __shfl_sync(0xffffffffu, wa, 31);
        all_b = __shfl_sync(0xffffffffu, wb, 31);
        before_a = __shfl_sync(0xffffffffu, wa, (warp + 31) & 31);
        before_b = __shfl_sync(0xffffffffu, wb, (warp + 31) & 31);
        if (warp == 0) before_a = before_b = 0;
    }
    a = before_a + xa - a;
    b = before_b + xb - b;
    *ta = all_a;
    *tb = all_b;
}

// The last entry of starts[0 .. n) that is <= x (starts[0] = 0 <= x).
__device__ __forceinline__ int find_start(const int *starts, int n, int x) {
    int lo = 0, hi = n;  // starts[lo] <= x < starts[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (starts[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

__device__ __forceinline__ int blocks_of(int tokens, int bs) { return tokens / bs + (tokens % bs != 0); }

struct TableScratch {
    int64_t scan[2 * (kTableWarps + 1)];
    int tok[kTableThreads + 1];    // tokens (grow) or freed blocks (trim) before each sequence of the chunk
    int blk[kTableThreads];        // blocks taken before it
    int len[kTableThreads];        // its tokens before the call (grow), its first freed entry (trim)
    int bad;
};

// One cluster. Every CTA sums over all sequences (1024 at a time, one thread
// each), so each knows what the step takes before anything is written: either
// all of it is given or nothing. New token t of the step is then one thread's:
// it finds its sequence in the chunk's prefix sums and its block in the table
// (the tail block the sequence had) or on the stack (the k-th block taken is
// the k-th from the top); the token that opens a block also writes the table
// entry. The reads of a chunk's lengths and the writes over them are a cluster
// barrier apart, so the outputs may be the inputs' own buffers.
__global__ void __launch_bounds__(kTableThreads)
    tables_grow_kernel(int32_t *block_tables, const int32_t *context_lens, const int32_t *new_tokens,
                       const int32_t *free_blocks, const int32_t *num_free, int32_t *new_lens, int32_t *query_start,
                       int64_t *slot_mapping, int32_t *num_free_out, int num_seqs, int num_slots,
                       int max_blocks_per_seq, int block_size, int num_blocks, int32_t *status) {
    __shared__ TableScratch sm;
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, rank = cluster.block_rank(), ctas = cluster.num_blocks();
    const int64_t cap = static_cast<int64_t>(max_blocks_per_seq) * block_size;
    const int top = *num_free;
    if (tid == 0) sm.bad = 0;
    __syncthreads();

    int64_t tokens = 0, blocks = 0;
    for (int s0 = 0; s0 < num_seqs; s0 += kTableThreads) {
        const int s = s0 + tid;
        int64_t n = 0, need = 0, tn, tb;
        if (s < num_seqs) {
            const int L = context_lens[s], add = new_tokens[s];
            if (L < 0 || add < 0 || static_cast<int64_t>(L) + add > cap) {
                atomicOr(&sm.bad, PKV_STATUS_BAD_CONTEXT_LEN);
            } else {
                n = add;
                need = blocks_of(L + add, block_size) - blocks_of(L, block_size);
            }
        }
        scan2(n, need, &tn, &tb, sm.scan);
        tokens += tn;
        blocks += tb;
    }
    __syncthreads();
    int bad = sm.bad;
    if (top < 0 || top > num_blocks)
        bad |= PKV_STATUS_BAD_BLOCK_ID;
    else if (blocks > top)
        bad |= PKV_STATUS_OUT_OF_BLOCKS;
    if (tokens > num_slots) bad |= PKV_STATUS_OUT_OF_SLOTS;

    const int total = bad ? 0 : static_cast<int>(tokens);
    int64_t tok0 = 0, blk0 = 0;
    for (int s0 = 0; s0 < num_seqs; s0 += kTableThreads) {
        const int s = s0 + tid, count = min(kTableThreads, num_seqs - s0);
        int L = 0;
        int64_t n = 0, need = 0, tn, tb;
        if (s < num_seqs) {
            L = context_lens[s];
            if (!bad) {
                n = new_tokens[s];
                need = blocks_of(L + static_cast<int>(n), block_size) - blocks_of(L, block_size);
            }
        }
        const int add = static_cast<int>(n);
        scan2(n, need, &tn, &tb, sm.scan);
        sm.tok[tid] = static_cast<int>(n);
        sm.blk[tid] = static_cast<int>(blk0 + need);
        sm.len[tid] = L;
        cluster.sync();
        if (rank == 0 && s < num_seqs) {
            new_lens[s] = L + add;
            query_start[s + 1] = static_cast<int>(tok0 + n) + add;
        }
        for (int t = rank * kTableThreads + tid; t < tn; t += ctas * kTableThreads) {
            const int i = find_start(sm.tok, count, t);
            const int pos = sm.len[i] + t - sm.tok[i];
            const int lb = pos / block_size, off = pos - lb * block_size;
            const int have = blocks_of(sm.len[i], block_size);
            int32_t *entry = block_tables + static_cast<int64_t>(s0 + i) * max_blocks_per_seq + lb;
            const int p = lb < have ? *entry : free_blocks[top - 1 - (sm.blk[i] + lb - have)];
            if (lb >= have && off == 0) *entry = p;
            const bool good = p >= 0 && p < num_blocks;
            if (!good) atomicOr(status, PKV_STATUS_BAD_BLOCK_ID);
            slot_mapping[tok0 + t] = good ? static_cast<int64_t>(p) * block_size + off : -1;
        }
        tok0 += tn;
        blk0 += tb;
        __syncthreads();  // the chunk's arrays are read before the next one's are written
    }
    for (int64_t t = total + rank * kTableThreads + tid; t < num_slots; t += ctas * kTableThreads) slot_mapping[t] = -1;
    if (num_seqs == 0) cluster.sync();  // the stack's height was read by every CTA
    if (rank == 0 && tid == 0) {
        query_start[0] = 0;
        *num_free_out = bad ? top : top - static_cast<int>(blocks);
        if (bad) atomicOr(status, bad);
    }
}

// The reverse: the blocks past keep_lens go back, the first one freed on top,
// so that a grow undone by a trim leaves the stack as it was.
__global__ void __launch_bounds__(kTableThreads)
    tables_trim_kernel(const int32_t *block_tables, const int32_t *context_lens, const int32_t *keep_lens,
                       int32_t *free_blocks, const int32_t *num_free, int32_t *num_free_out, int num_seqs,
                       int max_blocks_per_seq, int block_size, int num_blocks, int32_t *status) {
    __shared__ TableScratch sm;
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, rank = cluster.block_rank(), ctas = cluster.num_blocks();
    const int64_t cap = static_cast<int64_t>(max_blocks_per_seq) * block_size;
    const int top = *num_free;
    if (tid == 0) sm.bad = 0;
    __syncthreads();

    int64_t freed = 0;
    for (int s0 = 0; s0 < num_seqs; s0 += kTableThreads) {
        const int s = s0 + tid;
        int64_t gone = 0, zero = 0, tg, tz;
        if (s < num_seqs) {
            const int L = context_lens[s], keep = keep_lens[s];
            if (keep < 0 || keep > L || L > cap)
                atomicOr(&sm.bad, PKV_STATUS_BAD_CONTEXT_LEN);
            else
                gone = blocks_of(L, block_size) - blocks_of(keep, block_size);
        }
        scan2(gone, zero, &tg, &tz, sm.scan);
        freed += tg;
    }
    __syncthreads();
    int bad = sm.bad;
    if (top < 0 || top + freed > num_blocks) bad |= PKV_STATUS_BAD_BLOCK_ID;
    cluster.sync();  // every CTA has read the stack's height
    if (rank == 0 && tid == 0) {
        *num_free_out = bad ? top : top + static_cast<int>(freed);
        if (bad) atomicOr(status, bad);
    }
    if (bad) return;

    int64_t done = 0;
    for (int s0 = 0; s0 < num_seqs; s0 += kTableThreads) {
        const int s = s0 + tid, count = min(kTableThreads, num_seqs - s0);
        int64_t gone = 0, zero = 0, tg, tz;
        int first = 0;
        if (s < num_seqs) {
            first = blocks_of(keep_lens[s], block_size);
            gone = blocks_of(context_lens[s], block_size) - first;
        }
        scan2(gone, zero, &tg, &tz, sm.scan);
        sm.tok[tid] = static_cast<int>(gone);
        sm.len[tid] = first;
        __syncthreads();
        for (int k = rank * kTableThreads + tid; k < tg; k += ctas * kTableThreads) {
            const int i = find_start(sm.tok, count, k);
            int p = block_tables[static_cast<int64_t>(s0 + i) * max_blocks_per_seq + sm.len[i] + k - sm.tok[i]];
            if (p < 0 || p >= num_blocks) {
                atomicOr(status, PKV_STATUS_BAD_BLOCK_ID);
                p = -1;
            }
            free_blocks[top + freed - 1 - (done + k)] = p;
        }
        done += tg;
        __syncthreads();
    }
}

// One CTA per sequence, a thread per node: it walks up the tree. Ancestors are
// earlier nodes, so the walk meets the row's words from the last to the first
// and each is written once.
__global__ void __launch_bounds__(128)
    tree_mask_kernel(int32_t *tree_mask, int32_t *depths, const int32_t *parents, const int32_t *query_start,
                     int num_tokens, int max_query_len, int mask_words, int32_t *status) {
    extern __shared__ int up[];
    const int s = blockIdx.x, tid = threadIdx.x;
    const int q0 = query_start[s], q1 = query_start[s + 1], n = q1 - q0;
    if (q0 < 0 || n < 0 || q1 > num_tokens || n > max_query_len) {
        if (tid == 0) atomicOr(status, PKV_STATUS_BAD_CONTEXT_LEN);
        return;
    }
    for (int i = tid; i < n; i += blockDim.x) {
        int p = parents[q0 + i];
        if (p < -1 || p >= i) {
            atomicOr(status, PKV_STATUS_BAD_TREE);
            p = -1;
        }
        up[i] = p;
    }
    __syncthreads();
    for (int i = tid; i < n; i += blockDim.x) {
        int32_t *row = tree_mask + static_cast<int64_t>(q0 + i) * mask_words;
        int w = mask_words - 1, depth = -1;
        uint32_t word = 0;
        for (int j = i; j >= 0; j = up[j]) {
            for (; w > (j >> 5); --w, word = 0) row[w] = static_cast<int32_t>(word);
            word |= 1u << (j & 31);
            ++depth;
        }
        for (; w >= 0; --w, word = 0) row[w] = static_cast<int32_t>(word);
        depths[q0 + i] = depth;
    }
}

constexpr int kKeepThreads = 128;
constexpr int kKeepBatch = 8;  // rows in flight per thread

// One CTA per (sequence, pool, 2 KB of a row): a thread owns 16 bytes of every
// row and moves them in path order. The path rises, so row k's source is at
// or behind k: no earlier move has written it, and a thread never reads what
// another writes.
__global__ void __launch_bounds__(kKeepThreads)
    cache_keep_kernel(uint4 *k_cache, uint4 *v_cache, const int32_t *block_tables, const int32_t *context_lens,
                      const int32_t *query_start, const int32_t *accepted, const int32_t *num_accepted,
                      int32_t *new_lens, int max_accepted, int chunks_per_row, int block_size,
                      int max_blocks_per_seq, int num_blocks, int32_t *status) {
    __shared__ int bad;
    __shared__ int64_t src[kKeepThreads], dst[kKeepThreads];
    const int s = blockIdx.x, tid = threadIdx.x;
    const int c = blockIdx.z * kKeepThreads + tid;
    uint4 *pool = blockIdx.y ? v_cache : k_cache;
    const bool first = blockIdx.y == 0 && blockIdx.z == 0;
    const int L = context_lens[s], n = query_start[s + 1] - query_start[s], a = num_accepted[s];
    const int32_t *path = accepted + static_cast<int64_t>(s) * max_accepted;
    const int32_t *table = block_tables + static_cast<int64_t>(s) * max_blocks_per_seq;
    if (tid == 0) bad = 0;
    __syncthreads();
    if (L < 0 || n < 0 || n > L || L > static_cast<int64_t>(max_blocks_per_seq) * block_size) {
        if (tid == 0) bad = PKV_STATUS_BAD_CONTEXT_LEN;
    } else if (a < 0 || a > n || a > max_accepted) {
        if (tid == 0) bad = PKV_STATUS_BAD_TREE;
    } else {
        const int base = L - n;
        for (int k = tid; k < a; k += kKeepThreads) {
            const int p = path[k];
            if (p < 0 || p >= n || (k > 0 && path[k - 1] >= p)) {
                atomicOr(&bad, PKV_STATUS_BAD_TREE);
                continue;
            }
            const int b0 = table[(base + k) / block_size], b1 = table[(base + p) / block_size];
            if (b0 < 0 || b0 >= num_blocks || b1 < 0 || b1 >= num_blocks) atomicOr(&bad, PKV_STATUS_BAD_BLOCK_ID);
        }
    }
    __syncthreads();
    if (bad) {
        if (first && tid == 0) {
            atomicOr(status, bad);
            if (new_lens) new_lens[s] = L;
        }
        return;
    }
    const int base = L - n;
    if (first && tid == 0 && new_lens) new_lens[s] = base + a;
    for (int k0 = 0; k0 < a; k0 += kKeepThreads) {
        const int k = k0 + tid, count = min(kKeepThreads, a - k0);
        if (k < a) {
            const int from = base + path[k], to = base + k;
            src[tid] = (static_cast<int64_t>(table[from / block_size]) * block_size + from % block_size) * chunks_per_row;
            dst[tid] = (static_cast<int64_t>(table[to / block_size]) * block_size + to % block_size) * chunks_per_row;
        }
        __syncthreads();
        if (c < chunks_per_row) {
            for (int i = 0; i < count; i += kKeepBatch) {
                uint4 row[kKeepBatch];
#pragma unroll
                for (int e = 0; e < kKeepBatch; ++e)
                    if (i + e < count && src[i + e] != dst[i + e]) row[e] = pool[src[i + e] + c];
#pragma unroll
                for (int e = 0; e < kKeepBatch; ++e)
                    if (i + e < count && src[i + e] != dst[i + e]) pool[dst[i + e] + c] = row[e];
            }
        }
        __syncthreads();
    }
}

// One CTA for what a thread each can do in a few steps, up to a portable
// cluster of eight beyond.
int table_ctas(int64_t items) {
    const int64_t want = (items + 4 * kTableThreads - 1) / (4 * kTableThreads);
    return want <= 1 ? 1 : want <= 2 ? 2 : want <= 4 ? 4 : 8;
}

cudaLaunchConfig_t table_config(int ctas, cudaLaunchAttribute *attr, cudaStream_t stream) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kTableThreads);
    cfg.stream = stream;
    attr->id = cudaLaunchAttributeClusterDimension;
    attr->val.clusterDim.x = ctas;
    attr->val.clusterDim.y = 1;
    attr->val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cfg;
}

}  // namespace

cudaError_t tables_grow_launch(int32_t *block_tables, const int32_t *context_lens, const int32_t *new_tokens,
                               const int32_t *free_blocks, const int32_t *num_free, int32_t *new_lens,
                               int32_t *query_start, int64_t *slot_mapping, int32_t *num_free_out, int num_seqs,
                               int num_slots, int max_blocks_per_seq, int block_size, int num_blocks, int32_t *status,
                               cudaStream_t stream) {
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = table_config(table_ctas(num_slots), &attr, stream);
    return cudaLaunchKernelEx(&cfg, tables_grow_kernel, block_tables, context_lens, new_tokens, free_blocks, num_free,
                              new_lens, query_start, slot_mapping, num_free_out, num_seqs, num_slots,
                              max_blocks_per_seq, block_size, num_blocks, status);
}

cudaError_t tables_trim_launch(const int32_t *block_tables, const int32_t *context_lens, const int32_t *keep_lens,
                               int32_t *free_blocks, const int32_t *num_free, int32_t *num_free_out, int num_seqs,
                               int max_blocks_per_seq, int block_size, int num_blocks, int32_t *status,
                               cudaStream_t stream) {
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg =
        table_config(table_ctas(static_cast<int64_t>(num_seqs) * max_blocks_per_seq), &attr, stream);
    return cudaLaunchKernelEx(&cfg, tables_trim_kernel, block_tables, context_lens, keep_lens, free_blocks, num_free,
                              num_free_out, num_seqs, max_blocks_per_seq, block_size, num_blocks, status);
}

cudaError_t tree_mask_launch(int32_t *tree_mask, int32_t *depths, const int32_t *parents, const int32_t *query_start,
                             int num_seqs, int num_tokens, int max_query_len, int mask_words, int32_t *status,
                             cudaStream_t stream) {
    tree_mask_kernel<<<num_seqs, 128, static_cast<size_t>(max_query_len) * 4, stream>>>(
        tree_mask, depths, parents, query_start, num_tokens, max_query_len, mask_words, status);
    return cudaGetLastError();
}

cudaError_t cache_keep_launch(void *k_cache, void *v_cache, const int32_t *block_tables, const int32_t *context_lens,
                              const int32_t *query_start, const int32_t *accepted, const int32_t *num_accepted,
                              int32_t *new_lens, int num_seqs, int max_accepted, int row_bytes, int block_size,
                              int max_blocks_per_seq, int num_blocks, int32_t *status, cudaStream_t stream) {
    const int chunks = row_bytes / 16;
    const dim3 grid(num_seqs, 2, (chunks + kKeepThreads - 1) / kKeepThreads);
    cache_keep_kernel<<<grid, kKeepThreads, 0, stream>>>(
        static_cast<uint4 *>(k_cache), static_cast<uint4 *>(v_cache), block_tables, context_lens, query_start,
        accepted, num_accepted, new_lens, max_accepted, chunks, block_size, max_blocks_per_seq, num_blocks, status);
    return cudaGetLastError();
}

}  // namespace pkv
