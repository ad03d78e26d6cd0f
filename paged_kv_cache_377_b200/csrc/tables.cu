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
#include "step_utils.cuh"

namespace pkv {
namespace {

namespace cg = cooperative_groups;

constexpr int kTableThreads = 1024;  // = sequences scanned at a time
constexpr int kTableWarps = kTableThreads / 32;
// Consecutive blocks of a thread where there are over two for each: one search, and their loads side by side (32,000
// blocks 7.7 -> 5.7 us; where a thread has one at most, runs of four leave threads idle: 500 blocks 3.5 -> 4.1 us).
constexpr int kRun = 4;
constexpr uint32_t kMany = 0x7fffffffu;  // sums saturate here: more than any pool or step holds

__device__ __forceinline__ uint32_t add_sat(uint32_t a, uint32_t b) { return min(a + b, kMany); }  // a, b <= kMany

// Exclusive prefix sums (saturating) of a and b over the CTA's threads; *ta, *tb = totals. Three barriers.
__device__ __forceinline__ void scan2(uint32_t &a, uint32_t &b, uint32_t *ta, uint32_t *tb, uint2 *tmp) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t a0 = a, b0 = b;
    uint32_t xa = a, xb = b;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const uint32_t ya = __shfl_up_sync(0xffffffffu, xa, d), yb = __shfl_up_sync(0xffffffffu, xb, d);
        if (lane >= d) {
            xa = add_sat(xa, ya);
            xb = add_sat(xb, yb);
        }
    }
    __syncthreads();
    if (lane == 31) tmp[warp] = make_uint2(xa, xb);
    __syncthreads();
    if (warp == 0) {
        uint2 w = tmp[lane];
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t ya = __shfl_up_sync(0xffffffffu, w.x, d), yb = __shfl_up_sync(0xffffffffu, w.y, d);
            if (lane >= d) w = make_uint2(add_sat(w.x, ya), add_sat(w.y, yb));
        }
        tmp[lane] = w;
    }
    __syncthreads();
    const uint2 all = tmp[kTableWarps - 1], before = warp > 0 ? tmp[warp - 1] : make_uint2(0, 0);
    // inclusive minus own: exact wherever the total is (a saturated one is refused, its parts unused)
    a = add_sat(before.x, xa) - a0;
    b = add_sat(before.y, xb) - b0;
    *ta = all.x;
    *tb = all.y;
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
    uint2 scan[kTableWarps];
    int tok[kTableThreads];  // tokens (grow) or freed blocks (trim) before each sequence of the chunk
    int blk[kTableThreads];  // blocks taken before it
    int len[kTableThreads];  // its tokens before the call (grow), its first freed entry (trim)
    int bad;
};

// One cluster. Every CTA sums over all sequences (1024 at a time, one thread
// each), so each knows what the step takes before anything is written: either
// all of it is given or nothing. With SLOTS, new token t of the step is one
// thread's: it finds its sequence in the chunk's prefix sums and its block in
// the table (the tail block the sequence had) or on the stack (the k-th block
// taken is the k-th from the top); the token that opens a block also writes the
// table entry. Without (steps of many tokens), a thread per new block writes the
// table and tables_slots_kernel the slots. The reads of a chunk's lengths and
// the writes over them are a cluster barrier apart, so the outputs may be the
// inputs' own buffers.
template <bool SLOTS>
__global__ void __launch_bounds__(kTableThreads)
    tables_grow_kernel(int32_t *block_tables, const int32_t *context_lens, const int32_t *new_tokens,
                       const int32_t *free_blocks, const int32_t *num_free, int32_t *new_lens, int32_t *query_start,
                       int64_t *slot_mapping, int32_t *num_free_out, int num_seqs, int num_slots,
                       int max_blocks_per_seq, int block_size, int num_blocks, int32_t *status) {
    __shared__ TableScratch sm;
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, rank = cluster.block_rank(), ctas = cluster.num_blocks();
    const int64_t cap = static_cast<int64_t>(max_blocks_per_seq) * block_size;
    depend_wait();
    depend_release();
    const int top = *num_free;
    if (tid == 0) sm.bad = 0;
    __syncthreads();

    int L = 0;
    uint32_t n = 0, need = 0, tn = 0, tb = 0, tokens = 0, blocks = 0;
    auto load = [&](int s, bool check) {
        n = need = 0;
        if (s >= num_seqs) return;
        L = context_lens[s];
        const int add = new_tokens[s];
        if (L < 0 || add < 0 || static_cast<int64_t>(L) + add > cap) {
            if (check) atomicOr(&sm.bad, PKV_STATUS_BAD_CONTEXT_LEN);
            return;
        }
        n = add;
        need = blocks_of(L + add, block_size) - blocks_of(L, block_size);
    };
    for (int s0 = 0; s0 < num_seqs; s0 += kTableThreads) {
        load(s0 + tid, true);
        const uint32_t own_n = n, own_need = need;
        scan2(n, need, &tn, &tb, sm.scan);
        tokens = add_sat(tokens, tn);
        blocks = add_sat(blocks, tb);
        if (num_seqs > kTableThreads) {  // scanned again below
            n = own_n;
            need = own_need;
        } else {
            sm.tok[tid] = static_cast<int>(n);
            sm.blk[tid] = static_cast<int>(need);
            n = own_n;
        }
    }
    __syncthreads();
    int bad = sm.bad;
    if (top < 0 || top > num_blocks)
        bad |= PKV_STATUS_BAD_BLOCK_ID;
    else if (blocks > static_cast<uint32_t>(top))
        bad |= PKV_STATUS_OUT_OF_BLOCKS;
    if (tokens > static_cast<uint32_t>(num_slots)) bad |= PKV_STATUS_OUT_OF_SLOTS;

    const int total = bad ? 0 : static_cast<int>(tokens);
    int tok0 = 0, blk0 = 0;
    for (int s0 = 0; s0 < num_seqs; s0 += kTableThreads) {
        const int s = s0 + tid, count = min(kTableThreads, num_seqs - s0);
        int add = static_cast<int>(n);
        if (num_seqs > kTableThreads) {
            load(s, false);
            add = static_cast<int>(n);
            scan2(n, need, &tn, &tb, sm.scan);
            sm.tok[tid] = static_cast<int>(n);
            sm.blk[tid] = static_cast<int>(need);
        }
        sm.len[tid] = L;
        cluster.sync();
        if (rank == 0 && s < num_seqs) {
            new_lens[s] = bad ? L : L + add;
            query_start[s + 1] = bad ? 0 : tok0 + sm.tok[tid] + add;
        }
        if (!bad) {
            if (SLOTS) {
                for (int t = rank * kTableThreads + tid; t < static_cast<int>(tn); t += ctas * kTableThreads) {
                    const int i = find_start(sm.tok, count, t);
                    const int have = blocks_of(sm.len[i], block_size);
                    int32_t *row = block_tables + static_cast<int64_t>(s0 + i) * max_blocks_per_seq;
                    const int pos = sm.len[i] + (t - sm.tok[i]);
                    const int lb = pos / block_size, off = pos - lb * block_size;
                    const int p = lb < have ? row[lb] : free_blocks[top - 1 - (blk0 + sm.blk[i] + lb - have)];
                    if (lb >= have && off == 0) row[lb] = p;
                    const bool good = p >= 0 && p < num_blocks;
                    if (!good) atomicOr(status, PKV_STATUS_BAD_BLOCK_ID);
                    slot_mapping[tok0 + t] = good ? static_cast<int64_t>(p) * block_size + off : -1;
                }
            } else {
                const int run = static_cast<int>(tb) > 2 * ctas * kTableThreads ? kRun : 1;
                for (int k0 = (rank * kTableThreads + tid) * run; k0 < static_cast<int>(tb);
                     k0 += ctas * kTableThreads * run) {
                    int i = find_start(sm.blk, count, k0);
#pragma unroll
                    for (int j = 0; j < kRun; ++j) {
                        const int k = k0 + j;
                        if (j >= run || k >= static_cast<int>(tb)) break;
                        while (i + 1 < count && sm.blk[i + 1] <= k) ++i;
                        block_tables[static_cast<int64_t>(s0 + i) * max_blocks_per_seq + blocks_of(sm.len[i], block_size) + k -
                                     sm.blk[i]] = free_blocks[top - 1 - (blk0 + k)];
                    }
                }
            }
        }
        tok0 += static_cast<int>(tn);
        blk0 += static_cast<int>(tb);
        __syncthreads();  // the chunk's arrays are read before the next one's are written
    }
    if (SLOTS)
        for (int t = total + rank * kTableThreads + tid; t < num_slots; t += ctas * kTableThreads) slot_mapping[t] = -1;
    if (num_seqs == 0) cluster.sync();  // the stack's height was read by every CTA
    if (rank == 0 && tid == 0) {
        query_start[0] = 0;
        *num_free_out = bad ? top : top - static_cast<int>(blocks);
        if (bad) atomicOr(status, bad);
    }
}

constexpr int kSlotThreads = 256, kSlotSeqs = 8192;  // starts kept in shared memory

// The slots of a step of many tokens, from the lengths, starts and tables that tables_grow_kernel<false> wrote: a
// thread per token, over the whole device (the grow kernel's one cluster took 41 us for 256,000 tokens).
__global__ void __launch_bounds__(kSlotThreads)
    tables_slots_kernel(const int32_t *block_tables, const int32_t *new_lens, const int32_t *query_start,
                        int64_t *slot_mapping, int num_seqs, int num_slots, int max_blocks_per_seq, int block_size,
                        int num_blocks, int32_t *status) {
    extern __shared__ int kept[];
    depend_wait();
    depend_release();
    const int *starts = query_start;
    if (num_seqs <= kSlotSeqs) {
        for (int s = threadIdx.x; s <= num_seqs; s += kSlotThreads) kept[s] = query_start[s];
        __syncthreads();
        starts = kept;
    }
    const int total = starts[num_seqs], step = gridDim.x * kSlotThreads;
#pragma unroll 4
    for (int t = blockIdx.x * kSlotThreads + threadIdx.x; t < num_slots; t += step) {
        int64_t slot = -1;
        if (t < total) {
            const int s = find_start(starts, num_seqs, t);
            const int pos = new_lens[s] - (starts[s + 1] - t);
            const int p = block_tables[static_cast<int64_t>(s) * max_blocks_per_seq + pos / block_size];
            if (p >= 0 && p < num_blocks)
                slot = static_cast<int64_t>(p) * block_size + pos % block_size;
            else
                atomicOr(status, PKV_STATUS_BAD_BLOCK_ID);
        }
        slot_mapping[t] = slot;
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
    depend_wait();
    depend_release();
    const int top = *num_free;
    if (tid == 0) sm.bad = 0;
    __syncthreads();

    int first = 0;
    uint32_t gone = 0, zero = 0, tg = 0, tz = 0, sum = 0;
    auto load = [&](int s, bool check) {
        gone = zero = 0;
        if (s >= num_seqs) return;
        const int L = context_lens[s], keep = keep_lens[s];
        if (keep < 0 || keep > L || L > cap) {
            if (check) atomicOr(&sm.bad, PKV_STATUS_BAD_CONTEXT_LEN);
            return;
        }
        first = blocks_of(keep, block_size);
        gone = blocks_of(L, block_size) - first;
    };
    for (int s0 = 0; s0 < num_seqs; s0 += kTableThreads) {
        load(s0 + tid, true);
        scan2(gone, zero, &tg, &tz, sm.scan);
        sum = add_sat(sum, tg);
    }
    __syncthreads();
    int bad = sm.bad;
    if (top < 0 || top > num_blocks || sum > static_cast<uint32_t>(num_blocks - top)) bad |= PKV_STATUS_BAD_BLOCK_ID;
    cluster.sync();  // every CTA has read the stack's height
    const int freed = static_cast<int>(sum);
    if (rank == 0 && tid == 0) {
        *num_free_out = bad ? top : top + freed;
        if (bad) atomicOr(status, bad);
    }
    if (bad) return;

    int done = 0;
    for (int s0 = 0; s0 < num_seqs; s0 += kTableThreads) {
        const int count = min(kTableThreads, num_seqs - s0);
        if (num_seqs > kTableThreads) {
            load(s0 + tid, false);
            scan2(gone, zero, &tg, &tz, sm.scan);
        }
        sm.tok[tid] = static_cast<int>(gone);
        sm.len[tid] = first;
        __syncthreads();
        const uint32_t run = tg > 2u * ctas * kTableThreads ? kRun : 1;
        // (unsigned: a step past 2^31 - 1 blocks has to end the loop)
        for (uint32_t b0 = (rank * kTableThreads + tid) * run; b0 < tg; b0 += ctas * kTableThreads * run) {
            const int k0 = static_cast<int>(b0), left = static_cast<int>(min(tg - b0, run));
            int i = find_start(sm.tok, count, k0), p[kRun];
#pragma unroll
            for (int j = 0; j < kRun; ++j) {
                const int k = k0 + j;
                if (j >= left) break;
                while (i + 1 < count && sm.tok[i + 1] <= k) ++i;
                p[j] = block_tables[static_cast<int64_t>(s0 + i) * max_blocks_per_seq + sm.len[i] + k - sm.tok[i]];
            }
#pragma unroll
            for (int j = 0; j < kRun; ++j) {
                if (j >= left) break;
                if (p[j] < 0 || p[j] >= num_blocks) {
                    atomicOr(status, PKV_STATUS_BAD_BLOCK_ID);
                    p[j] = -1;
                }
                free_blocks[top + freed - 1 - (done + k0 + j)] = p[j];
            }
        }
        done += static_cast<int>(tg);
        __syncthreads();
    }
}

constexpr int kMaskThreads = 128;

// One CTA per sequence. Within a run of 32 nodes a warp closes the tree by
// pointer doubling: lane i gets the bits of its ancestors in the run, and the
// lowest of them leads out of it (ancestors are earlier nodes). A thread per
// node then hops from run to run, one mask word each, from the last to the
// first: at most n / 32 steps, where a walk from parent to parent took n (a
// chain of 256: 58 us).
__global__ void __launch_bounds__(kMaskThreads)
    tree_mask_kernel(int32_t *tree_mask, int32_t *depths, const int32_t *parents, const int32_t *query_start,
                     int num_tokens, int max_query_len, int mask_words, int32_t *status) {
    extern __shared__ int2 runs[];  // per node: its run's bits, the node that its run's topmost ancestor hangs from
    const int s = blockIdx.x, tid = threadIdx.x, lane = tid & 31;
    depend_wait();
    depend_release();
    int q0, n;
    if (!query_rows(query_start, s, num_tokens, q0, n) || n > max_query_len) {
        if (tid == 0) atomicOr(status, PKV_STATUS_BAD_CONTEXT_LEN);
        return;
    }
    for (int i0 = tid - lane; i0 < n; i0 += kMaskThreads) {
        const int i = i0 + lane;
        int up = i < n ? parents[q0 + i] : -1;
        if (up < -1 || up >= i) {
            atomicOr(status, PKV_STATUS_BAD_TREE);
            up = -1;
        }
        uint32_t bits = 1u << lane;
        int jump = up >= i0 ? up - i0 : -1;  // an ancestor in the run
#pragma unroll
        for (int d = 0; d < 5; ++d) {
            const int from = jump < 0 ? lane : jump;
            const uint32_t more = __shfl_sync(0xffffffffu, bits, from);
            const int next = __shfl_sync(0xffffffffu, jump, from);
            if (jump >= 0) {
                bits |= more;
                jump = next;
            }
        }
        const int out = __shfl_sync(0xffffffffu, up, __ffs(bits) - 1);
        if (i < n) runs[i] = make_int2(static_cast<int>(bits), out);
    }
    __syncthreads();
    for (int i = tid; i < n; i += kMaskThreads) {
        int32_t *row = tree_mask + static_cast<int64_t>(q0 + i) * mask_words;
        int w = mask_words - 1, depth = -1;
        for (int j = i; j >= 0;) {
            const int2 run = runs[j];
            for (; w > (j >> 5); --w) row[w] = 0;
            row[w--] = run.x;
            depth += __popc(static_cast<uint32_t>(run.x));
            j = run.y;
        }
        for (; w >= 0; --w) row[w] = 0;
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
    depend_wait();
    depend_release();
    int q0, n;
    const bool rows_good = query_rows(query_start, s, 0x7fffffff, q0, n);  // (the step's rows are not read here)
    const int L = context_lens[s], a = num_accepted[s];
    const int32_t *path = accepted + static_cast<int64_t>(s) * max_accepted;
    const int32_t *table = block_tables + static_cast<int64_t>(s) * max_blocks_per_seq;
    if (tid == 0) bad = 0;
    __syncthreads();
    if (!rows_good || L < 0 || n > L || L > static_cast<int64_t>(max_blocks_per_seq) * block_size) {
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

// A thread per item, in one CTA up to a portable cluster of eight (8192 slots:
// 10.5 us in one CTA, 6.9 in two, 4.0 in eight; a trim of 16 sequences 2.8 in
// one and 3.0 in eight).
int table_ctas(int64_t items) {
    const int64_t want = (items + kTableThreads - 1) / kTableThreads;
    return want <= 1 ? 1 : want <= 2 ? 2 : want <= 4 ? 4 : 8;
}

// Steps of more slots than this leave them to tables_slots_kernel (16,384 slots:
// 5.1 us in the cluster, 5.5 with the second kernel; 32,768: 7.5 and 6.3;
// 256,000: 41 and 10).
constexpr int kClusterSlots = 16384;

}  // namespace

cudaError_t tables_grow_launch(int32_t *block_tables, const int32_t *context_lens, const int32_t *new_tokens,
                               const int32_t *free_blocks, const int32_t *num_free, int32_t *new_lens,
                               int32_t *query_start, int64_t *slot_mapping, int32_t *num_free_out, int num_seqs,
                               int num_slots, int max_blocks_per_seq, int block_size, int num_blocks, int32_t *status,
                               cudaStream_t stream) {
    const bool few = num_slots <= kClusterSlots;
    const int ctas = table_ctas(few ? num_slots : num_slots / block_size + num_seqs);
    cudaError_t e = launch_overlapped(few ? tables_grow_kernel<true> : tables_grow_kernel<false>, dim3(ctas),
                                      kTableThreads, 0, ctas, stream, block_tables, context_lens, new_tokens,
                                      free_blocks, num_free, new_lens, query_start, slot_mapping, num_free_out, num_seqs,
                                      num_slots, max_blocks_per_seq, block_size, num_blocks, status);
    if (e != cudaSuccess || few) return e;
    const int blocks = (num_slots + kSlotThreads - 1) / kSlotThreads;
    return launch_overlapped(tables_slots_kernel, dim3(blocks < 148 * 8 ? blocks : 148 * 8), kSlotThreads,
                             num_seqs <= kSlotSeqs ? (static_cast<size_t>(num_seqs) + 1) * 4 : 0, 1, stream,
                             block_tables, new_lens, query_start, slot_mapping, num_seqs, num_slots, max_blocks_per_seq,
                             block_size, num_blocks, status);
}

cudaError_t tables_trim_launch(const int32_t *block_tables, const int32_t *context_lens, const int32_t *keep_lens,
                               int32_t *free_blocks, const int32_t *num_free, int32_t *num_free_out, int num_seqs,
                               int max_blocks_per_seq, int block_size, int num_blocks, int32_t *status,
                               cudaStream_t stream) {
    const int ctas = table_ctas(static_cast<int64_t>(num_seqs) * max_blocks_per_seq);
    return launch_overlapped(tables_trim_kernel, dim3(ctas), kTableThreads, 0, ctas, stream, block_tables, context_lens,
                             keep_lens, free_blocks, num_free, num_free_out, num_seqs, max_blocks_per_seq, block_size,
                             num_blocks, status);
}

cudaError_t tree_mask_launch(int32_t *tree_mask, int32_t *depths, const int32_t *parents, const int32_t *query_start,
                             int num_seqs, int num_tokens, int max_query_len, int mask_words, int32_t *status,
                             cudaStream_t stream) {
    return launch_overlapped(tree_mask_kernel, dim3(num_seqs), kMaskThreads, static_cast<size_t>(max_query_len) * 8, 1,
                             stream, tree_mask, depths, parents, query_start, num_tokens, max_query_len, mask_words,
                             status);
}

cudaError_t cache_keep_launch(void *k_cache, void *v_cache, const int32_t *block_tables, const int32_t *context_lens,
                              const int32_t *query_start, const int32_t *accepted, const int32_t *num_accepted,
                              int32_t *new_lens, int num_seqs, int max_accepted, int row_bytes, int block_size,
                              int max_blocks_per_seq, int num_blocks, int32_t *status, cudaStream_t stream) {
    const int chunks = row_bytes / 16;
    const dim3 grid(num_seqs, 2, (chunks + kKeepThreads - 1) / kKeepThreads);
    return launch_overlapped(cache_keep_kernel, grid, kKeepThreads, 0, 1, stream, static_cast<uint4 *>(k_cache),
                             static_cast<uint4 *>(v_cache), block_tables, context_lens, query_start, accepted,
                             num_accepted, new_lens, max_accepted, chunks, block_size, max_blocks_per_seq, num_blocks,
                             status);
}

}  // namespace pkv
