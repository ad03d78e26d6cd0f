// tree.cu -- attention of drafted trees over the paged cache (tcgen05).
//
// Sequence s brings n_s drafted tokens, the last n_s of its L_s cached ones.
// Draft i sees the committed positions 0 .. L_s - n_s - 1 and the drafts its
// mask row names: out = sum_j e^(scale q.k_j) v_j / sum_j e^(scale q.k_j) over
// what it sees, zero where it sees nothing.
//
// A row is a (draft, query head of the kv head's group) pair: 128 / G drafts
// make a row tile. Sequences, kv heads and row tiles make segments of 64-token
// iterations; the CTAs of one wave (two per SM) take equal shares of all
// iterations, plus a fixed cost per segment, so a long context is cut between
// many CTAs and short ones are strung together in one. Row tiles of a sequence
// go in pairs: k CTAs walk the first tiles of all pairs and k others, in step
// with them, the second ones, so that their reads of the same K and V are L2
// hits; what has no partner is the share of the remaining CTAs. (With the second
// tiles simply behind all first ones, a batch of one- and two-tile trees over 4K
// to 32K tokens read its cache almost twice, 456 MB for 246 MB.)
// A segment cut in two is joined by whichever of its CTAs comes second; one cut
// in more leaves fp32 partials (O, the maximum and the sum of each row) to
// tree_merge_kernel.
//
// Roles, each walking the CTA's share on its own: one warp brings Q and K by
// TMA, one V, one issues the MMAs (S = Q K^T into tensor memory, O += P V with P
// read from there), and four warps hold a row per thread: they load its 64
// logits, hide what the row does not see, keep the running maximum and sum in
// fp32, and write P in bf16 beside S. The mask only matters in the iterations
// that reach past the committed tokens: a row's bits for 64 positions are two
// words there.
// Over e4m3 pools S takes K's codes as they are: each row of Q, scaled by a power
// of two, is split into two e4m3 terms (four bits each of its eight), and S = Q1 K^T
// + Q2 K^T on kind::f8f6f4 costs what one bf16 product does. V is widened to f16 by
// two warps, exactly, and P written in f16: e4m3 terms of P would lose the small
// weights of a long context beside a large one. f16 has its own floor, so P's largest
// is kept between 2^7 and 2^15: weights down to 2^-21 of it keep eleven bits, the next
// ones steps of 2^-24 in P, and what is below 2^-32 of it rounds to zero. (Widening K to
// bf16 as well kept the integer pipe busy for longer than the copies take.)
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>

#include "device_utils.cuh"
#include "launch.h"
#include "step_utils.cuh"
#include "tcgen05_utils.cuh"

namespace pkv {
namespace {

constexpr int kRows = 128;       // rows of a tile (= tensor-memory lanes)
constexpr int kTokens = 64;      // positions of one iteration
constexpr int kBadRing = 8;      // iterations whose bad-block bits are kept (a loader is at most 5 ahead)
// Copies of what the softmax warps tell one another once a piece, by the piece's parity. One would not do: a warp may
// read a piece's word as late as the end of its stores, and nothing holds the others back until it loads S of the next
// piece's first iteration; if that is also its last one, they write the next piece's word before. Past that iteration
// they wait for it, so that the word of the piece after next is safe.
constexpr int kPieceSlots = 2;

// A CTA's share of the step, piece by piece (a piece: consecutive iterations of
// one segment). Every role walks it alike.
struct Walk {
    int x, x1;            // weight position, end of the share
    int e;                // entry of the weights: a sequence's pairs of row tiles, or (past num_seqs) its odd one
    bool second;          // whether the pairs' second tiles are walked
    int s;                // the piece's sequence
    int q0, n, L, h, i0;  // its queries, length, kv head and first draft
    int nit, it0, it1;    // iterations of its segment, and of the piece
    int it;

    __device__ __forceinline__ bool next_piece(const TreeArgs &a, const int *wp) {
        while (x < x1) {
            while (wp[e + 1] <= x) ++e;
            const bool alone = a.lists == 1 || e >= a.num_seqs;
            s = e >= a.num_seqs ? e - a.num_seqs : e;
            q0 = __ldg(a.query_start + s);
            n = __ldg(a.query_start + s + 1) - q0;
            L = __ldg(a.context_lens + s);
            nit = (L + kTokens - 1) / kTokens;
            const int w = nit + a.piece_cost, local = x - wp[e], seg = local / w, off = local - seg * w;
            int end = w;
            if (a.whole) {
                if (off > 0) {  // the segment began in another CTA's share
                    x += w - off;
                    continue;
                }
            } else if (w - off > x1 - x) {
                end = off + (x1 - x);
            }
            x += end - off;
            it0 = max(0, off - a.piece_cost);
            it1 = max(0, end - a.piece_cost);
            if (it1 > it0) {
                const int tiles = (n + a.tile_drafts - 1) / a.tile_drafts;
                const int pairs = tiles >> 1;
                h = alone ? seg : seg / pairs;
                i0 = (alone ? tiles - 1 : 2 * (seg - h * pairs) + (second ? 1 : 0)) * a.tile_drafts;
                it = it0;
                return true;
            }
        }
        return false;
    }
    // The next iteration (of this piece or the next one).
    __device__ __forceinline__ bool next(const TreeArgs &a, const int *wp) { return ++it < it1 || next_piece(a, wp); }
};

// The 64 visibility bits of a mask row (n drafts behind `first` committed positions) for positions t0 .. t0 + 63,
// where t0 + 63 is at or past the first draft.
__device__ __forceinline__ uint2 visible_bits(const int32_t *row, int n, int first, int t0) {
    const int j0 = t0 - first;  // draft of bit 0 (negative: committed positions before)
    const int w0 = max(j0, 0) >> 5, words = (n + 31) >> 5;
    uint32_t w[3];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        w[k] = w0 + k < words ? static_cast<uint32_t>(__ldg(row + w0 + k)) : 0u;
        const int left = n - 32 * (w0 + k);  // drafts from this word on
        if (left < 32) w[k] = left > 0 ? w[k] & ((1u << left) - 1u) : 0u;
    }
    if (j0 >= 0)
        return make_uint2(__funnelshift_r(w[0], w[1], j0 & 31), __funnelshift_r(w[1], w[2], j0 & 31));
    const uint64_t bits = (static_cast<uint64_t>(w[1]) << 32) | w[0];
    const uint64_t vis = (bits << -j0) | ((1ull << -j0) - 1ull);
    return make_uint2(static_cast<uint32_t>(vis), static_cast<uint32_t>(vis >> 32));
}

template <int D, bool FP8>
struct TreeShape {
    static constexpr int HALVES = D / 64;                     // 128-byte column slices of a 16-bit row
    static constexpr uint32_t kHalfKV = kTokens * 128;
    static constexpr uint32_t kTileV = HALVES * kHalfKV;      // V of one stage (16-bit)
    static constexpr uint32_t kTileK = FP8 ? kTokens * D : kTileV;
    static constexpr uint32_t kQHalf = kRows * 128;
    static constexpr uint32_t kTileQ = HALVES * kQHalf;
    // warps: 0 - 3 softmax; over bf16 pools the loaders of K and V and the MMAs; over e4m3 pools the loader of K, the
    // MMAs and V's two (which widen)
    static constexpr int kLoadK = 4, kLoadV = FP8 ? 6 : 5, kMma = FP8 ? 5 : 6, kThreads = FP8 ? 256 : 224;
    // stages of the operand tiles and of the codes of V: what leaves room for two CTAs per SM
    static constexpr int kStagesK = FP8 ? 3 : 2, kStagesV = 2, kRawV = 2;
    static constexpr uint32_t kRawTile = kTokens * D;  // V's codes of one iteration
    static constexpr uint32_t kRaw = FP8 ? kRawV * kRawTile : 0;
    static constexpr uint32_t kOperands = kTileQ + kStagesK * kTileK + kStagesV * kTileV + kRaw;
};

// A warp's `span` rows of codes (dense, D bytes each) into rows tok0 .. of an operand tile ([64-column half][row][128
// bytes], swizzled), as f16 (exact). Eight rows of four 16-code chunks a step; rows and halves alternate so that neither
// side's banks meet; four steps' codes are loaded before the first is stored, so that their latencies overlap.
// The hardware's conversion of two codes takes 2.0 cycles of a scheduler per warp instruction (63 lanes per SM-clock; 16
// independent values a thread, one to eight warps a scheduler), as one byte permute or one logic operation does:
// placing the bits by hand takes several of those.
template <int D>
__device__ __forceinline__ void widen_rows(const uint8_t *src, uint8_t *dst, int tok0, int span, int lane) {
    constexpr int HALVES = D / 64, BATCH = 4;
    const int row = lane >> 2, chunk = lane & 3;
    for (int i0 = 0; i0 < span / 8 * HALVES; i0 += BATCH) {
        uint4 codes[BATCH];
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
            const int i = i0 + k, t = i / HALVES * 8 + row, hf = HALVES == 1 ? 0 : (i ^ row) & 1;
            codes[k] = *reinterpret_cast<const uint4 *>(src + t * D + hf * 64 + chunk * 16);
        }
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
            const int i = i0 + k, t = i / HALVES * 8 + row, hf = HALVES == 1 ? 0 : (i ^ row) & 1;
            const uint32_t c[4] = {codes[k].x, codes[k].y, codes[k].z, codes[k].w};
            uint32_t w[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
                    static_cast<__nv_fp8x2_storage_t>(e & 1 ? c[e / 2] >> 16 : c[e / 2] & 0xffffu), __NV_E4M3);
                w[e] = *reinterpret_cast<const uint32_t *>(&h);
            }
            uint8_t *at = dst + hf * (kTokens * 128) + (tok0 + t) * 128;
            *reinterpret_cast<uint4 *>(at + (((2 * chunk) ^ (t & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
            *reinterpret_cast<uint4 *>(at + (((2 * chunk + 1) ^ (t & 7)) << 4)) = make_uint4(w[4], w[5], w[6], w[7]);
        }
    }
}

// A warp's 32 rows of the query tile, in place: the 64 bf16 of each 128-byte slab row become 64 + 64 e4m3 codes, q f = q1
// + q2 with f a power of two that puts the row's largest magnitude in [2^7, 2^8). q1 keeps four bits, q2 the next four
// (what is below 2^-10 of q f is lost: 2^-17 of the row's largest). Eight lanes a row, four rows a step. Returns 1 / f of
// the lane's own row. A row that is not finite becomes codes of NaN, as all its logits are: what it does not see is
// hidden behind them like any other, so the factor stays finite. A loop, like all that runs once a piece:
// unrolled, it took 6,000 to 10,000 cycles a piece.
template <int D>
__device__ __forceinline__ float split_queries(uint8_t *sq, int row0, int lane) {
    constexpr int HALVES = D / 64;
    const int ch = lane & 7;
    float mine = 1.f;
#pragma unroll 1
    for (int step = 0; step < 8; ++step) {
        const int r = row0 + step * 4 + (lane >> 3);
        uint8_t *row = sq + r * 128;
        uint32_t q[HALVES][4];
        uint32_t top = 0;  // largest magnitude: bf16 magnitudes order like their bits
#pragma unroll
        for (int hf = 0; hf < HALVES; ++hf) {
            const uint4 v = *reinterpret_cast<const uint4 *>(row + hf * (kRows * 128) + ((ch ^ (r & 7)) << 4));
            q[hf][0] = v.x;
            q[hf][1] = v.y;
            q[hf][2] = v.z;
            q[hf][3] = v.w;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                top = max(top, max(q[hf][i] & 0x7fffu, (q[hf][i] >> 16) & 0x7fffu));
        }
#pragma unroll
        for (int d = 1; d < 8; d <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
        const int e = static_cast<int>(top >> 7);                                                  // exponent field
        const float f = __uint_as_float(static_cast<uint32_t>(min(261 - e, 247)) << 23);           // 2^(134 - e) or 2^120
        const float inv = __uint_as_float(static_cast<uint32_t>(max(e - 7, 7)) << 23);
        const float its = __shfl_sync(0xffffffffu, inv, (lane & 3) * 8);
        if ((lane >> 2) == step) mine = its;
#pragma unroll
        for (int hf = 0; hf < HALVES; ++hf) {
            uint32_t w1[2] = {0, 0}, w2[2] = {0, 0};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float2 v = bf16x2_to_float2(q[hf][i]);
                v = make_float2(v.x * f, v.y * f);
                const __nv_fp8x2_storage_t c1 = __nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3);
                const __half2_raw back = __nv_cvt_fp8x2_to_halfraw2(c1, __NV_E4M3);
                const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&back));
                const __nv_fp8x2_storage_t c2 =
                    __nv_cvt_float2_to_fp8x2(make_float2(v.x - b.x, v.y - b.y), __NV_SATFINITE, __NV_E4M3);
                w1[i >> 1] |= static_cast<uint32_t>(c1) << (16 * (i & 1));
                w2[i >> 1] |= static_cast<uint32_t>(c2) << (16 * (i & 1));
            }
            if (e == 255) w1[0] = w1[1] = w2[0] = w2[1] = 0x7f7f7f7fu;
            __syncwarp();  // the rows' slabs are read
            uint8_t *slab = row + hf * (kRows * 128) + (ch & 1) * 8;
            *reinterpret_cast<uint2 *>(slab + (((ch >> 1) ^ (r & 7)) << 4)) = make_uint2(w1[0], w1[1]);
            *reinterpret_cast<uint2 *>(slab + (((4 + (ch >> 1)) ^ (r & 7)) << 4)) = make_uint2(w2[0], w2[1]);
        }
    }
    return mine;
}

constexpr int kSoftmaxWarps = 4;
constexpr uint32_t kTmemCols = 256;  // S | two buffers of P | O: two CTAs fill an SM's 512

struct TreeBars {
    uint64_t q_full, q_ready, q_empty, done;  // (q_ready: e4m3, the queries are split)
    uint64_t k_full[3], k_empty[3], v_full[2], v_empty[2];
    uint64_t raw_full[2][2];  // e4m3: V's codes, first and second 32 tokens
    // S is in tensor memory; the softmax threads have loaded it; P (buffer b) is written; O += P V of buffer b is
    // done; the piece's O is done
    uint64_t s_full, s_free, p_ready[2], pv_free[2], o_full;
    uint64_t all;  // the softmax warps meet
    int scan[16];
    uint32_t bad[kBadRing];  // blocks without a place in the pool, a bit each
    uint32_t tmem;
    int abort;
    int arrived[kPieceSlots];
    int poison[kPieceSlots];
    Walk walk[4];  // the softmax warps' pieces
    int start, total, ctas, index;  // the CTA's group: weight positions, CTAs, and its own place among them
    int bound_prev, bound_next;     // where the share of the CTA before begins and of the CTA after ends
};

// Waits (bounded) until the four warps of the CTA that came first have stored their partial.
__device__ __forceinline__ bool wait_stored(const unsigned *count, volatile int *abort, int32_t *status) {
    bool got = true;
    if ((threadIdx.x & 31) == 0) {
        const uint64_t t0 = globaltimer_ns();
        unsigned seen;
        for (uint32_t it = 1;; ++it) {
            asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(seen) : "l"(count) : "memory");
            if ((seen >> 4) == kSoftmaxWarps) break;
            if (*abort) {
                got = false;
                break;
            }
            if ((it & 63u) == 0 && globaltimer_ns() - t0 > kWaitLimitNs) {
                *abort = 1;
                atomicOr(status, PKV_STATUS_WAIT_TIMEOUT);
                got = false;
                break;
            }
        }
    }
    return __all_sync(0xffffffffu, got);
}

template <int D, int BS, bool FP8>
__global__ void __launch_bounds__(TreeShape<D, FP8>::kThreads, 2)
    paged_tree_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const TreeArgs a) {
    using Sh = TreeShape<D, FP8>;
    constexpr int HALVES = Sh::HALVES, BPI = kTokens / BS, kThreads = Sh::kThreads;
    constexpr int kStagesK = Sh::kStagesK, kStagesV = Sh::kStagesV;
    constexpr int kLoadK = Sh::kLoadK, kLoadV = Sh::kLoadV, kMma = Sh::kMma;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    // ---- shared memory: Q | K stages | V stages | V's codes | barriers | weights before each entry
    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sq = base;
    uint8_t *sk = sq + Sh::kTileQ;
    uint8_t *sv = sk + kStagesK * Sh::kTileK;
    uint8_t *raw = sv + kStagesV * Sh::kTileV;
    TreeBars &B = *reinterpret_cast<TreeBars *>(raw + Sh::kRaw);
    int *wp = reinterpret_cast<int *>(&B + 1);

    // ---- barriers and tensor memory, while the lengths are on their way
    if (warp == kMma) {  // all of the CTA's columns
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&B.tmem)),
                     "r"(kTmemCols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::);
        tc_fence_before();
    } else if (warp == kLoadK && lane == 0) {
        mbar_init(&B.q_full, 1);
        mbar_init(&B.q_empty, 1);
        mbar_init(&B.done, 1);
        mbar_init(&B.s_full, 1);
        mbar_init(&B.s_free, kSoftmaxWarps);
        mbar_init(&B.o_full, 1);
        mbar_init(&B.all, kSoftmaxWarps);
        mbar_init(&B.q_ready, kSoftmaxWarps);
        for (int i = 0; i < kStagesK; ++i) {
            mbar_init(&B.k_full[i], 1);
            mbar_init(&B.k_empty[i], 1);
        }
        for (int i = 0; i < kStagesV; ++i) {
            mbar_init(&B.v_full[i], FP8 ? 2 : 1);
            mbar_init(&B.v_empty[i], 1);
            mbar_init(&B.raw_full[0][i], 1);
            mbar_init(&B.raw_full[1][i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&B.p_ready[i], kSoftmaxWarps);
            mbar_init(&B.pv_free[i], 1);
        }
        for (int i = 0; i < kPieceSlots; ++i) B.poison[i] = 0;
        B.abort = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tm_q);
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
    }

    depend_wait();
    depend_release();
    // ---- weights: every CTA sums over all sequences (one contiguous run per thread)
    const int entries = a.num_seqs * a.lists;
    {
        const int per = (a.num_seqs + kThreads - 1) / kThreads;
        const int s0 = min(tid * per, a.num_seqs), s1 = min(s0 + per, a.num_seqs);
        int sum[2] = {0, 0};
        for (int s = s0; s < s1; ++s) {
            int q0, n, tiles = 0;
            const bool rows_good = query_rows(a.query_start, s, a.num_tokens, q0, n);
            const int L = __ldg(a.context_lens + s);
            if (!rows_good || n > a.max_query_len || n > L || L > static_cast<int64_t>(a.max_blocks_per_seq) * BS) {
                if (blockIdx.x == 0) atomicOr(a.status, PKV_STATUS_BAD_CONTEXT_LEN);
            } else {
                tiles = (n + a.tile_drafts - 1) / a.tile_drafts;
            }
            const int w = a.num_kv_heads * ((L + kTokens - 1) / kTokens + a.piece_cost);
            for (int k = 0; k < a.lists; ++k) {
                const int mine = tiles > 0 ? w * (k + 1 < a.lists ? tiles >> 1 : tiles & 1) : 0;
                wp[k * a.num_seqs + s + 1] = mine;
                sum[k] += mine;
            }
        }
        int inc[2] = {sum[0], sum[1]};
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int y0 = __shfl_up_sync(0xffffffffu, inc[0], d), y1 = __shfl_up_sync(0xffffffffu, inc[1], d);
            if (lane >= d) {
                inc[0] += y0;
                inc[1] += y1;
            }
        }
        if (lane == 31) {
            B.scan[warp] = inc[0];
            B.scan[8 + warp] = inc[1];
        }
        __syncthreads();
        int run[2] = {inc[0] - sum[0], inc[1] - sum[1]};
        for (int w = 0; w < kThreads / 32; ++w) {
            run[1] += B.scan[w];  // the tiles without a partner come behind the pairs
            if (w < warp) {
                run[0] += B.scan[w];
                run[1] += B.scan[8 + w];
            }
        }
        for (int k = 0; k < a.lists; ++k)
            for (int s = s0; s < s1; ++s) {
                run[k] += wp[k * a.num_seqs + s + 1];
                wp[k * a.num_seqs + s + 1] = run[k];
            }
        if (tid == 0) {
            wp[0] = 0;
            if (!a.whole) a.cuts[blockIdx.x] = make_int4(0, 0, 0, 0);
        }
    }
    __syncthreads();
    // C CTAs take shares: k the first tiles of the pairs, k the second ones, the rest what has no partner
    const int pairs = a.lists == 2 ? wp[a.num_seqs] : 0, alone = wp[entries] - pairs, W = 2 * pairs + alone;
    const int groups = (pairs > 0 ? 2 : 0) + (alone > 0 ? 1 : 0);
    const int C = max(groups, min(static_cast<int>(gridDim.x), W / a.min_weight + (W % a.min_weight != 0)));
    int k = 0;
    if (pairs > 0)
        k = alone == 0 ? C / 2
                       : min(max(static_cast<int>((2 * static_cast<int64_t>(C) * pairs + W) / (2 * static_cast<int64_t>(W))), 1),
                             (C - 1) / 2);
    const int c = blockIdx.x;
    const bool paired = c < 2 * k;
    const int ctas = paired ? k : C - 2 * k, index = !paired ? c - 2 * k : c < k ? c : c - k;  // the CTA in its group
    const int start = paired ? 0 : pairs, total = paired ? pairs : alone;
    auto share = [&](int i) {  // where the group's i-th share begins (a 32-bit division where the product fits)
        return start + (total <= 0x7fffffff / kTreeMaxCtas
                            ? static_cast<int>(static_cast<uint32_t>(total) * i / static_cast<uint32_t>(ctas))
                            : static_cast<int>(static_cast<int64_t>(total) * i / ctas));
    };
    if (c >= C || total == 0) {
        if (warp == kMma) {
            tc_fence_after();
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(B.tmem), "r"(kTmemCols));
        }
        return;
    }
    Walk walk;
    walk.x = share(index);
    walk.x1 = share(index + 1);
    walk.second = paired && c >= k;
    if (tid == 0) {
        B.start = start;
        B.total = total;
        B.ctas = ctas;
        B.index = index;
        B.bound_prev = index > 0 ? share(index - 1) : start;
        B.bound_next = index + 2 <= ctas ? share(index + 2) : start + total;
    }
    {
        int lo = 0, hi = entries;  // wp[lo] <= x < wp[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (wp[mid] <= walk.x)
                lo = mid;
            else
                hi = mid;
        }
        walk.e = lo;
    }
    __syncthreads();
    tc_fence_after();
    volatile int *abort_flag = &B.abort;
    const uint32_t tbase = B.tmem;

    uint32_t q_loads = 0;
    // The piece's queries, once the MMAs of the piece before are done with theirs (K's first loader).
    auto load_q = [&](const Walk &w) {
        if (q_loads > 0 && !warp_wait(&B.q_empty, (q_loads - 1) & 1u, abort_flag, a.status)) return false;
        if (lane == 0) {
            mbar_arrive_expect_tx(&B.q_full, HALVES * a.tile_drafts * a.group * 128);
#pragma unroll
            for (int q = 0; q < HALVES; ++q)
                tma_load_5d(sq + q * Sh::kQHalf, &tm_q, &B.q_full, 0, q, 0, w.h, w.q0 + w.i0);
        }
        __syncwarp();
        ++q_loads;
        return true;
    };

    if (warp == kLoadK || (!FP8 && warp == kLoadV)) {
        // ---------------- load warps: lane j copies one block, or one 128-byte column slice of it (16-bit rows)
        constexpr int kStages = FP8 ? kStagesK : kStagesV, kSlices = FP8 ? 1 : HALVES;
        constexpr uint32_t kTile = Sh::kTileK, kRowBytes = FP8 ? D : 128;
        static_assert(FP8 || kStagesK == kStagesV, "K and V alike");
        const bool is_v = warp == kLoadV;
        uint8_t *ring = is_v ? sv : sk;
        uint64_t *full = is_v ? B.v_full : B.k_full, *empty = is_v ? B.v_empty : B.k_empty;
        // (a row's slices side by side: with all first slices before all second ones, 8K contexts read 5% slower)
        const int jb = lane / kSlices, hf = lane % kSlices;
        const bool has = lane < BPI * kSlices;
        auto entry = [&](const Walk &w) {  // this lane's table entry of the iteration, -1: no such block
            const int b = w.it * BPI + jb;
            return has && b * BS < w.L ? __ldg(a.block_tables + static_cast<int64_t>(w.s) * a.max_blocks_per_seq + b)
                                       : -1;
        };
        uint32_t g = 0;
        bool more = walk.next_piece(a, wp), ok = true, fresh = true;
        int p = more ? entry(walk) : -1;
        while (more) {
            Walk ahead = walk;
            const bool more2 = ahead.next(a, wp);
            const int p2 = more2 ? entry(ahead) : -1;  // in flight while this iteration waits
            const int st = g % kStages;
            if (g >= kStages && !(ok = warp_wait(&empty[st], (g / kStages - 1) & 1u, abort_flag, a.status))) break;
            const bool there = has && (walk.it * BPI + jb) * BS < walk.L;
            const bool mine = there && p >= 0 && p < a.num_blocks;
            const unsigned m = __ballot_sync(0xffffffffu, mine), lost = __ballot_sync(0xffffffffu, there && !mine);
            if (!is_v) {
                uint32_t bits = 0;
                if (lost) {
#pragma unroll
                    for (int k = 0; k < BPI; ++k) bits |= ((lost >> (k * kSlices)) & 1u) << k;
                    if (lane == 0) atomicOr(a.status, PKV_STATUS_BAD_BLOCK_ID);
                }
                if (lane == 0) B.bad[g % kBadRing] = bits;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive_expect_tx(&full[st], static_cast<uint32_t>(__popc(m)) * BS * kRowBytes);
            __syncwarp();
            if (mine) {
                if (FP8)
                    tma_load_3d(ring + st * kTile + jb * BS * D, &tm_k, &full[st], 0, walk.h, p * BS);
                else
                    tma_load_4d(ring + st * kTile + hf * Sh::kHalfKV + jb * BS * 128, is_v ? &tm_v : &tm_k, &full[st], 0,
                                hf, walk.h, p * BS);
            }
            ++g;
            if (!is_v && fresh && !(ok = load_q(walk))) break;
            fresh = more2 && ahead.it == ahead.it0;
            walk = ahead;
            more = more2;
            p = p2;
        }
        // copies still in flight (only after a wait gave up) land before exit
        if (!ok || *abort_flag) {
            if (q_loads > 0) mbar_wait_drain(&B.q_full, (q_loads - 1) & 1u, a.status);
            for (uint32_t u = g > kStages ? g - kStages : 0; u < g; ++u)
                mbar_wait_drain(&full[u % kStages], (u / kStages) & 1u, a.status);
        }
        __syncwarp();
    } else if (FP8 && warp >= kLoadV) {
        // ---------------- V's warps over e4m3 pools, 32 tokens each: codes into the warp's own ring, widened into the
        // operand tile, and the ring's stage filled again.
        constexpr int kSpan = kTokens / 2, kBlocks = kSpan / BS, kRings = Sh::kRawV;
        const int part = warp - kLoadV, tok0 = part * kSpan;
        uint8_t *ring = raw + part * kRings * kSpan * D;
        uint64_t *filled = B.raw_full[part];
        const bool has = lane < kBlocks;
        auto entry = [&](const Walk &w) {
            const int b = w.it * BPI + part * kBlocks + lane;
            return has && b * BS < w.L ? __ldg(a.block_tables + static_cast<int64_t>(w.s) * a.max_blocks_per_seq + b)
                                       : -1;
        };
        uint32_t issued = 0, g = 0;
        bool more = walk.next_piece(a, wp), ok = true;
        int p = more ? entry(walk) : -1;
        auto issue = [&]() {  // the next iteration's codes into its ring stage
            Walk ahead = walk;
            const bool more2 = ahead.next(a, wp);
            const int p2 = more2 ? entry(ahead) : -1, st = issued % kRings;
            const bool mine = p >= 0 && p < a.num_blocks;
            const unsigned m = __ballot_sync(0xffffffffu, mine);
            if (lane == 0) mbar_arrive_expect_tx(&filled[st], static_cast<uint32_t>(__popc(m)) * BS * D);
            __syncwarp();
            if (mine)
                tma_load_3d(ring + (st * kSpan + lane * BS) * D, &tm_v, &filled[st], 0, walk.h, p * BS);
            ++issued;
            walk = ahead;
            more = more2;
            p = p2;
        };
        while (more && issued < kRings) issue();
        while (g < issued) {
            const int st = g % kRings, sv_st = g % kStagesV;
            if (!(ok = warp_wait(&filled[st], (g / kRings) & 1u, abort_flag, a.status))) break;
            if (g >= kStagesV && !(ok = warp_wait(&B.v_empty[sv_st], (g / kStagesV - 1) & 1u, abort_flag, a.status))) break;
            widen_rows<D>(ring + st * kSpan * D, sv + sv_st * Sh::kTileV, tok0, kSpan, lane);
            fence_proxy_async_shared();
            __syncwarp();
            if (lane == 0) mbar_arrive(&B.v_full[sv_st]);
            ++g;
            if (more) issue();
        }
        if (!ok || *abort_flag)
            for (uint32_t u = g; u < issued; ++u) mbar_wait_drain(&filled[u % kRings], (u / kRings) & 1u, a.status);
        __syncwarp();
    } else if (warp == kMma) {
        // ---------------- MMA warp: one elected lane issues. S(it + 1) is issued as soon as the softmax warps hold
        // S(it) in registers, and runs while they work on it; O += P(it) V(it) follows P(it).
        const bool leader = elect_one();
        const uint64_t dq = smem_desc(smem_u32(sq), 16, 1024),
                       dk = FP8 && D == 64 ? smem_desc_64b(smem_u32(sk), 16, 512) : smem_desc(smem_u32(sk), 16, 1024),
                       dv = smem_desc(smem_u32(sv), Sh::kHalfKV, 1024);
        const uint32_t t_p = tbase + 64, t_o = tbase + 128;
        Walk ws = walk, wv = walk;
        uint32_t gs = 0, gv = 0, pieces = 0;
        bool ok = true;
        auto step_s = [&]() {
            const int st = gs % kStagesK;
            if (ws.it == ws.it0) {
                if (!(ok = warp_wait(FP8 ? &B.q_ready : &B.q_full, pieces & 1u, abort_flag, a.status))) return;
                ++pieces;
            }
            if (!(ok = warp_wait(&B.k_full[st], (gs / kStagesK) & 1u, abort_flag, a.status))) return;
            if (gs > 0 && !(ok = warp_wait(&B.s_free, (gs - 1) & 1u, abort_flag, a.status))) return;
            tc_fence_after();
            if (leader) {
                if (FP8) {  // the two terms of Q against the same codes, 32 of them a step
#pragma unroll
                    for (int term = 0; term < 2; ++term)
#pragma unroll
                        for (int kk = 0; kk < D / 32; ++kk)
                            umma_f8(tbase, dq + ((kk / 2 * Sh::kQHalf + term * 64 + kk % 2 * 32) >> 4),
                                    dk + ((st * Sh::kTileK + kk * 32) >> 4), instr_desc(128, kTokens, false, true),
                                    (term | kk) != 0);
                } else {
#pragma unroll
                    for (int hf = 0; hf < HALVES; ++hf)
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            umma(tbase, dq + ((hf * Sh::kQHalf + kk * 32) >> 4),
                                 dk + ((st * Sh::kTileK + hf * Sh::kHalfKV + kk * 32) >> 4),
                                 instr_desc(128, kTokens, false), (hf | kk) != 0);
                }
                umma_commit(&B.s_full);
                umma_commit(&B.k_empty[st]);
                if (ws.it + 1 == ws.it1) umma_commit(&B.q_empty);
            }
            __syncwarp();
            ++gs;
        };
        auto step_v = [&]() {
            const int st = gv % kStagesV;
            const uint32_t b = gv & 1u;
            if (!(ok = warp_wait(&B.v_full[st], (gv / kStagesV) & 1u, abort_flag, a.status))) return;
            if (!(ok = warp_wait(&B.p_ready[b], (gv >> 1) & 1u, abort_flag, a.status))) return;
            tc_fence_after();
            if (leader) {
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    umma_ts(t_o, t_p + 32 * b + kk * 8, dv + ((st * Sh::kTileV + kk * 16 * 128) >> 4),
                            instr_desc(128, D, true, FP8), wv.it != wv.it0 || kk != 0);
                umma_commit(&B.pv_free[b]);
                umma_commit(&B.v_empty[st]);
                if (wv.it + 1 == wv.it1) umma_commit(&B.o_full);
            }
            __syncwarp();
            ++gv;
        };
        bool more_s = ws.next_piece(a, wp), more_v = more_s && wv.next_piece(a, wp);
        if (more_s) {
            step_s();
            more_s = ok && ws.next(a, wp);
        }
        while (ok && more_v) {
            // (over e4m3 pools the softmax warps split a piece's queries when they are through with the piece before:
            // its last P V cannot wait for the next piece's first S)
            const bool late = FP8 && more_s && ws.it == ws.it0;
            if (more_s && !late) {
                step_s();
                if (!ok) break;
                more_s = ws.next(a, wp);
            }
            step_v();
            if (!ok) break;
            more_v = wv.next(a, wp);
            if (late) {
                step_s();
                more_s = ok && ws.next(a, wp);
            }
        }
        // every MMA issued is done before the tensor memory is freed (one phase: nothing aliases)
        if (leader) umma_commit(&B.done);
        __syncwarp();
        mbar_wait_drain(&B.done, 0, a.status);
        __syncwarp();
    } else {
        // ---------------- softmax warps: thread r owns row r (tensor-memory lane r)
        const int r = tid;
        const uint32_t t_s = tbase + (static_cast<uint32_t>(warp * 32) << 16), t_p = t_s + 64, t_o = t_s + 128;
        const int G = a.group;
        float c2 = fabsf(a.scale_log2), v_scale = 1.f;
        bool negative = a.scale_log2 < 0.f;
        const bool spare = r >= a.tile_drafts * G;
        volatile int *poison = B.poison;
        // How far below a maximum the reference is put: with the 2^8 that it may lag behind, f16 (to 65504) has room for
        // 2^7. O, the sum and the partials belong to the reference as it is, so that it cancels. (8192 weights about
        // 2^-24.5 of a large one, P alone rounded: their sum is off by up to 7 % without, by 0.02 % with it.)
        constexpr float kLift = FP8 ? 7.f : 0.f;
        uint32_t g = 0, pieces = 0, met_all = 0;
        bool ok = true;
        auto signal = [&](uint64_t *bar) {  // one arrival per warp, after all its lanes
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
        };
        auto meet_all = [&]() {
            signal(&B.all);
            return ok = warp_wait(&B.all, met_all++ & 1u, abort_flag, a.status);
        };
        // the piece that is worked on lives in shared memory, a copy per warp: only what the loop needs takes registers
        Walk &now = B.walk[warp];
        if (lane == 0) now = walk;
        __syncwarp();
        while (ok) {
            Walk next = now;
            const bool more = next.next_piece(a, wp);
            __syncwarp();
            if (lane == 0) now = next;
            __syncwarp();
            if (!more) break;
            const uint32_t piece = pieces++, slot = piece % kPieceSlots;
            const int it0 = next.it0, it1 = next.it1, first = next.L - next.n;  // first draft's position
            const int draft = next.i0 + r / G;
            const bool live = !spare && draft < next.n;
            const bool warp_live = __any_sync(0xffffffffu, live);
            if (FP8) {
                // Queries are split by the threads that own them. The head's K scale and the split's factor go into
                // the logits' factor, V's scale into O.
                if (!(ok = warp_wait(&B.q_full, piece & 1u, abort_flag, a.status))) break;
                const float f = a.scale_log2 * __ldg(a.k_scale + next.h) * (warp_live ? split_queries<D>(sq, warp * 32, lane) : 1.f);
                fence_proxy_async_shared();
                signal(&B.q_ready);
                c2 = fabsf(f) < 1e-37f ? 1e-37f : fabsf(f);
                negative = f < 0.f;
                v_scale = __ldg(a.v_scale + next.h);
            }
            const int32_t *bits = a.tree_mask + static_cast<int64_t>(next.q0 + min(draft, next.n - 1)) * a.mask_words;
            float m_ref = -INFINITY, l_run = 0.f;
            for (int it = it0; it < it1; ++it, ++g) {
                const uint32_t b = g & 1u;
                const int t0 = it * kTokens;
                if (!(ok = warp_wait(&B.s_full, g & 1u, abort_flag, a.status))) break;
                const uint32_t bad = B.bad[g % kBadRing];
                const bool tail = t0 + kTokens > first;
                if (!warp_live) {
                    signal(&B.s_free);
                } else {
                    tc_fence_after();
                    float x[64];
                    tmem_ld64(t_s, x);
                    tc_fence_before();
                    signal(&B.s_free);
                    if (negative) {
#pragma unroll
                        for (int i = 0; i < 64; ++i) x[i] = -x[i];
                    }
                    if (tail || bad) {
                        uint2 vis = tail ? visible_bits(bits, now.n, first, t0) : make_uint2(~0u, ~0u);
                        if (bad) {
#pragma unroll
                            for (int k = 0; k < BPI; ++k) {
                                if (!((bad >> k) & 1u)) continue;
                                const uint32_t gone = BS == 32 ? ~0u : 0xffffu << (k % 2 * 16);
                                if (k * BS < 32)
                                    vis.x &= ~gone;
                                else
                                    vis.y &= ~gone;
                            }
                        }
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            if (!((vis.x >> i) & 1u)) x[i] = -INFINITY;
                            if (!((vis.y >> i) & 1u)) x[32 + i] = -INFINITY;
                        }
                    }
                    float mx;
                    {
                        float m4[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
                        for (int i = 4; i < 60; i += 8) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) m4[e] = fmax3(m4[e], x[i + e], x[i + 4 + e]);
                        }
#pragma unroll
                        for (int e = 0; e < 4; ++e) m4[e] = fmaxf(m4[e], x[60 + e]);
                        mx = fmax3(fmaxf(m4[0], m4[1]), m4[2], m4[3]);
                    }
                    // The reference, kLift below a maximum, moves only when that would be exceeded by more than 2^8. (f16: at
                    // any excess from 2^20 on, where what the products here are rounded by would use up what is left of
                    // its range; so it lasts to 2^26.)
                    float m_new = m_ref;
                    const float top = mx * c2, lag = FP8 && fabsf(top) >= 0x1p20f ? 0.f : 8.f;
                    if (top > m_ref + (kLift + lag)) m_new = top - kLift;
                    const float shift = m_new == -INFINITY ? 0.f : -m_new;  // a row that has seen nothing: P = 0
                    const float2 cc = make_float2(c2, c2), nm = make_float2(shift, shift);
                    float2 ps2a = make_float2(0.f, 0.f), ps2b = make_float2(0.f, 0.f);
                    // P's buffer is free: S(it) was committed behind the P V before last
#pragma unroll
                    for (int part = 0; part < 2; ++part) {
                        uint32_t w[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const int i = 32 * part + 2 * e;
                            const float2 arg = ffma2(make_float2(x[i], x[i + 1]), cc, nm);
                            const float2 pr = make_float2(fast_exp2(arg.x), fast_exp2(arg.y));
                            if (e & 1)
                                ps2b = fadd2(ps2b, pr);
                            else
                                ps2a = fadd2(ps2a, pr);
                            if (FP8) {
                                const __half2 v2 = __floats2half2_rn(pr.x, pr.y);
                                w[e] = *reinterpret_cast<const uint32_t *>(&v2);
                            } else {
                                const __nv_bfloat162 v2 = __floats2bfloat162_rn(pr.x, pr.y);
                                w[e] = *reinterpret_cast<const uint32_t *>(&v2);
                            }
                        }
                        tmem_st16(t_p + 32 * b + 16 * part, w);
                    }
                    const float alpha = m_new == m_ref ? 1.f : fast_exp2(m_ref - m_new);
                    const bool moved = it > it0 && __any_sync(0xffffffffu, alpha != 1.f);
                    l_run = l_run * alpha + ((ps2a.x + ps2b.x) + (ps2a.y + ps2b.y));
                    m_ref = m_new;
                    // rescale O where the reference moved, once O += P(it - 1) V(it - 1) is done
                    if (moved) {
                        if (!(ok = warp_wait(&B.pv_free[b ^ 1u], ((g - 1) >> 1) & 1u, abort_flag, a.status))) break;
                        tc_fence_after();
#pragma unroll 1
                        for (int cb = 0; cb < D / 32; ++cb) {
                            float o[32];
                            tmem_ld32(t_o + cb * 32, o);
#pragma unroll
                            for (int i = 0; i < 32; ++i) o[i] *= alpha;
                            tmem_st32(t_o + cb * 32, o);
                        }
                    }
                    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                }
                // V rows that hold no token (past the context, or of a bad block) may be anything: zero, so that
                // P = 0 there multiplies zeros. A draft's V that is not finite is hidden from the rows that do not
                // see it in the same way, and added back to the others at the end.
                if (tail || bad) {
                    const int st = g % kStagesV;
                    if (!(ok = warp_wait(&B.v_full[st], (g / kStagesV) & 1u, abort_flag, a.status))) break;
                    uint8_t *vt = sv + st * Sh::kTileV;
                    constexpr uint32_t kOdd = FP8 ? 0x7c00u : 0x7f80u;  // exponent of an infinity or a NaN
                    const int lo = bad ? 0 : max(first - t0, 0);  // rows before are committed tokens
#pragma unroll 1
                    for (int e = r; e < HALVES * (kTokens - lo) * 8; e += 128) {
                        const int tok = lo + e / (HALVES * 8), hf = e / 8 % HALVES, ch = e % 8;
                        uint4 *at = reinterpret_cast<uint4 *>(vt + hf * Sh::kHalfKV + tok * 128 + ((ch ^ (tok & 7)) << 4));
                        if (t0 + tok >= now.L || ((bad >> (tok / BS)) & 1u)) {
                            *at = make_uint4(0u, 0u, 0u, 0u);
                        } else if (t0 + tok >= first) {
                            uint4 v = *at;
                            uint32_t *w = &v.x;
                            bool any = false;
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                if ((w[i] & kOdd) == kOdd) {
                                    w[i] &= 0xffff0000u;
                                    any = true;
                                }
                                if ((w[i] & (kOdd << 16)) == kOdd << 16) {
                                    w[i] &= 0x0000ffffu;
                                    any = true;
                                }
                            }
                            if (any) {
                                poison[slot] = 1;
                                *at = v;
                            }
                        }
                    }
                    fence_proxy_async_shared();
                }
                tc_fence_before();
                signal(&B.p_ready[b]);
            }
            if (!ok) break;
            // ---- the piece's end. Of a segment cut in two, whoever gets here first leaves its partial and goes on; the
            // other joins the two from its registers (it waits, if at all, for stores already under way).
            const bool head = it0 == 0, whole = head && it1 == now.nit;
            int other = -1;  // the CTA of the other piece, where there are two
            if (!whole) {
                const int end = now.x + now.nit - it1;  // the segment's end
                if (head && end <= B.bound_next)
                    other = c + 1;
                else if (!head && it1 == now.nit && now.x - it1 >= B.bound_prev)
                    other = c - 1;
                else if (head && r == 0)
                    a.cuts[c] = make_int4(now.q0 + now.i0, now.n - now.i0, now.h,
                                          static_cast<int>((static_cast<int64_t>(end - B.start) * B.ctas - 1) / B.total) -
                                              B.index + 1);
            }
            unsigned *count = a.arrivals + (head ? c : c - 1);
            if (other >= 0 && r == 0) B.arrived[slot] = static_cast<int>(atomicAdd(count, 1u) & 15u);
            bool join = false;
            if (other >= 0) {
                if (!meet_all()) break;  // all know which comes first
                join = *reinterpret_cast<volatile int *>(&B.arrived[slot]) != 0;
            }
            const bool store = !whole && !join;
            const int64_t own_row = (c * 2 + (head ? 1 : 0)) * static_cast<int64_t>(kRows);
            const int64_t other_row = (other * 2 + (head ? 0 : 1)) * static_cast<int64_t>(kRows);
            const float4 *other_part = reinterpret_cast<const float4 *>(a.o_part + other_row * D) + r;
            float scale_mine = l_run == 0.f ? 0.f : 1.f / l_run, scale_other = 0.f;
            float4 v[4];  // the other piece's next 16 columns, asked for ahead: one by one, they wait in turn
            if (join) {
                if (!(ok = wait_stored(count, abort_flag, a.status))) break;
                const float2 ml = a.ml_part[other_row + r];
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = other_part[i * kRows];
                const float m = fmaxf(m_ref, ml.x);
                const float w0 = m_ref == -INFINITY ? 0.f : fast_exp2(m_ref - m);
                const float w1 = ml.x == -INFINITY ? 0.f : fast_exp2(ml.x - m);
                // the same whichever piece comes second: products and sums rounded one by one
                const float l = __fadd_rn(__fmul_rn(l_run, w0), __fmul_rn(ml.y, w1));
                const float inv = l == 0.f ? 0.f : 1.f / l;
                scale_mine = w0 * inv;
                scale_other = w1 * inv;
            } else if (store && live) {
                a.ml_part[own_row + r] = make_float2(m_ref, l_run);
            }
            if (!(ok = warp_wait(&B.o_full, piece & 1u, abort_flag, a.status))) break;
            tc_fence_after();
            const bool poisoned = poison[slot] != 0;
            if (poisoned) {
                if (!meet_all()) break;  // all have read the flag
                if (r == 0) poison[slot] = 0;
            }
            // a partial is [columns / 4][rows][4]: a warp's rows are side by side
            float4 *own_part = reinterpret_cast<float4 *>(a.o_part + own_row * D) + r;
            __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(a.out) +
                                 (static_cast<int64_t>(now.q0 + draft) * a.num_q_heads + now.h * G + r % G) * D;
            if (warp_live) {
#pragma unroll 1
                for (int col = 0; col < D; col += 16) {
                    float o[16];
                    tmem_ld16(t_o + col, o);
                    if (!live) continue;
                    if (FP8) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[i] *= v_scale;
                    }
                    if (store) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            own_part[(col / 4 + i) * kRows] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                        continue;
                    }
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[i] = __fmul_rn(o[i], scale_mine);
                    if (join) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            o[4 * i] = __fadd_rn(o[4 * i], __fmul_rn(v[i].x, scale_other));
                            o[4 * i + 1] = __fadd_rn(o[4 * i + 1], __fmul_rn(v[i].y, scale_other));
                            o[4 * i + 2] = __fadd_rn(o[4 * i + 2], __fmul_rn(v[i].z, scale_other));
                            o[4 * i + 3] = __fadd_rn(o[4 * i + 3], __fmul_rn(v[i].w, scale_other));
                        }
                        if (col + 16 < D) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) v[i] = other_part[((col + 16) / 4 + i) * kRows];
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 16; i += 8) {
                        uint32_t w[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const __nv_bfloat162 v2 = __floats2bfloat162_rn(o[i + 2 * e], o[i + 2 * e + 1]);
                            w[e] = *reinterpret_cast<const uint32_t *>(&v2);
                        }
                        *reinterpret_cast<uint4 *>(dst + col + i) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
                if (poisoned && live) {
                    // the drafts of this piece whose V is not finite, for the rows that see them
                    const int j1 = min(it1 * kTokens - first, now.n);
#pragma unroll 1
                    for (int j = max(it0 * kTokens - first, 0); j < j1; ++j) {
                        if (!((bits[j >> 5] >> (j & 31)) & 1)) continue;
                        const int pos = first + j;
                        const int p = __ldg(a.block_tables + static_cast<int64_t>(now.s) * a.max_blocks_per_seq + pos / BS);
                        if (p < 0 || p >= a.num_blocks) continue;
                        const int64_t at = ((static_cast<int64_t>(p) * BS + pos % BS) * a.num_kv_heads + now.h) * D;
#pragma unroll 1
                        for (int d = 0; d < D; ++d) {
                            float f;
                            if (FP8)
                                f = (static_cast<const uint8_t *>(a.v_cache)[at + d] & 0x7fu) == 0x7fu ? NAN : 0.f;
                            else
                                f = __bfloat162float(static_cast<const __nv_bfloat16 *>(a.v_cache)[at + d]);
                            if (isfinite(f)) continue;
                            if (store)
                                reinterpret_cast<float *>(own_part + d / 4 * kRows)[d % 4] += f;
                            else
                                dst[d] = __float2bfloat16(__bfloat162float(dst[d]) + f);
                        }
                    }
                }
            }
            if (store && other >= 0) {  // stored: one mark per warp
                __threadfence();
                __syncwarp();
                if (lane == 0) atomicAdd(count, 16u);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMma) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tbase), "r"(kTmemCols));
    }
}

constexpr int kMergeThreads = 256, kMergeWarps = kMergeThreads / 32;
constexpr int kMergeCols = 16, kMergeQuads = kMergeCols / 4;
constexpr int kMergeCtas = 296;  // two per SM

// Joins the partials of the segments cut into more than two pieces: out = sum_p O_p 2^(m_p - m) / sum_p l_p 2^(m_p - m).
// cuts[c] holds the segment that CTA c begins; the following CTAs' first partials are its other pieces. Every CTA lists
// the segments and takes its share of their (32 rows, 16 columns) items; in an item a lane is a row and a warp every
// eighth piece, four of which it loads at once: the 37 pieces of a 32K context are two round trips. Also clears the
// two-piece counters for the next launch.
template <int D>
__global__ void __launch_bounds__(kMergeThreads) tree_merge_kernel(const TreeArgs a, int ctas, int row_chunks) {
    __shared__ int segments[kTreeMaxCtas];
    __shared__ unsigned marks[kTreeMaxCtas / 32];
    __shared__ float2 ml_s[kMergeWarps][32];
    __shared__ float4 o_s[kMergeWarps][kMergeQuads][32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    depend_wait();
    depend_release();
    for (int k = warp; k < kTreeMaxCtas / 32; k += kMergeWarps) {
        const int c = k * 32 + lane;
        const unsigned m = __ballot_sync(0xffffffffu, c < ctas && a.cuts[c].w != 0);
        if (lane == 0) marks[k] = m;
        if (blockIdx.x == 0 && c < ctas) a.arrivals[c] = 0;
    }
    __syncthreads();
    int count = 0;  // the list is in the CTAs' order: the same in every merge CTA
#pragma unroll
    for (int k = 0; k < kTreeMaxCtas / 32; ++k) {
        if (k % kMergeWarps == warp && (marks[k] >> lane & 1u))
            segments[count + __popc(marks[k] & ((1u << lane) - 1u))] = k * 32 + lane;
        count += __popc(marks[k]);
    }
    __syncthreads();
    const int per_segment = row_chunks * (D / kMergeCols), items = count * per_segment;
    for (int item = blockIdx.x; item < items; item += gridDim.x) {
        const int c = segments[item / per_segment], rest = item % per_segment;
        const int r = rest / (D / kMergeCols) * 32 + lane, col = rest % (D / kMergeCols) * kMergeCols;
        const int4 cut = a.cuts[c];  // first row's draft, drafts from there on, kv head, pieces
        const bool live = r < min(cut.y, a.tile_drafts) * a.group;
        auto partial = [&](int p) { return ((c + p) * 2 + (p == 0 ? 1 : 0)) * static_cast<int64_t>(kRows); };
        float m = -INFINITY, l = 0.f;
        float4 o[kMergeQuads];
#pragma unroll
        for (int i = 0; i < kMergeQuads; ++i) o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (live) {
            for (int p0 = warp; p0 < cut.w; p0 += 4 * kMergeWarps) {
                float2 ml[4];
                float4 v[4][kMergeQuads];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int p = p0 + k * kMergeWarps;
                    if (p >= cut.w) break;
                    ml[k] = a.ml_part[partial(p) + r];
                    const float4 *part = reinterpret_cast<const float4 *>(a.o_part + partial(p) * D) + col / 4 * kRows + r;
#pragma unroll
                    for (int i = 0; i < kMergeQuads; ++i) v[k][i] = part[i * kRows];
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if (p0 + k * kMergeWarps >= cut.w) break;
                    const float top = fmaxf(m, ml[k].x);
                    const float keep = m == -INFINITY ? 0.f : fast_exp2(m - top);
                    const float w = ml[k].x == -INFINITY ? 0.f : fast_exp2(ml[k].x - top);
                    m = top;
                    l = l * keep + ml[k].y * w;
#pragma unroll
                    for (int i = 0; i < kMergeQuads; ++i) {
                        o[i].x = o[i].x * keep + v[k][i].x * w;
                        o[i].y = o[i].y * keep + v[k][i].y * w;
                        o[i].z = o[i].z * keep + v[k][i].z * w;
                        o[i].w = o[i].w * keep + v[k][i].w * w;
                    }
                }
            }
        }
        ml_s[warp][lane] = make_float2(m, l);
#pragma unroll
        for (int i = 0; i < kMergeQuads; ++i) o_s[warp][i][lane] = o[i];
        __syncthreads();
        if (warp >= kMergeQuads) {  // warp w < 4 joins the eight sums of columns 4 w .. 4 w + 3
            __syncthreads();
            continue;
        }
        float top = -INFINITY, sum = 0.f;
        float4 q = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < kMergeWarps; ++k) top = fmaxf(top, ml_s[k][lane].x);
#pragma unroll
        for (int k = 0; k < kMergeWarps; ++k) {
            const float2 ml = ml_s[k][lane];
            const float w = ml.x == -INFINITY ? 0.f : fast_exp2(ml.x - top);
            const float4 v = o_s[k][warp][lane];
            sum += ml.y * w;
            q.x += v.x * w;
            q.y += v.y * w;
            q.z += v.z * w;
            q.w += v.w * w;
        }
        if (live) {
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            const __nv_bfloat162 lo = __floats2bfloat162_rn(q.x * inv, q.y * inv), hi = __floats2bfloat162_rn(q.z * inv, q.w * inv);
            *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.out) +
                                       (static_cast<int64_t>(cut.x + r / a.group) * a.num_q_heads + cut.z * a.group +
                                        r % a.group) * D + col + 4 * warp) =
                make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
        }
        __syncthreads();
    }
}

template <int D, bool FP8>
size_t tree_smem_bytes(int entries) {
    const size_t bytes = TreeShape<D, FP8>::kOperands + sizeof(TreeBars) + (static_cast<size_t>(entries) + 1) * 4 + 1024;
    return bytes < 80 * 1024 ? 80 * 1024 : bytes;  // not more than two CTAs per SM: tensor memory holds no more
}

template <int D, int BS, bool FP8>
cudaError_t launch(const CUtensorMap &tm_q, const CUtensorMap &tm_k, const CUtensorMap &tm_v, const TreeArgs &a,
                   int ctas, cudaStream_t stream) {
    const size_t smem = tree_smem_bytes<D, FP8>(a.num_seqs * a.lists);
    auto *fn = paged_tree_kernel<D, BS, FP8>;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    static std::atomic<uint64_t> prepared{0};  // devices whose limit is set, to the largest that a launch asks for
    const uint64_t bit = 1ull << (dev & 63);
    if (dev > 63 || !(prepared.load() & bit)) {
        const size_t most = tree_smem_bytes<D, FP8>(2 * (FP8 ? kTreeMaxSeqsFp8 : kTreeMaxSeqs));
        e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(most));
        if (e != cudaSuccess) return e;
        prepared |= bit;
    }
    e = launch_overlapped(fn, dim3(ctas), TreeShape<D, FP8>::kThreads, smem, 1, stream, tm_q, tm_k, tm_v, a);
    if (e != cudaSuccess || a.whole || ctas == 1) return e;
    const int rows = (a.max_query_len < a.tile_drafts ? a.max_query_len : a.tile_drafts) * a.group;
    const int row_chunks = (rows + 31) / 32, most = ctas / 2 * row_chunks * (D / kMergeCols);  // three pieces or more each
    return launch_overlapped(tree_merge_kernel<D>, dim3(most < kMergeCtas ? most : kMergeCtas), kMergeThreads, 0, 1,
                             stream, a, ctas, row_chunks);
}

template <bool FP8>
cudaError_t launch_any(int D, const CUtensorMap &tm_q, const CUtensorMap &tm_k, const CUtensorMap &tm_v,
                       const TreeArgs &a, int ctas, cudaStream_t stream) {
    if (D == 64) return a.block_size == 16 ? launch<64, 16, FP8>(tm_q, tm_k, tm_v, a, ctas, stream)
                                           : launch<64, 32, FP8>(tm_q, tm_k, tm_v, a, ctas, stream);
    return a.block_size == 16 ? launch<128, 16, FP8>(tm_q, tm_k, tm_v, a, ctas, stream)
                              : launch<128, 32, FP8>(tm_q, tm_k, tm_v, a, ctas, stream);
}

}  // namespace

cudaError_t tree_launch(bool fp8, int head_dim, const CUtensorMap &tm_q, const CUtensorMap &tm_k,
                        const CUtensorMap &tm_v, const TreeArgs &a, int ctas, cudaStream_t stream) {
    return fp8 ? launch_any<true>(head_dim, tm_q, tm_k, tm_v, a, ctas, stream)
               : launch_any<false>(head_dim, tm_q, tm_k, tm_v, a, ctas, stream);
}

}  // namespace pkv
