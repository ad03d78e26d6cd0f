// tree.cu -- attention of drafted trees over the paged cache (tcgen05).
//
// Sequence s brings n_s drafted tokens, the last n_s of its L_s cached ones.
// Draft i sees the committed positions 0 .. L_s - n_s - 1 and the drafts its
// mask row names: out = sum_j e^(scale q.k_j) v_j / sum_j e^(scale q.k_j) over
// what it sees, zero where it sees nothing.
//
// A row is a (draft, query head of the kv head's group) pair: 128 / G drafts
// make a row tile, and one pass over a sequence's K and V serves a row group
// of TILES row tiles (1: two CTAs per SM; 2, for trees of more rows: one CTA
// per SM). Sequences, kv heads and row groups make segments of 64-token
// iterations; the CTAs of one wave take equal shares of all iterations (plus a
// fixed cost per segment), so a long context is cut between many CTAs and short
// ones are strung together in one. A cut segment leaves fp32 partials (O, the
// maximum and the sum of each row), which tree_merge_kernel joins.
//
// Roles, each walking the CTA's share on its own: one warp brings Q and K by
// TMA, one V, one per row tile issues its MMAs (S = Q K^T into tensor memory, O +=
// P V with P read from there), and four warps per row tile hold a row per thread: they
// load its 64 logits, hide what the row does not see, keep the running maximum
// and sum in fp32, and write P in bf16 beside S. The mask only matters in the
// iterations that reach past the committed tokens: a row's bits for 64 positions
// are two words there.
#include <cuda_bf16.h>

#include "device_utils.cuh"
#include "launch.h"
#include "tcgen05_utils.cuh"

namespace pkv {
namespace {

constexpr int kRows = 128;       // rows of a tile (= tensor-memory lanes)
constexpr int kTokens = 64;      // positions of one iteration
constexpr int kBadRing = 8;      // iterations whose bad-block bits are kept (a loader is at most 5 ahead)
constexpr int kPoisonRing = 16;  // pieces whose flag is kept (one tile's warps are at most 6 ahead of the other's)

// A CTA's share of the step, piece by piece (a piece: consecutive iterations of
// one segment). Every role walks it alike.
struct Walk {
    int64_t x, x1;  // weight position, end of the share
    int s;
    int q0, n, L, h, i0;  // the piece's sequence, kv head and first draft
    int nit, it0, it1;    // iterations of its segment, and of the piece
    int it;

    __device__ __forceinline__ bool next_piece(const TreeArgs &a, const int64_t *wp) {
        while (x < x1) {
            while (wp[s + 1] <= x) ++s;
            q0 = __ldg(a.query_start + s);
            n = __ldg(a.query_start + s + 1) - q0;
            L = __ldg(a.context_lens + s);
            nit = (L + kTokens - 1) / kTokens;
            const int64_t w = nit + a.piece_cost, local = x - wp[s], seg = local / w;
            const int off = static_cast<int>(local - seg * w);
            int end = static_cast<int>(w);
            if (a.whole) {
                if (off > 0) {  // the segment began in another CTA's share
                    x += w - off;
                    continue;
                }
            } else if (w - off > x1 - x) {
                end = off + static_cast<int>(x1 - x);
            }
            x += end - off;
            it0 = max(0, off - a.piece_cost);
            it1 = max(0, end - a.piece_cost);
            if (it1 > it0) {
                const int groups = (n + a.group_drafts - 1) / a.group_drafts;
                h = static_cast<int>(seg / groups);
                i0 = static_cast<int>(seg % groups) * a.group_drafts;
                it = it0;
                return true;
            }
        }
        return false;
    }
    // The next iteration (of this piece or the next one).
    __device__ __forceinline__ bool next(const TreeArgs &a, const int64_t *wp) {
        return ++it < it1 || next_piece(a, wp);
    }
    // Row tiles with a live row.
    __device__ __forceinline__ int tiles(const TreeArgs &a) const {
        return min(a.group_drafts, n - i0) > a.tile_drafts ? 2 : 1;
    }
};

// The 64 visibility bits of a mask row (n drafts, committed positions before
// them) for positions t0 .. t0 + 63; t0 is below the context's end and t0 + 63
// at or past its first draft.
__device__ __forceinline__ uint64_t visible_bits(const int32_t *row, int n, int first, int t0) {
    const int j0 = t0 - first;  // draft of bit 0 (negative: committed positions before)
    const int w0 = max(j0, 0) >> 5, words = (n + 31) >> 5;
    uint32_t w[3];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        w[k] = w0 + k < words ? static_cast<uint32_t>(__ldg(row + w0 + k)) : 0u;
        const int left = n - 32 * (w0 + k);  // drafts from this word on
        if (left < 32) w[k] = left > 0 ? w[k] & ((1u << left) - 1u) : 0u;
    }
    if (j0 >= 0) {
        const int sh = j0 & 31;
        const uint32_t lo = __funnelshift_r(w[0], w[1], sh), hi = __funnelshift_r(w[1], w[2], sh);
        return (static_cast<uint64_t>(hi) << 32) | lo;
    }
    const uint64_t bits = (static_cast<uint64_t>(w[1]) << 32) | w[0];
    return j0 <= -64 ? ~0ull : (bits << -j0) | ((1ull << -j0) - 1ull);
}

template <int D>
struct TreeShape {
    static constexpr int HALVES = D / 64;                     // 128-byte column slices of a row
    static constexpr uint32_t kHalfKV = kTokens * 128;
    static constexpr uint32_t kTileKV = HALVES * kHalfKV;     // K (or V) of one stage
    static constexpr uint32_t kQHalf = kRows * 128;
    static constexpr uint32_t kTileQ = HALVES * kQHalf;
};

constexpr int tree_stages(int tiles) { return tiles == 1 ? 2 : 4; }
constexpr int tree_threads(int tiles) { return tiles * 160 + 64; }

struct TreeBars {
    uint64_t q_full, q_empty, done[2];
    uint64_t k_full[4], k_empty[4], v_full[4], v_empty[4];
    // per tile: S is in tensor memory; the softmax threads have loaded it; P (buffer b) is written; O += P V
    // of buffer b is done; the piece's O is done
    uint64_t s_full[2], s_free[2], p_ready[2][2], pv_free[2][2], o_full[2];
    int64_t scan[16];
    uint32_t bad[kBadRing];
    uint32_t tmem;
    int abort;
    int poison[kPoisonRing];
};

template <int D, int BS, int TILES>
__global__ void __launch_bounds__(tree_threads(TILES), TILES == 1 ? 2 : 1)
    paged_tree_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const TreeArgs a) {
    using Sh = TreeShape<D>;
    constexpr int HALVES = Sh::HALVES, BPI = kTokens / BS, STAGES = tree_stages(TILES);
    constexpr int kThreads = tree_threads(TILES), kLoadK = 4 * TILES, kLoadV = kLoadK + 1, kMma = kLoadK + 2;
    constexpr uint32_t kTmemCols = 256 * TILES;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    // ---- shared memory: Q tiles | K stages | V stages | barriers | weights before each sequence
    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sq = base;
    uint8_t *sk = sq + TILES * Sh::kTileQ;
    uint8_t *sv = sk + STAGES * Sh::kTileKV;
    TreeBars &B = *reinterpret_cast<TreeBars *>(sv + STAGES * Sh::kTileKV);
    int64_t *wp = reinterpret_cast<int64_t *>(&B + 1);

    // ---- weights: every CTA sums over all sequences (one contiguous run per thread)
    {
        const int per = (a.num_seqs + kThreads - 1) / kThreads;
        const int s0 = min(tid * per, a.num_seqs), s1 = min(s0 + per, a.num_seqs);
        int64_t sum = 0;
        for (int s = s0; s < s1; ++s) {
            const int q0 = __ldg(a.query_start + s), n = __ldg(a.query_start + s + 1) - q0;
            const int L = __ldg(a.context_lens + s);
            int64_t w = 0;
            if (q0 < 0 || n < 0 || q0 > a.num_tokens - n || n > a.max_query_len || n > L ||
                L > static_cast<int64_t>(a.max_blocks_per_seq) * BS) {
                if (blockIdx.x == 0) atomicOr(a.status, PKV_STATUS_BAD_CONTEXT_LEN);
            } else if (n > 0) {
                w = static_cast<int64_t>(a.num_kv_heads) * ((n + a.group_drafts - 1) / a.group_drafts) *
                    ((L + kTokens - 1) / kTokens + a.piece_cost);
            }
            wp[s + 1] = w;
            sum += w;
        }
        int64_t inc = sum;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, inc, d);
            if (lane >= d) inc += y;
        }
        if (lane == 31) B.scan[warp] = inc;
        __syncthreads();
        int64_t run = inc - sum;
        for (int w = 0; w < warp; ++w) run += B.scan[w];
        for (int s = s0; s < s1; ++s) {
            run += wp[s + 1];
            wp[s + 1] = run;
        }
        if (tid == 0) {
            wp[0] = 0;
            if (!a.whole) a.cuts[blockIdx.x] = make_int4(0, 0, 0, 0);
        }
    }
    __syncthreads();
    const int64_t W = wp[a.num_seqs];
    const int64_t most = (W + a.min_weight - 1) / a.min_weight;
    const int C = static_cast<int>(most < gridDim.x ? most : gridDim.x);  // CTAs that take a share
    const int c = blockIdx.x;
    if (c >= C) return;
    Walk walk;
    walk.x = W * c / C;
    walk.x1 = W * (c + 1) / C;
    {
        int lo = 0, hi = a.num_seqs;  // wp[lo] <= x < wp[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (wp[mid] <= walk.x)
                lo = mid;
            else
                hi = mid;
        }
        walk.s = lo;
    }

    if (warp == kMma) {  // all of the CTA's columns
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&B.tmem)),
                     "r"(kTmemCols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::);
        tc_fence_before();
    } else if (warp == kLoadK && lane == 0) {
        mbar_init(&B.q_full, 1);
        mbar_init(&B.q_empty, TILES);
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(&B.k_full[i], 1);
            mbar_init(&B.k_empty[i], TILES);
            mbar_init(&B.v_full[i], 1);
            mbar_init(&B.v_empty[i], TILES);
        }
        for (int t = 0; t < TILES; ++t) {
            mbar_init(&B.done[t], 1);
            mbar_init(&B.s_full[t], 1);
            mbar_init(&B.s_free[t], 128);
            for (int i = 0; i < 2; ++i) {
                mbar_init(&B.p_ready[t][i], 128);
                mbar_init(&B.pv_free[t][i], 1);
            }
            mbar_init(&B.o_full[t], 1);
        }
        for (int i = 0; i < kPoisonRing; ++i) B.poison[i] = 0;
        B.abort = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tm_q);
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
    }
    __syncthreads();
    tc_fence_after();
    volatile int *abort_flag = &B.abort;
    const uint32_t tbase = B.tmem;

    if (warp == kLoadK || warp == kLoadV) {
        // ---------------- load warps: lane j copies one 128-byte column slice of one block
        const bool is_v = warp == kLoadV;
        uint8_t *ring = is_v ? sv : sk;
        uint64_t *full = is_v ? B.v_full : B.k_full, *empty = is_v ? B.v_empty : B.k_empty;
        const int jb = lane / HALVES, hf = lane % HALVES;
        auto entry = [&](const Walk &w) {  // this lane's table entry of the iteration, -1: no such block
            const int b = w.it * BPI + jb;
            return lane < BPI * HALVES && b * BS < w.L
                       ? __ldg(a.block_tables + static_cast<int64_t>(w.s) * a.max_blocks_per_seq + b)
                       : -1;
        };
        uint32_t g = 0, pieces = 0;
        bool more = walk.next_piece(a, wp), ok = true, fresh = true, q_issued = false;
        int p = more ? entry(walk) : -1;
        while (more) {
            Walk ahead = walk;
            const bool more2 = ahead.next(a, wp);
            const int p2 = more2 ? entry(ahead) : -1;  // in flight while this iteration waits
            const int st = g % STAGES;
            if (g >= STAGES && !(ok = warp_wait(&empty[st], (g / STAGES - 1) & 1u, abort_flag, a.status))) break;
            const bool there = lane < BPI * HALVES && (walk.it * BPI + jb) * BS < walk.L;
            const bool mine = there && p >= 0 && p < a.num_blocks;
            const unsigned m = __ballot_sync(0xffffffffu, mine), lost = __ballot_sync(0xffffffffu, there && !mine);
            if (!is_v) {
                if (lost && lane == 0) atomicOr(a.status, PKV_STATUS_BAD_BLOCK_ID);
                if (lane == 0) B.bad[g % kBadRing] = lost;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive_expect_tx(&full[st], static_cast<uint32_t>(__popc(m)) * BS * 128u);
            __syncwarp();
            if (mine)
                tma_load_4d(ring + st * Sh::kTileKV + hf * Sh::kHalfKV + jb * BS * 128, is_v ? &tm_v : &tm_k,
                            &full[st], 0, hf, walk.h, p * BS);
            ++g;
            if (!is_v && fresh) {
                // the piece's queries, once the MMAs of the piece before are done with theirs
                if (pieces > 0 && !(ok = warp_wait(&B.q_empty, (pieces - 1) & 1u, abort_flag, a.status))) break;
                if (lane == 0) {
                    const int tiles = TILES == 1 ? 1 : walk.tiles(a);
                    mbar_arrive_expect_tx(&B.q_full, tiles * HALVES * a.tile_drafts * a.group * 128);
                    for (int t = 0; t < tiles; ++t)
#pragma unroll
                        for (int q = 0; q < HALVES; ++q)
                            tma_load_5d(sq + t * Sh::kTileQ + q * Sh::kQHalf, &tm_q, &B.q_full, 0, q, 0, walk.h,
                                        walk.q0 + walk.i0 + t * a.tile_drafts);
                }
                __syncwarp();
                q_issued = true;
                ++pieces;
            }
            fresh = more2 && ahead.it == ahead.it0;
            walk = ahead;
            more = more2;
            p = p2;
        }
        // copies still in flight (only after a wait gave up) land before exit
        if (!ok || *abort_flag) {
            if (q_issued) mbar_wait_drain(&B.q_full, (pieces - 1) & 1u, a.status);
            for (uint32_t u = g > STAGES ? g - STAGES : 0; u < g; ++u)
                mbar_wait_drain(&full[u % STAGES], (u / STAGES) & 1u, a.status);
        }
        __syncwarp();
    } else if (warp >= kMma) {
        // ---------------- MMA warp of tile t: one elected lane issues. S(it + 1) is issued as soon as the softmax
        // warps hold S(it) in registers, and runs while they work on it; O += P(it) V(it) follows P(it).
        const int t = TILES == 1 ? 0 : warp - kMma;
        const bool leader = elect_one();
        const uint64_t dq = smem_desc(smem_u32(sq + t * Sh::kTileQ), 16, 1024), dk = smem_desc(smem_u32(sk), 16, 1024),
                       dv = smem_desc(smem_u32(sv), Sh::kHalfKV, 1024);
        const uint32_t t_s = tbase + 256 * t, t_p = t_s + 64, t_o = t_s + 128;
        Walk ws = walk, wv = walk;
        uint32_t gs = 0, gv = 0, pieces = 0, us = 0, uv = 0;  // iterations, pieces; iterations with a live tile
        bool ok = true;
        auto step_s = [&]() {
            const int st = gs % STAGES;
            const bool last = ws.it + 1 == ws.it1, live = t < ws.tiles(a);
            if (ws.it == ws.it0) {
                if (!(ok = warp_wait(&B.q_full, pieces & 1u, abort_flag, a.status))) return;
                ++pieces;
            }
            if (!(ok = warp_wait(&B.k_full[st], (gs / STAGES) & 1u, abort_flag, a.status))) return;
            if (live) {
                if (us > 0 && !(ok = warp_wait(&B.s_free[t], (us - 1) & 1u, abort_flag, a.status))) return;
                tc_fence_after();
                if (leader) {
#pragma unroll
                    for (int hf = 0; hf < HALVES; ++hf)
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            umma(t_s, dq + ((hf * Sh::kQHalf + kk * 32) >> 4),
                                 dk + ((st * Sh::kTileKV + hf * Sh::kHalfKV + kk * 32) >> 4),
                                 instr_desc(128, kTokens, false), (hf | kk) != 0);
                    umma_commit(&B.s_full[t]);
                    umma_commit(&B.k_empty[st]);
                    if (last) umma_commit(&B.q_empty);
                }
                ++us;
            } else if (lane == 0) {
                mbar_arrive(&B.k_empty[st]);
                if (last) mbar_arrive(&B.q_empty);
            }
            __syncwarp();
            ++gs;
        };
        auto step_v = [&]() {
            const int st = gv % STAGES;
            const uint32_t b = uv & 1u;
            if (!(ok = warp_wait(&B.v_full[st], (gv / STAGES) & 1u, abort_flag, a.status))) return;
            if (t < wv.tiles(a)) {
                if (!(ok = warp_wait(&B.p_ready[t][b], (uv >> 1) & 1u, abort_flag, a.status))) return;
                tc_fence_after();
                if (leader) {
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        umma_ts(t_o, t_p + 32 * b + kk * 8, dv + ((st * Sh::kTileKV + kk * 16 * 128) >> 4),
                                instr_desc(128, D, true), wv.it != wv.it0 || kk != 0);
                    umma_commit(&B.pv_free[t][b]);
                    umma_commit(&B.v_empty[st]);
                    if (wv.it + 1 == wv.it1) umma_commit(&B.o_full[t]);
                }
                ++uv;
            } else if (lane == 0) {
                mbar_arrive(&B.v_empty[st]);
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
            if (more_s) {
                step_s();
                if (!ok) break;
                more_s = ws.next(a, wp);
            }
            step_v();
            if (!ok) break;
            more_v = wv.next(a, wp);
        }
        // every MMA issued is done before the tensor memory is freed (one phase: nothing aliases)
        if (leader) umma_commit(&B.done[t]);
        __syncwarp();
        mbar_wait_drain(&B.done[t], 0, a.status);
        __syncwarp();
    } else {
        // ---------------- softmax warps: thread r of tile t owns a row (tensor-memory lane r)
        const int t = TILES == 1 ? 0 : warp >> 2, r = tid & 127, wlane = (warp & 3) * 32;
        const uint32_t t_s = tbase + 256 * t + (static_cast<uint32_t>(wlane) << 16), t_p = t_s + 64, t_o = t_s + 128;
        const int G = a.group, row_draft = t * a.tile_drafts + r / G;  // draft of this row within the row group
        const float c2 = fabsf(a.scale_log2);
        const bool negative = a.scale_log2 < 0.f, spare = r >= a.tile_drafts * G;
        volatile int *poison = B.poison;
        uint32_t u = 0, g = 0, mine = 0, pieces = 0;
        bool ok = true;
        while (ok && walk.next_piece(a, wp)) {
            const uint32_t piece = pieces++;
            if (t >= walk.tiles(a)) {  // no live row in this tile
                g += walk.it1 - walk.it0;
                continue;
            }
            const int draft = walk.i0 + row_draft;
            const bool live = !spare && row_draft < a.group_drafts && draft < walk.n;
            const bool warp_live = __any_sync(0xffffffffu, live);
            const int first = walk.L - walk.n;  // first draft's position
            const int32_t *bits = a.tree_mask + static_cast<int64_t>(walk.q0 + min(draft, walk.n - 1)) * a.mask_words;
            float m_ref = -INFINITY, l_run = 0.f;
            for (int it = walk.it0; it < walk.it1; ++it, ++u, ++g) {
                const uint32_t b = u & 1u;
                const int t0 = it * kTokens;
                if (!(ok = warp_wait(&B.s_full[t], u & 1u, abort_flag, a.status))) break;
                const uint32_t bad = B.bad[g % kBadRing];
                const bool tail = t0 + kTokens > first;
                if (!warp_live) {
                    mbar_arrive(&B.s_free[t]);
                } else {
                    tc_fence_after();
                    float x[64];
                    tmem_ld64(t_s, x);
                    tc_fence_before();
                    mbar_arrive(&B.s_free[t]);
                    if (negative) {
#pragma unroll
                        for (int i = 0; i < 64; ++i) x[i] = -x[i];
                    }
                    if (tail || bad) {
                        uint64_t vis = tail ? visible_bits(bits, walk.n, first, t0) : ~0ull;
                        if (bad) {
#pragma unroll
                            for (int k = 0; k < BPI; ++k)
                                if ((bad >> (k * HALVES)) & 1u) vis &= ~(((1ull << BS) - 1ull) << (k * BS));
                        }
                        const uint32_t lo = static_cast<uint32_t>(vis), hi = static_cast<uint32_t>(vis >> 32);
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            if (!((lo >> i) & 1u)) x[i] = -INFINITY;
                            if (!((hi >> i) & 1u)) x[32 + i] = -INFINITY;
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
                    // the reference moves only when it would be exceeded by more than 2^8
                    float m_new = m_ref;
                    if (mx * c2 > m_ref + 8.f) m_new = mx * c2;
                    const float alpha = m_new == m_ref ? 1.f : fast_exp2(m_ref - m_new);
                    const float shift = m_new == -INFINITY ? 0.f : -m_new;  // a row that has seen nothing: P = 0
                    const float2 cc = make_float2(c2, c2), nm = make_float2(shift, shift);
                    float2 ps2a = make_float2(0.f, 0.f), ps2b = make_float2(0.f, 0.f);
                    if (u >= 2 && !(ok = warp_wait(&B.pv_free[t][b], ((u >> 1) - 1) & 1u, abort_flag, a.status))) break;
                    tc_fence_after();
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        uint32_t w[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const int i = 32 * half + 2 * e;
                            const float2 arg = ffma2(make_float2(x[i], x[i + 1]), cc, nm);
                            const float2 pr = make_float2(fast_exp2(arg.x), fast_exp2(arg.y));
                            if (e & 1)
                                ps2b = fadd2(ps2b, pr);
                            else
                                ps2a = fadd2(ps2a, pr);
                            const __nv_bfloat162 v2 = __floats2bfloat162_rn(pr.x, pr.y);
                            w[e] = *reinterpret_cast<const uint32_t *>(&v2);
                        }
                        tmem_st16(t_p + 32 * b + 16 * half, w);
                    }
                    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                    l_run = l_run * alpha + ((ps2a.x + ps2b.x) + (ps2a.y + ps2b.y));
                    m_ref = m_new;
                    // rescale O where the reference moved, once O += P(it - 1) V(it - 1) is done
                    if (it > walk.it0 && __any_sync(0xffffffffu, alpha != 1.f)) {
                        if (!(ok = warp_wait(&B.pv_free[t][b ^ 1u], ((u - 1) >> 1) & 1u, abort_flag, a.status))) break;
                        tc_fence_after();
#pragma unroll
                        for (int cb = 0; cb < D / 32; ++cb) {
                            float o[32];
                            tmem_ld32(t_o + cb * 32, o);
#pragma unroll
                            for (int i = 0; i < 32; ++i) o[i] *= alpha;
                            tmem_st32(t_o + cb * 32, o);
                        }
                    }
                }
                // V rows that hold no token (past the context, or of a bad block) may be anything: zero, so that
                // P = 0 there multiplies zeros. A draft's V that is not finite is hidden from the rows that do not
                // see it in the same way, and added back to the others at the end. Each tile's warps do so before
                // their own P V; both write the same bytes, the flag always before the first of them.
                if (tail || bad) {
                    const int st = g % STAGES;
                    if (!(ok = warp_wait(&B.v_full[st], (g / STAGES) & 1u, abort_flag, a.status))) break;
                    uint8_t *vt = sv + st * Sh::kTileKV;
                    for (int e = r; e < HALVES * kTokens * 8; e += 128) {
                        const int hf = e / (kTokens * 8), tok = (e / 8) % kTokens, ch = e % 8;
                        uint4 *at = reinterpret_cast<uint4 *>(vt + hf * Sh::kHalfKV + tok * 128 + ((ch ^ (tok & 7)) << 4));
                        if (t0 + tok >= walk.L || ((bad >> (tok / BS * HALVES)) & 1u)) {
                            *at = make_uint4(0u, 0u, 0u, 0u);
                        } else if (t0 + tok >= first) {
                            uint4 v = *at;
                            uint32_t *w = &v.x;
                            bool any = false;
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                if ((w[i] & 0x7f80u) == 0x7f80u) {
                                    w[i] &= 0xffff0000u;
                                    any = true;
                                }
                                if ((w[i] & 0x7f800000u) == 0x7f800000u) {
                                    w[i] &= 0x0000ffffu;
                                    any = true;
                                }
                            }
                            if (any) {
                                poison[piece % kPoisonRing] = 1;
                                __threadfence_block();
                                *at = v;
                            }
                        }
                    }
                    __threadfence_block();
                    fence_proxy_async_shared();
                }
                tc_fence_before();
                mbar_arrive(&B.p_ready[t][b]);
            }
            if (!ok) break;
            if (!(ok = warp_wait(&B.o_full[t], mine & 1u, abort_flag, a.status))) break;
            ++mine;
            tc_fence_after();
            if (*abort_flag) break;
            const bool poisoned = poison[piece % kPoisonRing] != 0;
            if (t == 0 && r == 0) poison[(piece + kPoisonRing / 2) % kPoisonRing] = 0;
            const bool cut = walk.it0 > 0 || walk.it1 < walk.nit;
            const int64_t row = static_cast<int64_t>(c) * 2 + (walk.it0 > 0 ? 0 : 1);  // the CTA's partial
            float *part = nullptr;
            __nv_bfloat16 *dst = nullptr;
            if (cut) {
                const int64_t pr = row * (TILES * kRows) + t * kRows + r;
                part = a.o_part + pr * D;
                if (live) a.ml_part[pr] = make_float2(m_ref, l_run);
                if (t == 0 && r == 0 && walk.it0 == 0) {
                    // the segment's first piece: its last iteration's weight position tells how many follow
                    const int64_t w = walk.nit + a.piece_cost, left = w - (walk.it1 + a.piece_cost);
                    const int64_t last = walk.x + left - 1;
                    const int last_cta = static_cast<int>(((last + 1) * C - 1) / W);
                    a.cuts[c] = make_int4(walk.q0 + walk.i0, walk.n - walk.i0, walk.h, last_cta - c + 1);
                }
            } else {
                dst = static_cast<__nv_bfloat16 *>(a.out) +
                      (static_cast<int64_t>(walk.q0 + min(draft, walk.n - 1)) * a.num_q_heads + walk.h * G + r % G) * D;
            }
            const float inv = l_run == 0.f ? 0.f : 1.f / l_run;
            if (warp_live) {
#pragma unroll
                for (int cb = 0; cb < D / 32; ++cb) {
                    float o[32];
                    tmem_ld32(t_o + cb * 32, o);
                    if (poisoned && live) {
                        for (int j = max(walk.it0 * kTokens - first, 0); j < min(walk.it1 * kTokens - first, walk.n); ++j) {
                            if (!((bits[j >> 5] >> (j & 31)) & 1)) continue;
                            const int pos = first + j;
                            const int p = __ldg(a.block_tables + static_cast<int64_t>(walk.s) * a.max_blocks_per_seq + pos / BS);
                            if (p < 0 || p >= a.num_blocks) continue;
                            const __nv_bfloat16 *v = static_cast<const __nv_bfloat16 *>(a.v_cache) +
                                                     ((static_cast<int64_t>(p) * BS + pos % BS) * a.num_kv_heads + walk.h) * D +
                                                     cb * 32;
#pragma unroll
                            for (int i = 0; i < 32; ++i) {
                                const float f = __bfloat162float(v[i]);
                                if (!isfinite(f)) o[i] += f;
                            }
                        }
                    }
                    if (!live) continue;
                    if (cut) {
#pragma unroll
                        for (int i = 0; i < 32; i += 4)
                            *reinterpret_cast<float4 *>(part + cb * 32 + i) = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; i += 8) {
                            uint32_t w[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const __nv_bfloat162 v2 = __floats2bfloat162_rn(o[i + 2 * e] * inv, o[i + 2 * e + 1] * inv);
                                w[e] = *reinterpret_cast<const uint32_t *>(&v2);
                            }
                            *reinterpret_cast<uint4 *>(dst + cb * 32 + i) = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    }
                }
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

constexpr int kMergeWarps = 8;

// Joins the partials of a cut segment: out = sum_p O_p 2^(m_p - m) / sum_p l_p 2^(m_p - m). One warp per row;
// blockIdx.x is the CTA that holds the segment's first piece, the following CTAs' first partials are the others.
template <int D>
__global__ void __launch_bounds__(kMergeWarps * 32) tree_merge_kernel(const TreeArgs a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int c = blockIdx.x, lane = threadIdx.x & 31;
    const int4 cut = a.cuts[c];  // first row's draft, drafts from there on, kv head, pieces
    const int k = blockIdx.y * kMergeWarps + (threadIdx.x >> 5);
    if (cut.w == 0 || k >= min(cut.y, a.group_drafts) * a.group) return;
    constexpr int E = D / 32;
    const int tile_rows = a.tile_drafts * a.group;
    const int64_t rows = a.group_drafts > a.tile_drafts ? 2 * kRows : kRows;
    const int64_t at = k / tile_rows * kRows + k % tile_rows;  // the row's place in a partial
    auto partial = [&](int p) { return (static_cast<int64_t>(c + p) * 2 + (p == 0 ? 1 : 0)) * rows + at; };
    float m = -INFINITY;
    for (int p = lane; p < cut.w; p += 32) m = fmaxf(m, a.ml_part[partial(p)].x);
    for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    float o[E] = {}, l = 0.f;
    for (int p0 = 0; p0 < cut.w; p0 += 32) {
        const int count = min(32, cut.w - p0);
        float w = 0.f;
        if (lane < count) {
            const float2 ml = a.ml_part[partial(p0 + lane)];
            w = ml.x == -INFINITY ? 0.f : fast_exp2(ml.x - m);
            l += ml.y * w;
        }
#pragma unroll 4
        for (int p = 0; p < count; ++p) {
            const float wp = __shfl_sync(0xffffffffu, w, p);
            const float *src = a.o_part + partial(p0 + p) * D + lane * E;
            if (E == 4) {
                const float4 v = *reinterpret_cast<const float4 *>(src);
                o[0] += v.x * wp;
                o[1] += v.y * wp;
                o[E - 2] += v.z * wp;
                o[E - 1] += v.w * wp;
            } else {
                const float2 v = *reinterpret_cast<const float2 *>(src);
                o[0] += v.x * wp;
                o[1] += v.y * wp;
            }
        }
    }
    for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
    const float inv = l == 0.f ? 0.f : 1.f / l;
    __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(a.out) +
                         (static_cast<int64_t>(cut.x + k / a.group) * a.num_q_heads + cut.z * a.group + k % a.group) * D +
                         lane * E;
#pragma unroll
    for (int e = 0; e < E; e += 2)
        *reinterpret_cast<__nv_bfloat162 *>(dst + e) = __floats2bfloat162_rn(o[e] * inv, o[e + 1] * inv);
}

template <int D, int TILES>
size_t tree_smem_bytes(int num_seqs) {
    using Sh = TreeShape<D>;
    const size_t bytes = TILES * Sh::kTileQ + 2 * tree_stages(TILES) * Sh::kTileKV + sizeof(TreeBars) +
                         (static_cast<size_t>(num_seqs) + 1) * 8 + 1024;
    // not more CTAs per SM than its 512 tensor-memory columns hold
    return TILES == 1 ? (bytes < 80 * 1024 ? 80 * 1024 : bytes) : (bytes < 120 * 1024 ? 120 * 1024 : bytes);
}

template <int D, int BS, int TILES>
cudaError_t launch(const CUtensorMap &tm_q, const CUtensorMap &tm_k, const CUtensorMap &tm_v, const TreeArgs &a,
                   int ctas, cudaStream_t stream) {
    const size_t smem = tree_smem_bytes<D, TILES>(a.num_seqs);
    auto *fn = paged_tree_kernel<D, BS, TILES>;
    cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    fn<<<ctas, tree_threads(TILES), smem, stream>>>(tm_q, tm_k, tm_v, a);
    if ((e = cudaGetLastError()) != cudaSuccess || a.whole || ctas == 1) return e;
    const int rows = (a.max_query_len < a.group_drafts ? a.max_query_len : a.group_drafts) * a.group;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(ctas - 1, (rows + kMergeWarps - 1) / kMergeWarps);
    cfg.blockDim = dim3(kMergeWarps * 32);
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, tree_merge_kernel<D>, a);
}

template <int TILES>
cudaError_t launch_any(int D, int BS, const CUtensorMap &tm_q, const CUtensorMap &tm_k, const CUtensorMap &tm_v,
                       const TreeArgs &a, int ctas, cudaStream_t stream) {
    if (D == 64) return BS == 16 ? launch<64, 16, TILES>(tm_q, tm_k, tm_v, a, ctas, stream)
                                 : launch<64, 32, TILES>(tm_q, tm_k, tm_v, a, ctas, stream);
    return BS == 16 ? launch<128, 16, TILES>(tm_q, tm_k, tm_v, a, ctas, stream)
                    : launch<128, 32, TILES>(tm_q, tm_k, tm_v, a, ctas, stream);
}

}  // namespace

cudaError_t tree_launch(int head_dim, const CUtensorMap &tm_q, const CUtensorMap &tm_k, const CUtensorMap &tm_v,
                        const TreeArgs &a, int ctas, cudaStream_t stream) {
    return a.group_drafts > a.tile_drafts ? launch_any<2>(head_dim, a.block_size, tm_q, tm_k, tm_v, a, ctas, stream)
                                          : launch_any<1>(head_dim, a.block_size, tm_q, tm_k, tm_v, a, ctas, stream);
}

}  // namespace pkv
