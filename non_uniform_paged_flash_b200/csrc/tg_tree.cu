// Tree attention over the ragged paged cache: the verification step of speculative decoding. The
// drafted tokens of a sequence (up to 64, a tree or a chain) attend to the sequence's retained
// tokens, each KV head its own (Tangram's ragged paging), and to the drafted tokens that their
// mask names (their ancestors and themselves), whose keys and values are not in the cache yet.
//
//   s_t = scale q.k_t  (softcap c > 0: s_t <- c tanh(s_t / c)),
//   lse = ln sum_t exp(s_t),   out = sum_t exp(s_t - lse) v_t
// over the retained tokens t < head_kv_len and the drafted tokens with their mask bit set.
//
// Tree verification: Miao et al. 2023 (SpecInfer), Cai et al. 2024 (Medusa); online normaliser and
// its merge: CAP survey §2.4.3 "加速单个请求"; ragged page tables: "Tangram" 三大机制 2.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdio>
#include <cstring>
#include <memory>
#include <vector>

#include "tg.h"
#include "tg_internal.h"
#include "tg_ptx.cuh"

namespace tg {

// One work item: a page range of one (sequence, KV head) for one block of query rows. The item
// with the head's last pages also takes the drafted tokens.
struct TreeItem {
    int32_t bh;
    int32_t page_begin, page_end;
    int32_t slot;   // partial-result slot, -1: this item writes the final output
    int32_t row0;   // first query row (token * G + g) of the block
    int32_t draft;  // 1: takes the drafted tokens too
    int32_t cap;    // reserved tokens of the head
    int32_t pad;
};
static_assert(sizeof(TreeItem) == 32, "TreeItem is 32 bytes");

// A block of query rows whose head is split over nsplit >= 2 consecutive slots.
struct TreeMerge {
    int32_t bh, first_slot, nsplit, row0;
};

}  // namespace tg

struct tg_tree_plan {
    tg_shape shape{};
    int32_t G = 0, max_draft = 0, tiles = 1, m = 128;  // wide kernel: tiles of m rows
    bool host_only = true;
    bool any_pages = false;  // some head reserves a page
    int device = 0;
    uint64_t wait_ns = 4000000000ull;
    int32_t n_workers = 0;
    int32_t rows_item = 0;   // query rows of an item at most
    int32_t q_rows = 0;      // query rows that an item's Q load brings, per tile
    bool narrow = false;     // run by the narrow kernel
    int32_t smem_bytes = 0;
    int32_t n_slots = 0;
    std::vector<tg::TreeItem> items;      // each worker's items, then the dynamic ones
    std::vector<int32_t> worker_off;
    std::vector<tg::TreeMerge> merge;
    std::vector<int64_t> row_lo, row_hi;  // bounds of each KV head's group table

    void *dev_base = nullptr;
    int64_t dev_bytes = 0;
    tg::TreeItem *d_items = nullptr;
    int32_t *d_worker_off = nullptr;
    tg::TreeMerge *d_merge = nullptr;
    int64_t *d_row_lo = nullptr, *d_row_hi = nullptr;
    float *d_part_o = nullptr, *d_part_lse = nullptr;
    uint32_t *d_err = nullptr, *d_ticket = nullptr;  // d_ticket: next dynamic item, CTAs done
};

namespace tg {
namespace {

constexpr int kRows = 128;      // rows of a tile = tensor-memory lanes
constexpr int kBlock = 64;      // tokens of a block (4 pages)
constexpr int kHdr = 16;        // block headers kept
constexpr int kMaxEntries = 24; // ring entries at most: a header outlives its block (see the kernel)
constexpr int kCutPages = 4;    // heads are cut at whole blocks
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

// Block header flags.
constexpr int32_t kFirst = 1, kLast = 2, kDraft = 4, kStop = 8;
// The narrow kernel's, whose kFirst and kLast are per stream: the item's own ends, whether it takes the
// drafted tokens, and whether its first block is the second stream's.
constexpr int32_t kOpen = 16, kClose = 32, kTakesDraft = 64, kOdd = 128;

// What the block's consumers need to know, written by the producer before the block's K arrives.
struct alignas(16) BlockHdr {
    int32_t flags;  // | valid tokens << 8 | valid query rows of the item << 16
    int32_t tok0;   // the sequence's first drafted token
    int32_t h;      // KV head
    int32_t slot;   // partial-result slot or -1
    int32_t row0;   // first query row of the item
    int32_t v_fill; // ring fill (modulo 2 entries) that brings the block's V
    unsigned long long bad;  // drafted tokens whose V row holds an infinity or NaN
};
static_assert(sizeof(BlockHdr) == 32, "BlockHdr layout");

// Shared memory: a Q tile of M rows per tile, the K / V ring, block headers, barriers. Rows that the plan's
// drafts never use are zeros, so that they cost the products little power: the steps that the loads bound
// run under the power cap, whose clock goes down with what the padding rows multiply.
template <int D, int TILES, int M>
struct TreeLayout {
    static constexpr int kHalves = D / 64;             // 128-byte column halves
    static constexpr int kEntry = kBlock * D * 2;      // K or V of a block
    static constexpr int kGroup = 1024 * kHalves;      // 8 tokens of it: a swizzled atom per half
    // full[E], empty[E], q_full, q_empty, per tile: s_full[2], p_full[2], o_done[2], drain, and with
    // two tiles turn[4]
    static constexpr int kControl = kHdr * static_cast<int>(sizeof(BlockHdr)) + 8 * (2 * kMaxEntries + 2 + (TILES == 1 ? 7 : 11) * TILES) + 16;
    // one CTA of two tiles, or two CTAs of one tile, per SM (228 KB, 1 KB of it reserved per CTA)
    static constexpr int kLimit = TILES == 1 ? (228 * 1024) / 2 - 1024 : 227 * 1024;
    static constexpr int kThreads = 32 * (5 * TILES + 1);
    static constexpr uint32_t kCols = 256u * TILES;    // tensor-memory columns
    static constexpr int kQTile = M * D * 2;
    static constexpr int kEntries = (kLimit - TILES * kQTile - kControl) / kEntry < kMaxEntries
                                        ? (kLimit - TILES * kQTile - kControl) / kEntry
                                        : kMaxEntries;
    static constexpr int kRing = TILES * kQTile;
    static constexpr int kBytes = kRing + kEntries * kEntry + kControl;
};

struct TreeArgs {
    const TreeItem *items;
    const int32_t *worker_off;
    int32_t n_items;
    int32_t G, g_shift, Hq, Hkv, max_draft, q_rows, rows_item;
    int64_t n_tokens, num_pages;
    float scale_log2;       // scale * log2 e
    float cap2;             // softcap * log2 e
    float cap_x, cap_x_signed;  // |scale| / softcap, scale / softcap
    float cap_p[4];         // cap2 tanh(cap_x_signed s) = s (p0 + p1 s^2 + ...) for small s
    const __nv_bfloat16 *v_draft;
    int64_t v_stride;
    const unsigned long long *mask;
    const int32_t *draft_off;
    const int32_t *table;
    const int64_t *head_off, *row_lo, *row_hi;
    const int32_t *kv_len;
    __nv_bfloat16 *out;
    float *lse;
    float *part_o, *part_lse;
    uint32_t *err, *ticket;
    uint64_t wait_ns;
};

// The device state of an item's head, as the producer reads it.
struct ItemState {
    TreeItem it;
    int32_t tok0, nb, len;
    int64_t off;
};

__device__ __forceinline__ bool any_nonfinite(uint32_t w) {  // two bf16: an exponent of all ones
    return (((w & 0x7F807F80u) + 0x00800080u) & 0x80008000u) != 0u;
}

// A CTA's way through its items, for the producer warp: its own list, then dynamic items by ticket.
struct ItemWalk {
    const TreeArgs &a;
    int32_t i1, n_static;
    const int lane;
    int32_t cur;   // current item, -1 at the end
    ItemState nx;  // its state

    __device__ __forceinline__ ItemWalk(const TreeArgs &args, int32_t i0, int32_t end, int32_t stat, const TreeItem &first, int l)
        : a(args), i1(end), n_static(stat), lane(l), nx{} {
        cur = i0 < i1 ? i0 : after(i1 - 1);
        if (cur >= 0) nx = state_of(i0 < end ? first : a.items[cur]);
    }
    __device__ __forceinline__ ItemState state_of(const TreeItem &it) const {
        ItemState s;
        s.it = it;
        const int32_t b = it.bh / a.Hkv;
        s.tok0 = a.draft_off[b];
        s.nb = a.draft_off[b + 1] - s.tok0;
        s.len = a.kv_len[it.bh];
        s.off = a.head_off[it.bh];
        return s;
    }
    __device__ __forceinline__ int32_t after(int32_t i) {
        if (i + 1 < i1) return i + 1;
        if (n_static >= a.n_items) return -1;
        int32_t k = 0;
        if (lane == 0) k = static_cast<int32_t>(atomicAdd(a.ticket, 1u));
        k = n_static + __shfl_sync(0xffffffffu, k, 0);
        if (k >= a.n_items) return -1;
        i1 = 0;  // from here on by ticket
        return k;
    }
    __device__ __forceinline__ bool own_next() const { return cur + 1 < i1; }
    __device__ __forceinline__ void advance() {
        cur = after(cur);
        if (cur >= 0) nx = state_of(a.items[cur]);
    }
    // one lane, once: the last CTA to come here readies the tickets for the next call
    __device__ __forceinline__ void finish() const {
        if (n_static < a.n_items && atomicAdd(a.ticket + 1, 1u) == gridDim.x - 1) {
            a.ticket[0] = 0u;
            a.ticket[1] = 0u;
        }
    }
};

// What an item amounts to under the current lengths.
struct ItemShape {
    int32_t h, nrow, np, nc;  // KV head, query rows, pages that hold tokens, blocks of them

    // False: nothing to do. A bad sequence or head is reported and skipped whole: nothing of it is
    // read. A part of a growing head that holds nothing yet is marked empty for the merge.
    __device__ __forceinline__ bool of(const TreeArgs &a, const ItemState &s, int block_pages, int lane) {
        const int32_t b = s.it.bh / a.Hkv;
        h = s.it.bh - b * a.Hkv;
        uint32_t err = 0;
        if (s.nb < 0 || s.nb > a.max_draft || s.tok0 < 0 || static_cast<int64_t>(s.tok0) + s.nb > a.n_tokens) err |= kErrPlan;
        if (s.len < 0 || s.len > s.it.cap) err |= kErrPlan;
        const int32_t pages = (s.len + 15) / 16;
        if (!err && pages > 0 && (s.off < a.row_lo[h] || s.off + pages > a.row_hi[h])) err |= kErrBadRow;
        if (err) {
            if (lane == 0) atomicOr(a.err, err);
            return false;
        }
        nrow = min(s.nb * a.G - s.it.row0, a.rows_item);
        if (nrow <= 0) return false;
        np = max(0, min(s.it.page_end, pages) - s.it.page_begin);
        nc = (np + block_pages - 1) / block_pages;
        if (nc + s.it.draft == 0) {
            for (int32_t r = lane; r < nrow; r += 32) a.part_lse[static_cast<int64_t>(s.it.slot) * a.rows_item + r] = -INFINITY;
            return false;
        }
        return true;
    }
};

// One warp: zeros the V rows between the nv valid tokens and the end of their 16-row box (stale rows
// may hold NaN, which a zero probability does not silence); of drafted V rows, zeros infinities and
// NaN and marks their tokens in *bad (their elements are added back for the rows that see them).
template <int HALVES>
__device__ __forceinline__ void clean_v(uint32_t v, int32_t nv, bool draft, unsigned long long *bad, int lane) {
    constexpr int CH = 8 * HALVES;  // 16-byte chunks of a row
    const int32_t end = (nv + 15) & ~15;
    auto at = [&](int32_t r, int32_t q) { return v + (r >> 3) * (1024 * HALVES) + (q >> 3) * 1024 + (r & 7) * 128 + (((q & 7) ^ (r & 7)) << 4); };
    for (int32_t c = lane; c < (end - nv) * CH; c += 32)
        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(at(nv + c / CH, c % CH)), "r"(0u) : "memory");
    if (draft) {
        for (int32_t r = lane; r < nv; r += 32) {
            uint32_t seen = 0u;
#pragma unroll
            for (int q = 0; q < CH; ++q) {
                uint4 x;
                asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(at(r, q)) : "memory");
                if (any_nonfinite(x.x) | any_nonfinite(x.y) | any_nonfinite(x.z) | any_nonfinite(x.w)) seen |= 1u << q;
            }
            if (seen) {
                atomicOr(bad, 1ull << r);
                __threadfence_block();
                for (int q = 0; q < CH; ++q)
                    if (seen >> q & 1u)
                        for (int w = 0; w < 8; ++w) {
                            uint16_t x;
                            asm volatile("ld.shared.u16 %0, [%1];" : "=h"(x) : "r"(at(r, q) + 2 * w) : "memory");
                            if ((x & 0x7F80u) == 0x7F80u)
                                asm volatile("st.shared.u16 [%0], %1;" ::"r"(at(r, q) + 2 * w), "h"(static_cast<uint16_t>(0)) : "memory");
                        }
            }
        }
    }
    ptx::fence_async_smem();
    __syncwarp();
}

// tanh on |x| <= kTanhNear as x p(x^2), p of degree 3 fitted for the least maximum relative error
// (Lawson's reweighted least squares; 9.8e-08 in exact arithmetic). Scores of a capped head are mostly
// this small, and five multiplications and additions on pairs of scores cost less than the general
// form's two special-function calls each (three with the exponential, on a quarter-rate unit that
// bounds wide drafts). The host folds the scales into the coefficients.
constexpr float kTanhNear = 0.4f;
constexpr double kTanh[4] = {0.999999901901, -0.333313624587, 0.132709767556, -0.0475536034831};

// Capped scores in log2 units, in place: c tanh(s scale / c) log2 e. The two forms differ in their last
// bits, so only what counts may choose: a warp takes the polynomial where every score of its block
// counts (`whole`) and all of them are small; lanes that hold no row of the item (`counts`) have no say.
// Blocks with scores that do not count (stale rows of a page or of the ring, masked drafted tokens)
// take the general form, on the 16-column groups that hold any of the n tokens. Zeroing such scores to
// let the others choose cost every block more registers (16 drafted, capped: 164 us with the choice
// left to all scores, 168 so, 175 to 182 with zeroed ones). Returns the choice.
template <int N>
__device__ __forceinline__ bool cap_scores(uint32_t (&sr)[N], const TreeArgs &a, bool whole, bool counts, int32_t n) {
    using namespace ptx;
    float far = 0.f;
#pragma unroll
    for (int c = 0; c < N; c += 2) far = max3(far, fabsf(__uint_as_float(sr[c])), fabsf(__uint_as_float(sr[c + 1])));
    const bool near = __all_sync(0xffffffffu, whole && (!counts || far * a.cap_x <= kTanhNear));
    if (near) {
        const f2 c0 = pair(a.cap_p[0], a.cap_p[0]), c1 = pair(a.cap_p[1], a.cap_p[1]), c2 = pair(a.cap_p[2], a.cap_p[2]),
                 c3 = pair(a.cap_p[3], a.cap_p[3]);
#pragma unroll
        for (int c = 0; c < N; c += 2) {
            const f2 x = pair(__uint_as_float(sr[c]), __uint_as_float(sr[c + 1]));
            const f2 y = mul2(x, x);
            const f2 p = mul2(x, fma2(fma2(fma2(c3, y, c2), y, c1), y, c0));
            float u, w;
            split(p, u, w);
            sr[c] = __float_as_uint(u);
            sr[c + 1] = __float_as_uint(w);
        }
    } else {
        // tanh(x) = 1 - 2 / (1 + e^2x): absolute error of a few 2^-24 c, limits +-c
        const float k2 = 2.f * kLog2e * a.cap_x_signed;
#pragma unroll
        for (int b = 0; b < N; b += 16)
            if (b < n) {
#pragma unroll
                for (int c = b; c < b + 16 && c < N; ++c) {
                    const float e = ex2(__uint_as_float(sr[c]) * k2);
                    sr[c] = __float_as_uint(a.cap2 * fmaf(-2.f, rcp(1.f + e), 1.f));
                }
            }
    }
    return near;
}

// ------------------------------------------------------------------------------------------
// Tree kernel: a persistent CTA per worker walks the worker's items (equal shares of most of the
// reserved pages, cut ahead of time), then items of the rest by ticket, which evens out what the
// SMs' different memory rates leave. Per CTA and tile of 128 query rows:
//   warps 0-3 (and 4-7):  softmax; thread i owns query row i = tensor-memory lane i, so a row's
//                         max and sum need no shuffles
//   one warp per tile:    MMA issue (lane 0)
//   last warp:            producer: page ids, TMA loads of K and V (64 tokens per block, K and V
//                         separate ring entries) and of the item's Q rows, and the block headers
// Blocks are numbered on through the items, so the producer fills the ring for the next item
// while the softmax warps write the last one out. Per block: S = Q K^T in one of two buffers in
// tensor memory, softmax with the lazily moved running maximum, P as bf16 back over S, O += P V
// with P from tensor memory.
// Query rows are (token, head of the group) pairs, contiguous per token in q, so one 3-D tensor
// map box loads them in order; rows past the draft are loaded or stale and never stored. Drafted
// K and V are a last block of up to 64 tokens with the mask applied to its scores.
// M = 64 (up to 64 rows) halves what the padding rows cost in power and shared memory: a warp then
// has 16 rows, on its first 16 lanes. TILES = 1 (up to 128 rows): two CTAs per SM, so one's softmax and output overlap the other's
// products. TILES = 2 (up to 256 rows): one CTA per SM whose tiles share the K and V ring; wider
// drafts (G = 8) take several row blocks.
// Bound: DRAM, at the clock that the power limit leaves (1.5 to 1.65 GHz of 1.97 with the step repeated).
// 256 sequences of 32/8 heads, 4096 to 32768 tokens at 5 to 50 %, 5 drafted tokens: 5.13 GB in 854 us,
// 6.01 TB/s. 64 sequences, 2048 to 8192 at 10 to 90 %, 16 drafted: 677 MB in 140 us, 4.8 TB/s (127 us at
// the full clock), of which about 16 us are the first loads' latency, the shares' uneven ends and the
// merge. 13 sequences, 8192 to 32768 at 30 to 90 %, 64 drafted, capped: 757 MB in 292 us (381 us where
// scores pass 0.4 of the cap, so that the general form runs), set by the softmax warps' chain of loads,
// polynomials and exponentials, 2800 clocks of a warp per 64 tokens: the tensor pipe is 32 % and issue
// 37 % busy.
// What masked places hold cannot leak: scores are selected, not added to; V rows past the valid
// tokens are zeroed in shared memory before the product (0 * NaN); and an infinity or NaN in a
// drafted V row is taken out of the product and added back only for the rows that attend to it.
// ------------------------------------------------------------------------------------------

template <int D, int TILES, int M, bool CAP>
__global__ void __launch_bounds__(TreeLayout<D, TILES, M>::kThreads, TILES == 1 ? 2 : 1)
    tree_kernel(const __grid_constant__ TreeArgs a, const __grid_constant__ CUtensorMap tm_q,
                const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                const __grid_constant__ CUtensorMap tm_kd, const __grid_constant__ CUtensorMap tm_vd) {
    using TL = TreeLayout<D, TILES, M>;
    using namespace ptx;
    constexpr int RW = M / 4;  // rows of a warp
    constexpr unsigned FULL = 0xffffffffu;
    constexpr int KS = D / 16;
    extern __shared__ __align__(1024) unsigned char smem[];
    const uint32_t sbase = smem_addr(smem);
    constexpr int NE = TL::kEntries;
    const uint32_t ring = sbase + TL::kRing;
    unsigned char *control = smem + TL::kRing + NE * TL::kEntry;
    BlockHdr *hdrs = reinterpret_cast<BlockHdr *>(control);
    const uint32_t full = smem_addr(control) + kHdr * static_cast<uint32_t>(sizeof(BlockHdr));
    const uint32_t empty = full + 8 * kMaxEntries, q_full = empty + 8 * kMaxEntries, q_empty = q_full + 8;
    const uint32_t s_full = q_empty + 8, p_full = s_full + 16 * TILES, o_done = p_full + 16 * TILES,
                   drain = o_done + 16 * TILES, turn = drain + 8 * TILES;
    volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(control + TL::kControl - 16);
    volatile int32_t *abort_flag = reinterpret_cast<volatile int32_t *>(tmem_slot + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr uint32_t q_half = M * 128u;  // bytes of one column half of a Q tile

    // the Q rows that no draft of the plan fills
    for (int c = threadIdx.x; c < (M - a.q_rows) * 8 * TL::kHalves; c += TL::kThreads) {
        const int hf = c / ((M - a.q_rows) * 8), r = c - hf * ((M - a.q_rows) * 8);
        *reinterpret_cast<uint4 *>(smem + hf * q_half + a.q_rows * 128 + r * 16) = make_uint4(0u, 0u, 0u, 0u);
    }
    ptx::fence_async_smem();
    if (threadIdx.x == 0) {
        for (int e = 0; e < NE; ++e) {
            mbar_init(full + 8 * e, 1);
            mbar_init(empty + 8 * e, TILES);
        }
        mbar_init(q_full, 1);
        mbar_init(q_empty, TILES);
        for (int k = 0; k < 2 * TILES; ++k) {
            mbar_init(s_full + 8 * k, 1);
            mbar_init(p_full + 8 * k, 4);
            mbar_init(o_done + 8 * k, 1);
        }
        for (int t = 0; t < TILES; ++t) mbar_init(drain + 8 * t, 1);
        for (int t = 0; TILES > 1 && t < 4 * TILES; ++t) mbar_init(turn + 8 * t, 1);
        *abort_flag = (sbase & 1023u) ? 1 : 0;  // swizzled tiles need 1024-byte alignment
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 4 * TILES) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_addr(const_cast<uint32_t *>(tmem_slot))), "r"(TL::kCols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    // the plan's own lists do not change between calls: read before the preceding kernel is done (and
    // what they point to is brought near; it is read after)
    int32_t i0 = 0, i1 = 0, n_static = 0;
    TreeItem first{};
    if (warp == 5 * TILES) {
        i0 = a.worker_off[blockIdx.x];
        i1 = a.worker_off[blockIdx.x + 1];
        n_static = a.worker_off[gridDim.x];
        if (i0 < i1) {
            first = a.items[i0];
            prefetch_l2(a.kv_len + first.bh);
            prefetch_l2(a.head_off + first.bh);
            prefetch_l2(a.draft_off + first.bh / a.Hkv);
        }
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = *tmem_slot;
    grid_wait();
    grid_launch();
    auto timed_out = [&]() {
        atomicOr(a.err, kErrTimeout);
        *abort_flag = 1;
    };

    if (warp == 5 * TILES) {
        // ================================ producer warp ================================
        ItemWalk walk(a, i0, i1, n_static, first, lane);
        int32_t ent = 0, blk = 0, qn = 0, fills = 0;
        uint32_t eph = 1u;  // parity that says entry `ent` is free
        bool stop = *abort_flag != 0;
        if (stop && lane == 0) atomicOr(a.err, kErrPlan);
        auto wait_entry = [&]() {
            int32_t bad = 0;
            if (lane == 0 && !mbar_wait(empty + 8 * ent, eph, a.wait_ns, abort_flag)) {
                timed_out();
                bad = 1;
            }
            return __shfl_sync(FULL, bad, 0) == 0;
        };
        while (walk.cur >= 0 && !stop) {
            const ItemState s = walk.nx;
            ItemShape sh;
            if (!sh.of(a, s, kCutPages, lane)) {
                walk.advance();
                continue;
            }
            const int32_t h = sh.h, nrow = sh.nrow, np = sh.np, nc = sh.nc, nblk = nc + s.it.draft;
            // the next item is looked up while this one's blocks are in flight; a ticket is drawn late,
            // so that it is not held back from a CTA that is done earlier
            const int32_t look = walk.own_next() ? 0 : max(0, nblk - 2);
            const int32_t *row = a.table + s.off + s.it.page_begin;
            int32_t ids = lane < np ? __ldg(row + lane) : -1;
            int32_t ids_next = 32 + lane < np ? __ldg(row + 32 + lane) : -1;
            // Fills go in the order of use: K(0), then K(j) and V(j - 1), then V of the last block.
            int32_t pid = 0, p_pid = 0, boxes = 0, p_boxes = 0;
            bool is_draft = false, p_draft = false;
            auto fill = [&](bool is_v, bool draft, int32_t page, int32_t n16) {
                const uint32_t fb = full + 8 * ent;
                if (lane == 0) mbar_expect_tx(fb, static_cast<uint32_t>(n16) * 16u * D * 2u);
                __syncwarp();
                if (lane < (draft ? 2 * n16 : n16)) {
                    const uint32_t dst = ring + ent * TL::kEntry;
                    if (draft) tma_4d(dst + lane * TL::kGroup, is_v ? &tm_vd : &tm_kd, 0, s.tok0 + 8 * lane, 0, h, fb);
                    else tma_4d(dst + lane * 2 * TL::kGroup, is_v ? &tm_v : &tm_k, 0, 0, 0, page * 2, fb);
                }
                ++fills;
                if (++ent == NE) {
                    ent = 0;
                    eph ^= 1u;
                }
            };
            for (int32_t j = 0; j < nblk && !stop; ++j, ++blk) {
                p_pid = pid;
                p_boxes = boxes;
                p_draft = is_draft;
                is_draft = j == nc;
                int32_t nv;
                if (is_draft) {
                    nv = s.nb;
                    boxes = (nv + 15) / 16;
                } else {
                    boxes = min(4, np - 4 * j);
                    nv = min(16 * boxes, s.len - 16 * (s.it.page_begin + 4 * j));
                    if (j > 0 && (j & 7) == 0) {
                        ids = ids_next;
                        ids_next = 4 * j + 32 + lane < np ? __ldg(row + 4 * j + 32 + lane) : -1;
                    }
                }
                // lane p loads page p of K, later of V; of the draft, 8 tokens
                pid = is_draft ? 0 : __shfl_sync(FULL, ids, (4 * j + (lane & 3)) & 31);
                if (!is_draft && lane < boxes && (pid < 0 || pid >= a.num_pages)) {
                    atomicOr(a.err, kErrBadPage);
                    pid = 0;  // a page of the pool; the row is flagged as unspecified
                }
                const bool last = j == nblk - 1;
                if (!wait_entry()) {
                    stop = true;
                    break;
                }
                if (lane == 0) {
                    BlockHdr *hd = hdrs + (blk % kHdr);
                    hd->flags = (j == 0 ? kFirst : 0) | (last ? kLast : 0) | (is_draft ? kDraft : 0) | (nv << 8) | (nrow << 16);
                    hd->tok0 = s.tok0;
                    hd->h = h;
                    hd->slot = s.it.slot;
                    hd->row0 = s.it.row0;
                    hd->v_fill = (fills + 1 + (j > 0) + !last) % (2 * NE);
                    hd->bad = 0ull;
                }
                fill(false, is_draft, pid, boxes);
                if (j == 0) {
                    // the item's query rows, once the last item's scores are done
                    int32_t bad = 0;
                    if (lane == 0) {
                        if (!mbar_wait(q_empty, (static_cast<uint32_t>(qn) & 1u) ^ 1u, a.wait_ns, abort_flag)) {
                            timed_out();
                            bad = 1;
                        } else {
                            mbar_expect_tx(q_full, static_cast<uint32_t>(a.q_rows) * D * 2u * TILES);
#pragma unroll
                            for (int t = 0; t < TILES; ++t)
#pragma unroll
                                for (int qh = 0; qh < TL::kHalves; ++qh)
                                    tma_3d(sbase + t * TL::kQTile + qh * q_half, &tm_q, qh * 64, h * a.G,
                                           s.tok0 + ((s.it.row0 + t * M) >> a.g_shift), q_full);
                        }
                    }
                    if (__shfl_sync(FULL, bad, 0)) {
                        stop = true;
                        break;
                    }
                    ++qn;
                } else {
                    if (!wait_entry()) {
                        stop = true;
                        break;
                    }
                    fill(true, p_draft, p_pid, p_boxes);
                }
                if (j == look) walk.advance();
            }
            if (!stop) {
                if (wait_entry()) fill(true, is_draft, pid, boxes);
                else stop = true;
            }
        }
        const bool ended = !stop && wait_entry();
        if (ended && lane == 0) {  // the end marker, in the entry that the oldest copy has left
            hdrs[blk % kHdr].flags = kStop;
            mbar_arrive(full + 8 * ent);
        }
        if (lane == 0) {
            // no copy may be in flight when the CTA exits
            const uint64_t lim = a.wait_ns < kDrainNs ? a.wait_ns : kDrainNs;
            for (int32_t f = max(0, fills - NE + (ended ? 1 : 0)); f < fills; ++f)
                mbar_wait(full + 8 * (f % NE), static_cast<uint32_t>(f / NE) & 1u, lim);
            if (qn > 0) mbar_wait(q_full, static_cast<uint32_t>(qn - 1) & 1u, lim);
            walk.finish();
        }
        __syncwarp();
    } else if (warp >= 4 * TILES) {
        // ================================ MMA warps ================================
        // S(blk) is issued before PV(blk - 1), so the next scores are ready when the softmax has
        // finished a block. P(blk) lies over S(blk) in its buffer; S(blk + 2), which reuses it, is
        // issued by this thread after PV(blk), and the MMAs of one thread run in issue order. One
        // thread's instructions are the longest chain of a block when little else is to do, so
        // addresses are sums and waits that have passed cost one test.
        const int t = warp - 4 * TILES;
        if (lane == 0) {
            constexpr uint32_t hi_q = sdesc_hi(1024), hi_kv = sdesc_hi(TL::kGroup);
            constexpr uint32_t id_s = idesc_bf16(kBlock, M, 0), id_o = idesc_bf16(D, M, 1);
            const uint32_t tm = tmem + 256 * t, t_o = tm + 128;
            const uint32_t k_lo = sdesc_lo(ring, 16), v_lo = sdesc_lo(ring, 1024), q_lo = sdesc_lo(sbase + t * TL::kQTile, 16);
            bool ok = *abort_flag == 0;
            int32_t qn = 0, ent = 0;  // the ring's entries come in the order of use
            uint32_t eph = 0u;
            int32_t p_info = 0;
            bool p_on = false;
            auto next_entry = [&]() {
                if (++ent == NE) {
                    ent = 0;
                    eph ^= 1u;
                }
            };
            auto pv = [&](int32_t blk) {  // O += P V of block blk - 1
                const uint32_t pf = (blk & 1) ^ 1u;
                if (!mbar_wait(full + 8 * ent, eph, a.wait_ns, abort_flag) ||
                    !mbar_wait(p_full + 8 * (2 * t + pf), static_cast<uint32_t>((blk - 1) >> 1) & 1u, a.wait_ns, abort_flag))
                    return false;
                fence_after();
                if (p_on) {
                    const uint32_t v = v_lo + ent * (TL::kEntry >> 4), pa = tm + 64 * pf;
                    const int nk = (((p_info >> 8) & 0xFF) + 15) >> 4;
                    mma_ts(t_o, pa, v, hi_kv, id_o, !(p_info & kFirst));
#pragma unroll
                    for (int k = 1; k < 4; ++k)
                        if (k < nk) mma_ts(t_o, pa + 8 * k, v + k * (2 * TL::kGroup >> 4), hi_kv, id_o, 1);
                    mma_commit(o_done + 8 * (2 * t + pf));
                    mma_commit(empty + 8 * ent);
                } else {
                    mbar_arrive(o_done + 8 * (2 * t + pf));
                    mbar_arrive(empty + 8 * ent);
                }
                next_entry();
                return true;
            };
            for (int32_t blk = 0; ok; ++blk) {
                const uint32_t bf = blk & 1;
                // The header comes with the block's K, which follows the last item's last V: at a change
                // of items that V is the next entry.
                if (p_info & kLast) {
                    if (!(ok = pv(blk))) break;
                }
                ok = mbar_wait(full + 8 * ent, eph, a.wait_ns, abort_flag);
                if (!ok) break;
                const volatile BlockHdr *hd = hdrs + (blk % kHdr);
                const int32_t info = hd->flags;
                const bool on = (info >> 16) > t * M;
                if (!(info & kStop)) {
                    if (info & kFirst) {
                        ok = mbar_wait(q_full, static_cast<uint32_t>(qn) & 1u, a.wait_ns, abort_flag);
                        if (!ok) break;
                        ++qn;
                    }
                    fence_after();
                    if (on) {
                        const uint32_t k = k_lo + ent * (TL::kEntry >> 4);
#pragma unroll
                        for (int ks = 0; ks < KS; ++ks)
                            mma_ss(tm + 64 * bf, q_lo + (ks / 4) * (q_half >> 4) + (ks % 4) * 2, hi_q,
                                   k + (ks / 4) * (1024 >> 4) + (ks % 4) * 2, hi_kv, id_s, ks > 0);
                        mma_commit(s_full + 8 * (2 * t + bf));
                        mma_commit(empty + 8 * ent);
                        if (info & kLast) mma_commit(q_empty);
                    } else {
                        mbar_arrive(s_full + 8 * (2 * t + bf));
                        mbar_arrive(empty + 8 * ent);
                        if (info & kLast) mbar_arrive(q_empty);
                    }
                } else {
                    mbar_arrive(s_full + 8 * (2 * t + bf));
                    break;
                }
                next_entry();
                if (!(info & kFirst) && !(ok = pv(blk))) break;
                p_info = info;
                p_on = on;
            }
            if (!ok) timed_out();
            // every MMA of this thread has finished before tensor memory is released
            mma_commit(drain + 8 * t);
            mbar_wait(drain + 8 * t, 0, a.wait_ns < kDrainNs ? a.wait_ns : kDrainNs);
        }
        __syncwarp();
    } else {
        // ================================ softmax warps ================================
        const int t = warp >> 2, qd = warp & 3;
        const int w0 = M * t + RW * qd;            // the warp's first row of the item
        const int i = w0 + lane;
        const bool live = RW == 32 || lane < RW;   // M = 64: a warp's 16 rows are its first 16 lanes
        const uint32_t lanes = static_cast<uint32_t>(32 * qd) << 16;
        const uint32_t t_s = tmem + lanes + 256 * t, t_o = t_s + 128;
        float m = -INFINITY, le = 0.f;
        unsigned long long mask = 0ull;
        bool ok = *abort_flag == 0;
        // With two tiles and capped scores, the two warps of a scheduler take turns at the exponentials, so
        // that one's share of the special-function unit falls on the other's polynomials (64-token capped
        // trees over 757 MB: 296 us against 315; without a cap there is too little other work: 271 us
        // against 266).
        constexpr bool TURNS = TILES > 1 && CAP;
        auto my_turn = [&](int32_t blk) {
            return !TURNS || mbar_wait(turn + 8 * (4 * t + qd), static_cast<uint32_t>(t == 0 ? blk + 1 : blk) & 1u, a.wait_ns, abort_flag);
        };
        auto pass_turn = [&]() {
            __syncwarp();
            if (TURNS && lane == 0) mbar_arrive(turn + 8 * (4 * (t ^ 1) + qd));
        };
        for (int32_t blk = 0; ok; ++blk) {
            const int bf = blk & 1;
            ok = mbar_wait(s_full + 8 * (2 * t + bf), static_cast<uint32_t>(blk >> 1) & 1u, a.wait_ns, abort_flag);
            if (!__all_sync(FULL, ok)) { ok = false; break; }
            fence_after();
            BlockHdr *hd = hdrs + (blk % kHdr);
            const volatile BlockHdr *vh = hd;
            const int32_t info = vh->flags;
            if (info & kStop) break;
            const int32_t nv = (info >> 8) & 0xFF, nrow = info >> 16;
            const bool valid = live && i < nrow;
            if (w0 >= nrow) {  // no row of this warp
                ok = my_turn(blk);
                pass_turn();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full + 8 * (2 * t + bf));
                continue;
            }
            uint32_t sr[64];
            tmem_ld64(t_s + 64 * bf, sr);
            if (info & kFirst) {
                m = -INFINITY;
                le = 0.f;
                mask = valid ? __ldg(a.mask + vh->tok0 + ((vh->row0 + i) >> a.g_shift)) : 0ull;
            }
            // places of this block that count: the valid tokens; of the draft, those of the mask
            unsigned long long sees = nv >= 64 ? ~0ull : (1ull << nv) - 1ull;
            if (info & kDraft) sees &= mask;
            // V rows between the valid tokens and the end of their 16-row box: zeros (stale rows may
            // hold NaN, which a zero probability does not silence); an infinity or NaN in a drafted
            // V row leaves the product too (added back below for the rows that see it)
            if (qd == 0 && ((nv & 15) || (info & kDraft))) {
                const int32_t v_fill = vh->v_fill, v_ent = v_fill >= NE ? v_fill - NE : v_fill;
                ok = mbar_wait(full + 8 * v_ent, v_fill >= NE, a.wait_ns, abort_flag);
                if (!__all_sync(FULL, ok)) { ok = false; break; }
                clean_v<TL::kHalves>(ring + v_ent * TL::kEntry, nv, info & kDraft, &hd->bad, lane);
            }
            tmem_wait_ld();
            float sl2 = CAP ? 1.f : a.scale_log2;
            if (CAP) {
                cap_scores<64>(sr, a, sees == ~0ull, valid, nv);
            } else if (sl2 < 0.f) {  // the maximum below is of the products: turn them under a negative scale
#pragma unroll
                for (int c = 0; c < 64; ++c) sr[c] ^= 0x80000000u;
                sl2 = -sl2;
            }
            if (!__all_sync(FULL, sees == ~0ull)) {
                // a score that does not count becomes -inf, so that its probability is zero; the
                // scale goes in first (it may be zero)
                const uint32_t lo = static_cast<uint32_t>(sees), hi = static_cast<uint32_t>(sees >> 32);
#pragma unroll
                for (int c = 0; c < 64; ++c) {
                    const bool on = ((c < 32 ? lo : hi) >> (c & 31)) & 1u;
                    sr[c] = __float_as_uint(on ? __uint_as_float(sr[c]) * sl2 : -INFINITY);
                }
                sl2 = 1.f;
            }
            float mr[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) mr[c] = -INFINITY;
#pragma unroll
            for (int c = 0; c < 64; c += 2)
                mr[(c >> 1) & 3] = max3(mr[(c >> 1) & 3], __uint_as_float(sr[c]), __uint_as_float(sr[c + 1]));
            const float mx = max3(fmaxf(mr[0], mr[1]), mr[2], mr[3]) * sl2;
            const bool up = live && mx > m + 8.f;
            if (__any_sync(FULL, up)) {
                const float mn = up ? mx : m;
                const float c0 = !up ? 1.f : (m == -INFINITY ? 0.f : ex2(m - mn));
                if (!(info & kFirst)) {
                    // O holds the products up to PV(blk - 1): wait for it, then scale in place
                    ok = mbar_wait(o_done + 8 * (2 * t + (bf ^ 1)), static_cast<uint32_t>((blk - 1) >> 1) & 1u, a.wait_ns, abort_flag);
                    if (!__all_sync(FULL, ok)) { ok = false; break; }
                    fence_after();
#pragma unroll 1
                    for (int ch = 0; ch < D / 32; ++ch) {
                        uint32_t o[32];
                        tmem_ld32(t_o + 32 * ch, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * c0);
                        tmem_st32(t_o + 32 * ch, o);
                    }
                    tmem_wait_st();
                }
                le *= c0;
                m = mn;
            }
            // p = 2^(s - m), bf16 for the product (its operand type; half a step is 2^-8 of p), fp32
            // for the sum; m stays -inf while nothing counted: p = 0 then
            const float nm = m == -INFINITY ? 0.f : -m;
            const f2 nm2 = pair(nm, nm), sc2 = pair(sl2, sl2);
            if (TURNS) {
                ok = my_turn(blk);
                if (!__all_sync(FULL, ok)) { ok = false; break; }
            }
            f2 ls[4] = {pair(0.f, 0.f), pair(0.f, 0.f), pair(0.f, 0.f), pair(0.f, 0.f)};
            uint32_t pw[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) {
                float p0, p1;
                split(fma2(pair(__uint_as_float(sr[2 * e]), __uint_as_float(sr[2 * e + 1])), sc2, nm2), p0, p1);
                p0 = ex2(p0);
                p1 = ex2(p1);
                ls[e & 3] = add2(ls[e & 3], pair(p0, p1));
                pw[e] = pack_bf16(p0, p1);
            }
            pass_turn();
            tmem_st32(t_s + 64 * bf, pw);
            {
                float u, w;
                split(add2(add2(ls[0], ls[1]), add2(ls[2], ls[3])), u, w);
                le += u + w;
            }
            tmem_wait_st();
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(p_full + 8 * (2 * t + bf));
            if (!(info & kLast)) continue;

            // ---- the item's rows: out = O / le, lse = (m + log2 le) ln 2 ----
            const int32_t tok0 = vh->tok0, h = vh->h, slot = vh->slot, row0 = vh->row0;
            ok = mbar_wait(o_done + 8 * (2 * t + bf), static_cast<uint32_t>(blk >> 1) & 1u, a.wait_ns, abort_flag);
            if (!__all_sync(FULL, ok)) { ok = false; break; }
            fence_after();
            const float inv = le > 0.f ? 1.f / le : (le == 0.f ? 0.f : le);
            const unsigned long long bad = (info & kDraft) ? *const_cast<volatile unsigned long long *>(&hd->bad) & sees : 0ull;
            // The rows leave 16 at a time in the fragment that puts 4 lanes on 32 bytes of a row, so
            // that a store instruction writes whole sectors of 8 rows and not 16 bytes of 32.
            const bool fin = slot < 0;
            auto row_of = [&](int32_t rr) {  // final output row of the item's row rr
                const int32_t r = row0 + rr;
                return static_cast<int64_t>(tok0 + (r >> a.g_shift)) * a.Hq + h * a.G + (r & (a.G - 1));
            };
            const bool any_bad = __any_sync(FULL, bad != 0ull);
#pragma unroll 1
            for (int r16 = 0; r16 < RW && w0 + r16 < nrow; r16 += 16) {
                const int32_t ra = w0 + r16 + (lane >> 2), rb = ra + 8;  // this thread's two rows
                const float ia = __shfl_sync(FULL, inv, r16 + (lane >> 2)), ib = __shfl_sync(FULL, inv, r16 + (lane >> 2) + 8);
                const bool va = ra < nrow, vb = rb < nrow;
                const int c0 = 2 * (lane & 3);
                const int64_t oa = va ? row_of(ra) * D + c0 : 0, ob = vb ? row_of(rb) * D + c0 : 0;
                float *pa = fin ? nullptr : a.part_o + (static_cast<int64_t>(slot) * a.rows_item + ra) * D + c0;
#pragma unroll
                for (int half = 0; half < TL::kHalves; ++half) {
                    uint32_t o[32];
                    tmem_ld_16x64(t_o + (static_cast<uint32_t>(r16) << 16) + 64 * half, o);
                    tmem_wait_ld();
                    float f[32];
#pragma unroll
                    for (int c = 0; c < 32; ++c) f[c] = __uint_as_float(o[c]) * (c & 2 ? ib : ia);
                    if (any_bad) {
#pragma unroll
                        for (int side = 0; side < 2; ++side) {
                            unsigned long long rest = __shfl_sync(FULL, bad, r16 + (lane >> 2) + 8 * side);
                            for (; rest; rest &= rest - 1) {
                                const int j = __ffsll(static_cast<long long>(rest)) - 1;
                                const __nv_bfloat16 *vr = a.v_draft + (static_cast<int64_t>(tok0) + j) * a.v_stride + h * D + 64 * half + c0;
#pragma unroll
                                for (int k = 0; k < 16; ++k) {
                                    const float x = __bfloat162float(vr[8 * (k >> 1) + (k & 1)]);
                                    if (!isfinite(x)) f[4 * (k >> 1) + 2 * side + (k & 1)] += x;
                                }
                            }
                        }
                    }
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const int at = 64 * half + 8 * k;
                        if (fin) {
                            if (va) *reinterpret_cast<uint32_t *>(a.out + oa + at) = pack_bf16(f[4 * k], f[4 * k + 1]);
                            if (vb) *reinterpret_cast<uint32_t *>(a.out + ob + at) = pack_bf16(f[4 * k + 2], f[4 * k + 3]);
                        } else {
                            if (va) *reinterpret_cast<float2 *>(pa + at) = make_float2(f[4 * k], f[4 * k + 1]);
                            if (vb) *reinterpret_cast<float2 *>(pa + 8 * D + at) = make_float2(f[4 * k + 2], f[4 * k + 3]);
                        }
                    }
                }
            }
            if (valid) {
                const float l = le == 0.f ? -INFINITY : (m + lg2(le)) * kLn2;
                if (fin) a.lse[row_of(i)] = l;
                else a.part_lse[static_cast<int64_t>(slot) * a.rows_item + i] = l;
            }
            fence_before();
        }
        if (!ok && lane == 0) timed_out();
    }
    // all warps meet before tensor memory is released
    fence_before();
    __syncthreads();
    fence_after();
    if (warp == 4 * TILES)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TL::kCols) : "memory");
}

// ------------------------------------------------------------------------------------------
// Narrow tree kernel (D = 128, up to 16 query rows: the single-token step and the shortest drafts), one
// persistent CTA per SM. With so few rows one softmax thread per row leaves most lanes idle and the
// wide kernel's tiles are mostly padding. Here the products are turned over, so that tokens and head
// dimensions fill the 128 lanes and the rows are the N side (NR = 16):
//   S^T [128 tokens][NR] = K Q^T           (A = K, B = Q, both K-major in shared memory)
//   O^T [128 dims][NR]  += V^T P^T         (A = V as stored, M-major; B = P^T, written to shared
//                                           memory by the softmax threads, N-major)
// A block is 128 tokens (8 pages). Blocks alternate between two streams with their own softmax
// warpgroup, S and O in tensor memory, P buffer, and running maximum and sum, joined at the item's end.
//   warps 0-3 / 4-7: softmax of the even / odd blocks; thread i owns token i of the block
//   warp 8:          MMA issue (lane 0), tensor memory
//   warp 9:          producer, as in the wide kernel; 32 KB ring entries
// Softmax with a token per thread: the row's base m need not be its maximum, only near enough for
// 2^(s - m) to stay in range, since floating point keeps the relative precision: m starts as the
// score of the stream's first token and moves, with sums and O rescaled, only when a score exceeds
// it by kNarrowSlack in log2 units (a score that stays below it is a true one, so the largest
// probability is never under 1). A row's base moves by that row's scores alone, so neither the next
// sequence's queries in the rows past a short draft nor a drafted key that only other rows attend to
// changes a row's bits. Row sums stay in the threads, one per row, and are added across
// threads once per item in a fixed order.
// Bound: DRAM: one drafted token, 64 sequences of 32/8 heads, 2048 to 8192 tokens at 10 to 90 %: 661 MB
// in 120 us with the merge, 5.55 TB/s; tensor pipe 4 % busy, issue 15 %.
// ------------------------------------------------------------------------------------------
constexpr int kNBlock = 128;           // tokens of a block
constexpr int kNPages = 8;
constexpr float kNarrowSlack = 20.f;   // sums of 2^30 tokens' 2^20 |v| stay in fp32 up to |v| = 2^77
constexpr float kNarrowLook = 19.f;    // excess from which the maxima are looked for
constexpr float kNoScore = -1e30f;     // base of a row that has seen no score

constexpr int kNarrowRows = 16;        // query rows
struct NarrowLayout {
    static constexpr int D = 128, NR = kNarrowRows;
    static constexpr int kEntry = kNBlock * D * 2;
    static constexpr int kGroup = 2048;                   // 8 tokens: an atom per 64-column half
    static constexpr int kQBox = NR * D * 2;
    static constexpr int kQBoxes = 2;
    static constexpr int kPitch = NR * 2;                 // bytes of a P row (a token)
    static constexpr int kP = kNBlock * kPitch;
    static constexpr int kMax = 6;                        // ring entries at most
    // barriers: full[6], empty[6], q_full[2], q_empty[2], s_full[4], p_full[2], o_done[2], drain, join
    static constexpr int kControl = kHdr * static_cast<int>(sizeof(BlockHdr)) + 2 * NR * 4 /* m */ + 2 * NR * 4 /* weights */ +
                                    8 * (2 * kMax + 14) + 32;
    static constexpr int kEntries = (227 * 1024 - kQBoxes * kQBox - 2 * kP - kControl) / kEntry;
    static constexpr int kRing = kQBoxes * kQBox + 2 * kP;
    static constexpr int kCtl = kRing + kEntries * kEntry;
    static constexpr int kBytes = kCtl + kControl;
    static constexpr int kThreads = 10 * 32;
    static_assert(kEntries >= 4 && kEntries <= kMax, "ring entries");
};

// Order-preserving map of floats to unsigned integers (for integer maxima), and back.
__device__ __forceinline__ uint32_t float_key(float x) {
    const uint32_t u = __float_as_uint(x);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float key_float(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k); }

template <bool CAP>
__global__ void __launch_bounds__(NarrowLayout::kThreads, 1)
    tree_narrow_kernel(const __grid_constant__ TreeArgs a, const __grid_constant__ CUtensorMap tm_q,
                       const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                       const __grid_constant__ CUtensorMap tm_kd, const __grid_constant__ CUtensorMap tm_vd) {
    using NL = NarrowLayout;
    using namespace ptx;
    constexpr unsigned FULL = 0xffffffffu;
    constexpr int D = 128, NR = kNarrowRows, NE = NL::kEntries;
    extern __shared__ __align__(1024) unsigned char smem[];
    const uint32_t sbase = smem_addr(smem);
    const uint32_t ring = sbase + NL::kRing, pbuf = sbase + NL::kQBoxes * NL::kQBox;
    BlockHdr *hdrs = reinterpret_cast<BlockHdr *>(smem + NL::kCtl);
    float *base_m = reinterpret_cast<float *>(smem + NL::kCtl + kHdr * sizeof(BlockHdr));  // [2][NR]
    float *weight = base_m + 2 * NR;                                                       // [2][NR]
    const uint32_t full = smem_addr(weight + 2 * NR), empty = full + 8 * NL::kMax, q_full = empty + 8 * NL::kMax,
                   q_empty = q_full + 16, s_full = q_empty + 16, p_full = s_full + 32, o_done = p_full + 16, drain = o_done + 16,
                   join = drain + 8;
    unsigned char *tail = smem + NL::kCtl + NL::kControl - 32;
    volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(tail);
    volatile int32_t *abort_flag = reinterpret_cast<volatile int32_t *>(tail + 4);
    volatile int32_t *used = reinterpret_cast<volatile int32_t *>(tail + 8);                        // [2] stream has tokens
    volatile unsigned long long *item_bad = reinterpret_cast<volatile unsigned long long *>(tail + 16);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    // Q rows that no draft of the plan fills are zeros (see TreeLayout)
    for (int c = threadIdx.x; c < NL::kQBoxes * NL::kQBox / 16; c += NL::kThreads) reinterpret_cast<uint4 *>(smem)[c] = make_uint4(0u, 0u, 0u, 0u);
    fence_async_smem();
    if (threadIdx.x == 0) {
        for (int e = 0; e < NE; ++e) {
            mbar_init(full + 8 * e, 1);
            mbar_init(empty + 8 * e, 1);
        }
        for (int k = 0; k < 2; ++k) {
            mbar_init(q_full + 8 * k, 1);
            mbar_init(q_empty + 8 * k, 1);
            mbar_init(s_full + 8 * k, 1);
            mbar_init(s_full + 16 + 8 * k, 1);
            mbar_init(p_full + 8 * k, 4);
            mbar_init(o_done + 8 * k, 1);
        }
        mbar_init(drain, 1);
        *abort_flag = (sbase & 1023u) ? 1 : 0;  // swizzled tiles need 1024-byte alignment
        mbar_init(join, 8);
        *item_bad = 0ull;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 8) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_addr(const_cast<uint32_t *>(tmem_slot))), "r"(512u) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    // the plan's own lists do not change between calls: read before the preceding kernel is done (and
    // what they point to is brought near; it is read after)
    int32_t i0 = 0, i1 = 0, n_static = 0;
    TreeItem first{};
    if (warp == 9) {
        i0 = a.worker_off[blockIdx.x];
        i1 = a.worker_off[blockIdx.x + 1];
        n_static = a.worker_off[gridDim.x];
        if (i0 < i1) {
            first = a.items[i0];
            prefetch_l2(a.kv_len + first.bh);
            prefetch_l2(a.head_off + first.bh);
            prefetch_l2(a.draft_off + first.bh / a.Hkv);
        }
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = *tmem_slot;
    grid_wait();
    grid_launch();
    auto timed_out = [&]() {
        atomicOr(a.err, kErrTimeout);
        *abort_flag = 1;
    };

    if (warp == 9) {
        // ================================ producer warp ================================
        ItemWalk walk(a, i0, i1, n_static, first, lane);
        int32_t ent = 0, blk = 0, qn = 0, fills = 0;
        uint32_t eph = 1u;
        bool stop = *abort_flag != 0;
        if (stop && lane == 0) atomicOr(a.err, kErrPlan);
        auto wait_entry = [&]() {
            int32_t bad = 0;
            if (lane == 0 && !mbar_wait(empty + 8 * ent, eph, a.wait_ns, abort_flag)) {
                timed_out();
                bad = 1;
            }
            return __shfl_sync(FULL, bad, 0) == 0;
        };
        while (walk.cur >= 0 && !stop) {
            const ItemState s = walk.nx;
            ItemShape sh;
            if (!sh.of(a, s, kNPages, lane)) {
                walk.advance();
                continue;
            }
            // every item has a block for each stream, if need be one without tokens
            const int32_t nblk = max(2, sh.nc + s.it.draft);
            const int32_t look = walk.own_next() ? 0 : max(0, nblk - 2);
            const int32_t *row = a.table + s.off + s.it.page_begin;
            int32_t ids = lane < sh.np ? __ldg(row + lane) : -1;
            int32_t ids_next = 32 + lane < sh.np ? __ldg(row + 32 + lane) : -1;
            const int qb = qn & 1;
            // Fills go in the order of use: K(0), K(1), then K(j) and V(j - 2), then the last two V.
            const int32_t fill0 = fills;
            int32_t pid[3] = {0, 0, 0}, boxes[3] = {0, 0, 0};  // of blocks j, j - 1, j - 2
            auto fill = [&](bool is_v, bool draft, int32_t page, int32_t n16) {
                const uint32_t fb = full + 8 * ent;
                if (lane == 0) {
                    if (n16) mbar_expect_tx(fb, static_cast<uint32_t>(n16) * 16u * D * 2u);
                    else mbar_arrive(fb);
                }
                __syncwarp();
                if (lane < (draft ? 2 * n16 : n16)) {
                    const uint32_t dst = ring + ent * NL::kEntry;
                    if (draft) tma_4d(dst + lane * NL::kGroup, is_v ? &tm_vd : &tm_kd, 0, s.tok0 + 8 * lane, 0, sh.h, fb);
                    else tma_4d(dst + lane * 2 * NL::kGroup, is_v ? &tm_v : &tm_k, 0, 0, 0, page * 2, fb);
                }
                ++fills;
                if (++ent == NE) {
                    ent = 0;
                    eph ^= 1u;
                }
            };
            for (int32_t j = 0; j < nblk && !stop; ++j, ++blk) {
                pid[2] = pid[1];
                pid[1] = pid[0];
                boxes[2] = boxes[1];
                boxes[1] = boxes[0];
                const bool is_draft = s.it.draft && j == sh.nc;
                int32_t nv = 0;
                boxes[0] = 0;
                if (is_draft) {
                    nv = s.nb;
                    boxes[0] = (nv + 15) / 16;
                } else if (j < sh.nc) {
                    boxes[0] = min(kNPages, sh.np - kNPages * j);
                    nv = min(16 * boxes[0], s.len - 16 * (s.it.page_begin + kNPages * j));
                    if (j > 0 && (j & 3) == 0) {
                        ids = ids_next;
                        ids_next = kNPages * j + 32 + lane < sh.np ? __ldg(row + kNPages * j + 32 + lane) : -1;
                    }
                }
                pid[0] = __shfl_sync(FULL, ids, (kNPages * j + (lane & 7)) & 31);
                if (!is_draft && lane < boxes[0] && (pid[0] < 0 || pid[0] >= a.num_pages)) {
                    atomicOr(a.err, kErrBadPage);
                    pid[0] = 0;  // a page of the pool; the row is flagged as unspecified
                }
                const bool last = j == nblk - 1;
                if (!wait_entry()) {
                    stop = true;
                    break;
                }
                if (lane == 0) {
                    BlockHdr *hd = hdrs + (blk % kHdr);
                    // first and last block of each of the two streams
                    hd->flags = (j < 2 ? kFirst : 0) | (j >= nblk - 2 ? kLast : 0) | (is_draft ? kDraft : 0) | (j == 0 ? kOpen : 0) |
                                (last ? kClose : 0) | (s.it.draft ? kTakesDraft : 0) |
                                ((blk - j) & 1 ? kOdd : 0) | (nv << 8) | (sh.nrow << 16);
                    hd->tok0 = s.tok0;
                    hd->h = sh.h;
                    hd->slot = s.it.slot;
                    hd->row0 = s.it.row0;
                    hd->v_fill = (fill0 + (last ? 2 * nblk - 1 : j == nblk - 2 ? 2 * nblk - 2 : 2 * j + 3)) % (2 * NE);
                    hd->bad = 0ull;
                }
                fill(false, is_draft, pid[0], boxes[0]);
                if (j == 0) {
                    // the item's query rows, into a box whose last scores are done
                    int32_t bad = 0;
                    if (lane == 0) {
                        if (!mbar_wait(q_empty + 8 * qb, (static_cast<uint32_t>(qn >> 1) & 1u) ^ 1u, a.wait_ns, abort_flag)) {
                            timed_out();
                            bad = 1;
                        } else {
                            mbar_expect_tx(q_full + 8 * qb, static_cast<uint32_t>(a.q_rows) * D * 2u);
#pragma unroll
                            for (int qh = 0; qh < 2; ++qh)
                                tma_3d(sbase + qb * NL::kQBox + qh * (NL::kQBox / 2), &tm_q, qh * 64, sh.h * a.G,
                                       s.tok0 + (s.it.row0 >> a.g_shift), q_full + 8 * qb);
                        }
                    }
                    if (__shfl_sync(FULL, bad, 0)) {
                        stop = true;
                        break;
                    }
                    ++qn;
                } else if (j > 1) {
                    if (!wait_entry()) {
                        stop = true;
                        break;
                    }
                    fill(true, false, pid[2], boxes[2]);
                }
                if (j == look) walk.advance();
            }
            // the drafted tokens, when the item takes them, are block nc (the last, or the last but one)
            for (int32_t z = 1; z >= 0 && !stop; --z) {
                if (wait_entry()) fill(true, s.it.draft && nblk - 1 - z == sh.nc, pid[z], boxes[z]);
                else stop = true;
            }
        }
        // an end marker for each stream; only the first takes a ring entry's turn
        const bool ended = !stop && wait_entry();
        if (ended && lane == 0) {
            hdrs[blk % kHdr].flags = kStop;
            hdrs[(blk + 1) % kHdr].flags = kStop;
            mbar_arrive(full + 8 * ent);
        }
        if (lane == 0) {
            // no copy may be in flight when the CTA exits
            const uint64_t lim = a.wait_ns < kDrainNs ? a.wait_ns : kDrainNs;
            for (int32_t f = max(0, fills - NE + (ended ? 1 : 0)); f < fills; ++f)
                mbar_wait(full + 8 * (f % NE), static_cast<uint32_t>(f / NE) & 1u, lim);
            for (int32_t k = max(0, qn - 2); k < qn; ++k)
                mbar_wait(q_full + 8 * (k & 1), static_cast<uint32_t>(k >> 1) & 1u, lim);
            walk.finish();
        }
        __syncwarp();
    } else if (warp == 8) {
        // ================================ MMA warp ================================
        // Order: S(blk), then the product of block blk - 2, so that a stream finds its next scores ready
        // when it has finished a block. Each stream has two score buffers: S(blk) overwrites the scores
        // of block blk - 4, which its softmax had read before that block's product was issued.
        if (lane == 0) {
            constexpr uint32_t hi_q = sdesc_hi(1024), hi_kv = sdesc_hi(NL::kGroup);
            // P^T: 8 tokens of 16 rows are an atom of 256 bytes under the 32-byte swizzle (mode 6)
            constexpr uint32_t hi_p = ((8 * NL::kPitch) >> 4) | (1u << 14) | (6u << 29);
            constexpr uint32_t id_s = idesc_bf16(NR, kRows, 0), id_o = idesc_bf16(NR, kRows, 1) | (1u << 15);
            const uint32_t k_lo = sdesc_lo(ring, 16), v_lo = sdesc_lo(ring, 1024), q_lo = sdesc_lo(sbase, 16), p_lo = sdesc_lo(pbuf, 16);
            bool ok = *abort_flag == 0;
            int32_t qn = 0, ent = 0, p_info[2] = {0, 0};  // of blocks blk - 1, blk - 2
            uint32_t eph = 0u;
            auto next_entry = [&]() {
                if (++ent == NE) {
                    ent = 0;
                    eph ^= 1u;
                }
            };
            auto pv = [&](int32_t pb, int32_t info) {  // the product of block pb
                const uint32_t st = pb & 1;
                if (!mbar_wait(full + 8 * ent, eph, a.wait_ns, abort_flag) ||
                    !mbar_wait(p_full + 8 * st, static_cast<uint32_t>(pb >> 1) & 1u, a.wait_ns, abort_flag))
                    return false;
                fence_after();
                const int nk = (((info >> 8) & 0xFF) + 15) >> 4;
                if (nk) {
                    const uint32_t v = v_lo + ent * (NL::kEntry >> 4), p = p_lo + st * (NL::kP >> 4);
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (k < nk)
                            mma_ss(tmem + 256 + 64 * st, v + k * (2 * NL::kGroup >> 4), hi_kv, p + k * (16 * NL::kPitch >> 4), hi_p, id_o,
                                   k > 0 || !(info & kFirst));
                    mma_commit(o_done + 8 * st);
                    mma_commit(empty + 8 * ent);
                } else {
                    mbar_arrive(o_done + 8 * st);
                    mbar_arrive(empty + 8 * ent);
                }
                next_entry();
                return true;
            };
            for (int32_t blk = 0; ok; ++blk) {
                const uint32_t st = blk & 1;
                // the ring brings an item's last two V before the next item's first K
                if (p_info[0] & kClose) {
                    if (!(ok = pv(blk - 2, p_info[1]) && pv(blk - 1, p_info[0]))) break;
                }
                ok = mbar_wait(full + 8 * ent, eph, a.wait_ns, abort_flag);
                if (!ok) break;
                const volatile BlockHdr *hd = hdrs + (blk % kHdr);
                const int32_t info = hd->flags;
                const uint32_t sb = 2 * st + ((blk >> 1) & 1);  // score buffer
                if (info & kStop) {
                    mbar_arrive(s_full + 8 * sb);
                    mbar_arrive(s_full + 8 * (2 * (st ^ 1u) + (((blk + 1) >> 1) & 1)));
                    break;
                }
                if (info & kOpen) {
                    ok = mbar_wait(q_full + 8 * (qn & 1), static_cast<uint32_t>(qn >> 1) & 1u, a.wait_ns, abort_flag);
                    if (!ok) break;
                    ++qn;
                }
                fence_after();
                if ((info >> 8) & 0xFF) {
                    const uint32_t q = q_lo + ((qn - 1) & 1) * (NL::kQBox >> 4), k = k_lo + ent * (NL::kEntry >> 4);
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks)
                        mma_ss(tmem + 64 * sb, k + (ks / 4) * (1024 >> 4) + (ks % 4) * 2, hi_kv,
                               q + (ks / 4) * (NL::kQBox / 2 >> 4) + (ks % 4) * 2, hi_q, id_s, ks > 0);
                    mma_commit(s_full + 8 * sb);
                    mma_commit(empty + 8 * ent);
                } else {
                    mbar_arrive(s_full + 8 * sb);
                    mbar_arrive(empty + 8 * ent);
                }
                if (info & kClose) mma_commit(q_empty + 8 * ((qn - 1) & 1));
                next_entry();
                // an item's third block on: the one before the last
                if (!(info & kOpen) && !(p_info[0] & kOpen) && !(ok = pv(blk - 2, p_info[1]))) break;
                p_info[1] = p_info[0];
                p_info[0] = info;
            }
            if (!ok) timed_out();
            // every MMA of this thread has finished before tensor memory is released
            mma_commit(drain);
            mbar_wait(drain, 0, a.wait_ns < kDrainNs ? a.wait_ns : kDrainNs);
        }
        __syncwarp();
    } else {
        // ================================ softmax warpgroups ================================
        const int st = warp >> 2, qd = warp & 3;
        const int i = 32 * qd + lane;  // token of the block; lane of tensor memory
        const uint32_t lanes = static_cast<uint32_t>(32 * qd) << 16;
        const uint32_t t_o = tmem + lanes + 256;
        const uint32_t p_row = pbuf + st * NL::kP + i * NL::kPitch;
        const uint32_t p_xor = (i >> 2) & 1;  // which 16-byte half of a P row goes first under the 32-byte swizzle
        float *m_row = base_m + st * NR;
        f2 le[NR / 2];
        bool ok = *abort_flag == 0;
        auto wg_sync = [&]() { asm volatile("bar.sync %0, 128;" ::"r"(1 + st) : "memory"); };
        // both warpgroups meet; bounded, since one of them may have given up
        uint32_t jph = 0u;
        auto both_sync = [&]() {
            __syncwarp();
            if (lane == 0) mbar_arrive(join);
            if (!mbar_wait(join, jph, a.wait_ns, abort_flag)) ok = false;
            jph ^= 1u;
            __syncwarp();
        };
        auto wg_any = [&](bool v) {
            uint32_t r;
            asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %2, 0;\n\tbar.red.or.pred q, %1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                         : "=r"(r) : "r"(1 + st), "r"(static_cast<uint32_t>(v)) : "memory");
            return r != 0;
        };
        for (int32_t blk = st;; blk += 2) {
            const uint32_t ph = static_cast<uint32_t>(blk >> 1) & 1u;
            // the warpgroup's barriers count all its threads, so they take every branch around them
            // together, and after a failure leave together here
            const uint32_t sb = 2 * st + ((blk >> 1) & 1);
            const uint32_t t_s = tmem + lanes + 64 * sb;
            ok = !wg_any(!ok || !mbar_wait(s_full + 8 * sb, static_cast<uint32_t>(blk >> 2) & 1u, a.wait_ns, abort_flag));
            if (!ok) break;
            fence_after();
            BlockHdr *hd = hdrs + (blk % kHdr);
            const volatile BlockHdr *vh = hd;
            const int32_t info = vh->flags;
            if (info & kStop) break;
            const int32_t nv = (info >> 8) & 0xFF, nrow = info >> 16;
            if (info & kFirst) {
#pragma unroll
                for (int r = 0; r < NR / 2; ++r) le[r] = pair(0.f, 0.f);
                if (i == 0) used[st] = nv > 0;
                if (nv == 0 && i < NR) m_row[i] = kNoScore;
            }
            if (nv > 0) {
                uint32_t sr[NR];
                tmem_ld<NR>(t_s, sr);
                // V rows between the valid tokens and the end of their 16-row box, and infinities and NaN
                // of drafted V rows, leave the product (see the wide kernel)
                if (qd == 0 && ((nv & 15) || (info & kDraft))) {
                    const int32_t v_fill = vh->v_fill, v_ent = v_fill >= NE ? v_fill - NE : v_fill;
                    ok = mbar_wait(full + 8 * v_ent, v_fill >= NE, a.wait_ns, abort_flag);
                    ok = __all_sync(FULL, ok);
                    if (ok) clean_v<2>(ring + v_ent * NL::kEntry, nv, info & kDraft, &hd->bad, lane);
                }
                // rows that this thread's token counts for
                uint32_t sees = i < nv ? ~0u : 0u;
                if (info & kDraft) {
                    sees = 0u;
                    if (i < nv) {
                        const unsigned long long *mk = a.mask + vh->tok0 + (vh->row0 >> a.g_shift);
                        const uint32_t group = (1u << a.G) - 1u;
#pragma unroll 4
                        for (int32_t r = 0; r < nrow; r += a.G)
                            if (__ldg(mk + (r >> a.g_shift)) >> i & 1ull) sees |= group << r;
                    }
                }
                const bool masked = __any_sync(FULL, (info & kDraft) || i >= nv);
                const bool in_box = i < ((nv + 15) & ~15);
                tmem_wait_ld();
                float *m = m_row;
                float sl2 = a.scale_log2;
                bool near = false;
                if (CAP) {
                    if (nrow < NR) {  // rows that are not the item's
#pragma unroll
                        for (int r = 0; r < NR; ++r) sr[r] = r < nrow ? sr[r] : 0u;
                    }
                    near = cap_scores<NR>(sr, a, !masked, true, NR);
                    sl2 = 1.f;
                }
                if (masked) {  // scores times scale, -inf where they do not count
#pragma unroll
                    for (int r = 0; r < NR; ++r) sr[r] = __float_as_uint((sees >> r & 1u) ? __uint_as_float(sr[r]) * sl2 : -INFINITY);
                    sl2 = 1.f;
                }
                if (info & kFirst) {
                    // a base to start with: the first token's score, which counts for every row; drafted
                    // tokens do not, so there the base is found below
                    if (info & kDraft) {
                        if (i < NR) m[i] = kNoScore;
                    } else if (i == 0) {
#pragma unroll
                        for (int r = 0; r < NR; ++r) {
                            const float x = __uint_as_float(sr[r]) * sl2;
                            m[r] = x == -INFINITY ? kNoScore : x;
                        }
                    }
                    wg_sync();
                }
                const f2 k = pair(sl2, sl2);
                float top = -INFINITY;
#pragma unroll
                for (int r = 0; r < NR; r += 4) {
                    const float4 mm = *reinterpret_cast<const float4 *>(m + r);
                    float t0, t1, t2, t3;
                    split(fma2(pair(__uint_as_float(sr[r]), __uint_as_float(sr[r + 1])), k, pair(-mm.x, -mm.y)), t0, t1);
                    split(fma2(pair(__uint_as_float(sr[r + 2]), __uint_as_float(sr[r + 3])), k, pair(-mm.z, -mm.w)), t2, t3);
                    top = max3(max3(top, t0, t1), t2, t3);
                }
                if (wg_any(top > kNarrowLook)) {
                    // Far above the base: the base of such a row moves to the exact maximum, sums and O with it.
                    // Rows that are not far keep theirs; since a row is looked at well before it is far, no other
                    // row's scores decide about it. Rare, so small code: the scores are read again, 8 rows at a
                    // time.
                    uint32_t *key = reinterpret_cast<uint32_t *>(weight + st * NR);
                    if (i < NR) key[i] = float_key(m[i] == m[i] ? m[i] : kNoScore);
                    wg_sync();
#pragma unroll 1
                    for (int r8 = 0; r8 < NR; r8 += 8) {
                        uint32_t x[8];
                        tmem_ld<8>(t_s + r8, x);
                        tmem_wait_ld();
                        if (CAP) cap_scores<8>(x, a, near, false, 8);
                        const uint32_t on = sees >> r8;
#pragma unroll
                        for (int r = 0; r < 8; ++r) {
                            const float y = __uint_as_float(x[r]) * (CAP ? 1.f : a.scale_log2);
                            const uint32_t u = __reduce_max_sync(FULL, float_key((on >> r & 1u) && y > kNoScore ? y : kNoScore));
                            if (lane == 0) atomicMax(key + r8 + r, u);
                        }
                    }
                    wg_sync();
                    float factor = 1.f, moved = 0.f;
                    if (i < NR) {
                        const float most = key_float(key[i]);
                        const bool far = most - m[i] > kNarrowSlack;  // false for a base of NaN or infinity
                        moved = far ? most : m[i];
                        factor = far ? ex2(m[i] - moved) : 1.f;
                    }
                    wg_sync();
                    if (i < NR) {
                        m[i] = moved;
                        weight[st * NR + i] = factor;
                    }
                    wg_sync();
                    const float *f = weight + st * NR;
                    if (!(info & kFirst)) {
                        // the stream's last product is done before O is scaled
                        if (!mbar_wait(o_done + 8 * st, ph ^ 1u, a.wait_ns, abort_flag)) ok = false;
                        fence_after();
#pragma unroll 1
                        for (int r8 = 0; r8 < NR; r8 += 8) {
                            uint32_t o[8];
                            tmem_ld<8>(t_o + 64 * st + r8, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int r = 0; r < 8; ++r) o[r] = __float_as_uint(__uint_as_float(o[r]) * f[r8 + r]);
                            tmem_st8(t_o + 64 * st + r8, o);
                        }
                        tmem_wait_st();
                    }
#pragma unroll
                    for (int r = 0; r < NR / 2; ++r)
                        le[r] = mul2(le[r], pair(f[2 * r], f[2 * r + 1]));
                    wg_sync();
                }
                // the P buffer's last reader is done
                if (!(info & kFirst) && !mbar_wait(o_done + 8 * st, ph ^ 1u, a.wait_ns, abort_flag)) ok = false;
#pragma unroll
                for (int r = 0; r < NR; r += 8) {
                    uint32_t pw[4];
#pragma unroll
                    for (int c = 0; c < 8; c += 4) {
                        const float4 mm = *reinterpret_cast<const float4 *>(m + r + c);
                        float p0, p1, p2, p3;
                        split(fma2(pair(__uint_as_float(sr[r + c]), __uint_as_float(sr[r + c + 1])), k, pair(-mm.x, -mm.y)), p0, p1);
                        split(fma2(pair(__uint_as_float(sr[r + c + 2]), __uint_as_float(sr[r + c + 3])), k, pair(-mm.z, -mm.w)), p2, p3);
                        p0 = ex2(p0);
                        p1 = ex2(p1);
                        p2 = ex2(p2);
                        p3 = ex2(p3);
                        const int at = (r + c) / 2;
                        le[at] = add2(le[at], pair(p0, p1));
                        le[at + 1] = add2(le[at + 1], pair(p2, p3));
                        pw[c / 2] = pack_bf16(p0, p1);
                        pw[c / 2 + 1] = pack_bf16(p2, p3);
                    }
                    if (in_box)
                        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
                                     ::"r"(p_row + (((r / 8) ^ p_xor) << 4)), "r"(pw[0]), "r"(pw[1]), "r"(pw[2]), "r"(pw[3]) : "memory");
                }
                fence_async_smem();
            }
            fence_before();
            __syncwarp();
            if (info & kDraft) {  // for the rows' corrections below
                wg_sync();
                if (i == 0) *item_bad = *const_cast<volatile unsigned long long *>(&hd->bad);
            }
            if (!__all_sync(FULL, ok)) ok = false;
            if (lane == 0 && ok) mbar_arrive(p_full + 8 * st);
            if (!(info & kLast)) continue;

            // ---- the item's rows ----
            const int32_t tok0 = vh->tok0, h = vh->h, slot = vh->slot, row0 = vh->row0;
            if (wg_any(!ok || !mbar_wait(o_done + 8 * st, ph, a.wait_ns, abort_flag))) ok = false;
            fence_after();
            // row sums over the warp's tokens: halves of the rows change sides with the lanes, so that
            // NR values need NR shuffles, not 5 NR; lane l ends with the row of index bits from l
            float v[NR];
#pragma unroll
            for (int r = 0; r < NR / 2; ++r) split(le[r], v[2 * r], v[2 * r + 1]);
            constexpr int STEPS = 4;  // of the 5 that halve 32 lanes: NR = 2^4
#pragma unroll
            for (int z = 0; z < STEPS; ++z) {
                const int half = NR >> (z + 1);
                const bool up = lane >> z & 1;
#pragma unroll
                for (int r = 0; r < half; ++r) {
                    const float mine = up ? v[r + half] : v[r], other = up ? v[r] : v[r + half];
                    v[r] = mine + __shfl_xor_sync(FULL, other, 1 << z);
                }
            }
            v[0] += __shfl_xor_sync(FULL, v[0], 16);
            // lane l holds row sum_z bit_z(l) NR / 2^(z + 1)
            int32_t r_at = 0;
#pragma unroll
            for (int z = 0; z < STEPS; ++z) r_at += (lane >> z & 1) * (NR >> (z + 1));
            // the stream's P buffer is free: the warps' sums, joined in warp order
            float *sums = reinterpret_cast<float *>(smem + NL::kQBoxes * NL::kQBox + st * NL::kP);  // [4][NR]
            if (lane < NR) sums[qd * NR + r_at] = v[0];
            both_sync();
            // this warpgroup's half of the rows: weights of the two streams, lse
            constexpr int HR = NR / 2;
            const int32_t r_lo = st * HR;
            if (i < HR) {
                const int32_t r = r_lo + i;
                // the stream of the item's first block comes first, whichever it is: an item gives the same bits
                // wherever in a CTA's run it falls
                const int f0 = info & kOdd ? 1 : 0, f1 = f0 ^ 1;
                const float *sums0 = reinterpret_cast<const float *>(smem + NL::kQBoxes * NL::kQBox);
                const float *s0 = sums0 + f0 * (NL::kP / 4), *s1 = sums0 + f1 * (NL::kP / 4);
                const float l0 = (s0[r] + s0[NR + r]) + (s0[2 * NR + r] + s0[3 * NR + r]);
                const float l1 = (s1[r] + s1[NR + r]) + (s1[2 * NR + r] + s1[3 * NR + r]);
                const float m0 = base_m[f0 * NR + r], m1 = base_m[f1 * NR + r];
                const float M = m0 != m0 || m1 != m1 ? NAN : fmaxf(m0, m1);
                const float e0 = ex2(m0 - M), e1 = ex2(m1 - M);
                const float L = l0 * e0 + l1 * e1;
                const float inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);
                weight[r] = used[f0] ? e0 * inv : 0.f;
                weight[NR + r] = used[f1] ? e1 * inv : 0.f;
                if (r < nrow) {
                    const float l = L == 0.f ? -INFINITY : (M + lg2(L)) * kLn2;
                    const int32_t q = row0 + r;
                    if (slot < 0) a.lse[static_cast<int64_t>(tok0 + (q >> a.g_shift)) * a.Hq + h * a.G + (q & (a.G - 1))] = l;
                    else a.part_lse[static_cast<int64_t>(slot) * a.rows_item + r] = l;
                }
            }
            wg_sync();
            const unsigned long long bad = (info & kTakesDraft) ? *item_bad : 0ull;
            const uint32_t f0 = info & kOdd ? 1u : 0u;
            const bool u0 = used[f0], u1 = used[f0 ^ 1u];
            // out^T = w0 O0^T + w1 O1^T; thread i holds dimension i, so a warp writes 32 consecutive elements
            // of a row at a time
            constexpr int C = HR < 16 ? HR : 16;
#pragma unroll 1
            for (int r8 = 0; r8 < HR && r_lo + r8 < nrow; r8 += C) {
                uint32_t oa[C], ob[C];
                tmem_ld<C>(t_o + 64 * f0 + r_lo + r8, oa);
                tmem_ld<C>(t_o + 64 * (f0 ^ 1u) + r_lo + r8, ob);
                tmem_wait_ld();
                float x[C];
#pragma unroll
                for (int r = 0; r < C; ++r) {
                    const int32_t rr = r_lo + r8 + r;
                    x[r] = (u0 ? __uint_as_float(oa[r]) * weight[rr] : 0.f) + (u1 ? __uint_as_float(ob[r]) * weight[NR + rr] : 0.f);
                }
                if (bad) {
#pragma unroll 1
                    for (int r = 0; r < C && r_lo + r8 + r < nrow; ++r) {
                        unsigned long long rest = bad & __ldg(a.mask + tok0 + ((row0 + r_lo + r8 + r) >> a.g_shift));
                        float add = 0.f;
                        for (; rest; rest &= rest - 1) {
                            const int j = __ffsll(static_cast<long long>(rest)) - 1;
                            const float y = __bfloat162float(a.v_draft[(static_cast<int64_t>(tok0) + j) * a.v_stride + h * D + i]);
                            if (!isfinite(y)) add += y;
                        }
#pragma unroll
                        for (int q = 0; q < C; ++q) x[q] = q == r ? x[q] + add : x[q];
                    }
                }
                if (slot < 0) {
#pragma unroll
                    for (int r = 0; r < C; ++r) {
                        const int32_t q = row0 + r_lo + r8 + r;
                        if (r_lo + r8 + r < nrow)
                            a.out[(static_cast<int64_t>(tok0 + (q >> a.g_shift)) * a.Hq + h * a.G + (q & (a.G - 1))) * D + i] = __float2bfloat16_rn(x[r]);
                    }
                } else {
                    float *po = a.part_o + (static_cast<int64_t>(slot) * a.rows_item + r_lo + r8) * D + i;
#pragma unroll
                    for (int r = 0; r < C; ++r)
                        if (r_lo + r8 + r < nrow) po[r * D] = x[r];
                }
            }
            fence_before();
            both_sync();  // O, the sums and the item's mask are free for the next item
            fence_after();
        }
        if (!ok && lane == 0) timed_out();
    }
    // all warps meet before tensor memory is released
    fence_before();
    __syncthreads();
    fence_after();
    if (warp == 8)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
}

// ------------------------------------------------------------------------------------------
// Merge of the split heads: a warp per query row, by log-sum-exp over its parts in order (page
// ranges ascending; a part that holds nothing has lse -inf). Lane j weighs part j; the parts'
// loads do not wait for one another. Bound: one round of loads from L2, where the parts were just
// written (15 500 rows of D = 128 with 16 MB of parts: 12 us alone on a cold cache).
// ------------------------------------------------------------------------------------------
struct TreeMergeArgs {
    const TreeMerge *merge;
    const int32_t *draft_off;
    int32_t G, Hq, Hkv, max_draft, rows_item;
    int64_t n_tokens;
    const float *part_o, *part_lse;
    __nv_bfloat16 *out;
    float *lse;
};
constexpr int kMergeWarps = 8;
constexpr int kMergeParts = 4;  // parts of a row in flight

template <int D>
__global__ void __launch_bounds__(kMergeWarps * 32) tree_merge_kernel(const __grid_constant__ TreeMergeArgs a) {
    constexpr int E = D / 32;  // elements per lane
    constexpr unsigned FULL = 0xffffffffu;
    const TreeMerge mg = a.merge[blockIdx.x];  // the plan's own list
    const int lane = threadIdx.x & 31;
    const int32_t i = blockIdx.y * kMergeWarps + (threadIdx.x >> 5);
    const int32_t b = mg.bh / a.Hkv, h = mg.bh - b * a.Hkv;
    ptx::grid_wait();
    ptx::grid_launch();
    if (i >= a.rows_item) return;
    const int32_t tok0 = a.draft_off[b], nb = a.draft_off[b + 1] - tok0;
    const float *pl = a.part_lse + static_cast<int64_t>(mg.first_slot) * a.rows_item + i;
    const float *po = a.part_o + (static_cast<int64_t>(mg.first_slot) * a.rows_item + i) * D + lane * E;
    const int64_t step = static_cast<int64_t>(a.rows_item) * D;
    float m = -INFINITY, l = 0.f, o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
    for (int32_t j0 = 0; j0 < mg.nsplit; j0 += 32) {
        const int32_t nj = min(32, mg.nsplit - j0);
        float w = lane < nj ? pl[static_cast<int64_t>(j0 + lane) * a.rows_item] * kLog2e : -INFINITY;
        float x[kMergeParts][E];
        auto load = [&](int32_t j) {
#pragma unroll
            for (int k = 0; k < kMergeParts; ++k)
#pragma unroll
                for (int e = 0; e < E; ++e) x[k][e] = j + k < nj ? po[(j0 + j + k) * step + e] : 0.f;
        };
        load(0);
        float mx = w;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, d));
        const float mn = fmaxf(m, mx);
        const float base = mn == -INFINITY ? 0.f : mn;
        const float c0 = exp2f(m - base);  // 0 for m = -inf
        w = exp2f(w - base);
        float sum = w;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(FULL, sum, d);
        l = l * c0 + sum;
        m = mn;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] *= c0;
        for (int32_t j = 0; j < nj; j += kMergeParts) {
            if (j > 0) load(j);
#pragma unroll
            for (int k = 0; k < kMergeParts; ++k) {
                const float wk = __shfl_sync(FULL, w, (j + k) & 31);
                if (j + k < nj && wk != 0.f) {  // a part of weight 0 may never have been written
#pragma unroll
                    for (int e = 0; e < E; ++e) o[e] = fmaf(wk, x[k][e], o[e]);
                }
            }
        }
    }
    const int32_t r = mg.row0 + i;
    if (nb < 0 || nb > a.max_draft || tok0 < 0 || static_cast<int64_t>(tok0) + nb > a.n_tokens || r >= nb * a.G) return;
    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
    const int64_t orow = static_cast<int64_t>(tok0 + r / a.G) * a.Hq + h * a.G + r % a.G;
    uint32_t *dst = reinterpret_cast<uint32_t *>(a.out + orow * D + lane * E);
#pragma unroll
    for (int e = 0; e < E / 2; ++e) dst[e] = ptx::pack_bf16(o[2 * e] * inv, o[2 * e + 1] * inv);
    if (lane == 0) a.lse[orow] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// ------------------------------------------------------------------------------------------
// Host side
// ------------------------------------------------------------------------------------------
#define TG_TRY(expr)                                     \
    do {                                                 \
        cudaError_t e_ = (expr);                         \
        if (e_ != cudaSuccess) {                         \
            set_cuda_error(#expr, static_cast<int>(e_)); \
            return TG_ECUDA;                             \
        }                                                \
    } while (0)

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static const EncodeTiledFn fn = [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return static_cast<EncodeTiledFn>(nullptr);
        return reinterpret_cast<EncodeTiledFn>(ptr);
    }();
    return fn;
}

// bf16 tensor map of `rank` dimensions, boxes of 64 columns, 128-byte swizzle, zeros outside.
int make_map(CUtensorMap *tm, const void *base, int rank, const cuuint64_t *dims, const cuuint64_t *strides,
             const cuuint32_t *box) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) {
        set_cuda_error("cuTensorMapEncodeTiled unavailable", 0);
        return TG_ECUDA;
    }
    const cuuint32_t one[4] = {1, 1, 1, 1};
    const CUresult r = fn(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, static_cast<cuuint32_t>(rank), const_cast<void *>(base),
                          dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) {
        set_cuda_error("cuTensorMapEncodeTiled", static_cast<int>(cudaErrorInvalidValue));
        return TG_ECUDA;
    }
    return TG_OK;
}

// A pool of pages as (column of a 64-column half, row of an 8-row group, half, group): one box is a
// whole page, 4 KB at D = 128, laid out in shared memory group by group, a swizzled atom per half.
int pool_map(CUtensorMap *tm, const void *base, int32_t D, int64_t pages) {
    const cuuint64_t row = static_cast<cuuint64_t>(D) * 2;
    const cuuint64_t dims[4] = {64, 8, static_cast<cuuint64_t>(D / 64), static_cast<cuuint64_t>(pages) * 2};
    const cuuint64_t strides[3] = {row, 128, 8 * row};
    const cuuint32_t box[4] = {64, 8, static_cast<cuuint32_t>(D / 64), 2};
    return make_map(tm, base, 4, dims, strides, box);
}

// Drafted tokens' rows as (column of a half, token, half, head): boxes of 8 tokens of one head, from
// any token on, in the layout of a page's group.
int draft_map(CUtensorMap *tm, const void *base, int32_t D, int32_t heads, int64_t n, int64_t stride) {
    const cuuint64_t row = static_cast<cuuint64_t>(D) * 2;
    const cuuint64_t dims[4] = {64, static_cast<cuuint64_t>(n), static_cast<cuuint64_t>(D / 64), static_cast<cuuint64_t>(heads)};
    const cuuint64_t strides[3] = {static_cast<cuuint64_t>(stride) * 2, 128, row};
    const cuuint32_t box[4] = {64, 8, static_cast<cuuint32_t>(D / 64), 1};
    return make_map(tm, base, 4, dims, strides, box);
}

// Token rows [n][heads][D] with a token stride (elements): boxes of `hb` heads x `tb` tokens.
int token_map(CUtensorMap *tm, const void *base, int32_t D, int32_t heads, int64_t n, int64_t stride, int32_t hb,
              int32_t tb) {
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(n)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(stride) * 2};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(hb), static_cast<cuuint32_t>(tb)};
    return make_map(tm, base, 3, dims, strides, box);
}

bool al16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Pages' worth of an item's fixed work (draft block, Q, joining, output), the wide kernel's and the
// narrow one's; and the shares of the cost laid out ahead of time. Swept in 1 s loops. Wide: 64 sequences
// of 32/8 heads, 2048 to 8192 tokens at 10 to 90 %, 16 drafted | 256 of 300 to 900 tokens, 8 drafted | 128
// of 16/8 heads of D = 64: 18 pages and 98 % take 140.0 | 144.5 | 165.5 us, 10 and 98 % 141.2 | 150.0 |
// 168.5, 14 and 95 % 143.3 | 142.0 | 169.1, 14 and 100 % 141.5 | 149.4 | 166.7. Narrow, the first of them
// with 1 drafted token: 116.3 us at 20 to 30 pages and 90 %, 118 at 95 %, 126 at 30 and 100 %, 161 at 12
// and 100 %.
constexpr int kItemCost = 18, kItemCostNarrow = 24;
constexpr int kMinShare = 4;    // pages of a worker in a step too small to fill the machine
constexpr int kStaticPermille = 980, kStaticPermilleNarrow = 900;

// Work list. A unit is a (head, row block): a run of pages plus a fixed cost. Units are taken longest
// first; the first kStaticPermille of the cost is laid end to end and cut into equal shares, one per
// worker, at whole blocks. The rest (the shortest heads, mostly whole) become dynamic items that
// shrink towards the end, none below the size at which writing a part's rows would cost more than an
// eighth of reading its pages. A small step, which does not fill the machine, is all static.
void build_items(tg_tree_plan *p, const int32_t *cap, int32_t num_workers) {
    const tg_shape &s = p->shape;
    const int64_t BH = static_cast<int64_t>(s.B) * s.Hkv;
    const int32_t rows = p->max_draft * p->G;
    const int32_t rblocks = (rows + p->rows_item - 1) / p->rows_item;
    std::vector<int32_t> order(static_cast<size_t>(BH));
    for (int64_t i = 0; i < BH; ++i) order[static_cast<size_t>(i)] = static_cast<int32_t>(i);
    std::stable_sort(order.begin(), order.end(), [&](int32_t x, int32_t y) { return cap[x] > cap[y]; });
    // A step that leaves workers without kMinShare pages is bound by latency: items cost nothing extra
    // there, every head goes to as many workers as it has shares, and nothing is left for tickets. A head
    // without pages, whose drafted tokens are all its work, counts as a page, so that such heads are
    // dealt out and not left to one worker.
    int64_t total = 0, empty = 0;
    for (int64_t i = 0; i < BH; ++i) {
        total += (cap[i] + 15) / 16;
        empty += cap[i] == 0;
    }
    total *= rblocks;
    const bool small = total < static_cast<int64_t>(num_workers) * kMinShare;
    const int32_t item_cost = small ? 0 : p->narrow ? kItemCostNarrow : kItemCost;
    total += BH * rblocks * item_cost + (small ? empty * rblocks : 0);
    const int64_t nw = std::max<int64_t>(1, small ? std::min<int64_t>(num_workers, std::max<int64_t>(total / kMinShare, BH * rblocks)) : num_workers);
    const int64_t fixed = !small && nw > 1 && p->tiles == 1
                              ? total * (p->narrow ? kStaticPermilleNarrow : kStaticPermille) / 1000
                              : total;
    const int32_t cut = p->narrow ? kNPages : kCutPages;  // heads are cut at whole blocks
    const int64_t min_dyn = p->narrow ? 32 : std::max<int64_t>(24, p->rows_item / 4 / cut * cut);
    p->worker_off.assign(1, 0);
    int64_t done = 0;  // cost laid out so far
    int64_t w = 1;     // the current worker's share ends at fixed * w / nw
    for (int32_t i : order)
        for (int32_t rb = 0; rb < rblocks; ++rb) {
            const int32_t pages = (cap[i] + 15) / 16;
            const int32_t unit_cost = small && pages == 0 ? 1 : item_cost;  // beside its pages
            const int32_t first_slot = p->n_slots;
            const size_t first = p->items.size();
            int32_t at = 0;
            for (;;) {
                int64_t room;  // pages this item may take
                // the share is full when what is left of it would hold less than a block
                while (w <= nw && done + (at == 0 ? unit_cost : 0) + std::min(cut, pages - at) > fixed * w / nw) {
                    if (w == nw && fixed == total) break;  // all static: the last worker takes the rest
                    p->worker_off.push_back(static_cast<int32_t>(p->items.size()));
                    ++w;
                }
                if (w <= nw) {
                    room = w == nw && fixed == total ? INT_MAX : fixed * w / nw - done - (at == 0 ? unit_cost : 0);
                } else {
                    room = std::max<int64_t>(min_dyn, (total - done) / (2 * nw));
                    if (pages - at <= room + room / 2) room = pages - at;
                }
                room = std::max<int64_t>(cut, room / cut * cut);
                int32_t end = static_cast<int32_t>(std::min<int64_t>(pages, at + room));
                if (pages - end < 2 * cut) end = pages;  // no sliver of a head for the next worker
                TreeItem it{};
                it.bh = i;
                it.page_begin = at;
                it.page_end = end;
                it.row0 = rb * p->rows_item;
                it.draft = end == pages;
                it.cap = cap[i];
                it.slot = -1;
                p->items.push_back(it);
                done += (end - at) + (at == 0 ? unit_cost : 0);
                at = end;
                if (at == pages) break;
            }
            const int32_t n = static_cast<int32_t>(p->items.size() - first);
            if (n > 1) {
                for (int32_t j = 0; j < n; ++j) p->items[first + j].slot = first_slot + j;
                p->n_slots += n;
                TreeMerge mg{};
                mg.bh = i;
                mg.first_slot = first_slot;
                mg.nsplit = n;
                mg.row0 = rb * p->rows_item;
                p->merge.push_back(mg);
            }
        }
    while (static_cast<int64_t>(p->worker_off.size()) <= nw) p->worker_off.push_back(static_cast<int32_t>(p->items.size()));
    p->n_workers = static_cast<int32_t>(nw);
}

template <int D, int TILES, int M>
int set_smem() {
    TG_TRY(cudaFuncSetAttribute(tree_kernel<D, TILES, M, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, TreeLayout<D, TILES, M>::kBytes));
    TG_TRY(cudaFuncSetAttribute(tree_kernel<D, TILES, M, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, TreeLayout<D, TILES, M>::kBytes));
    return TG_OK;
}
template <int D>
int set_smem_wide(const tg_tree_plan *p) {
    return p->m == 64 ? set_smem<D, 1, 64>() : p->tiles == 1 ? set_smem<D, 1, 128>() : set_smem<D, 2, 128>();
}
int set_smem_narrow() {
    TG_TRY(cudaFuncSetAttribute(tree_narrow_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, NarrowLayout::kBytes));
    TG_TRY(cudaFuncSetAttribute(tree_narrow_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, NarrowLayout::kBytes));
    return TG_OK;
}

// Selects the plan's device for a scope and puts the caller's back.
struct DeviceScope {
    int before = -1, now = -1;
    cudaError_t enter(int dev) {
        cudaError_t e = cudaGetDevice(&before);
        if (e == cudaSuccess && dev != before) e = cudaSetDevice(dev);
        now = dev;
        return e;
    }
    ~DeviceScope() {
        if (before >= 0 && now != before) cudaSetDevice(before);
    }
};

int tree_device_init(tg_tree_plan *p) {
    DeviceScope scope;
    TG_TRY(scope.enter(p->device));
    const int rc = p->narrow ? set_smem_narrow() : p->shape.D == 128 ? set_smem_wide<128>(p) : set_smem_wide<64>(p);
    if (rc != TG_OK) return rc;
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        const int64_t here = at;
        at += (bytes + 255) / 256 * 256;
        return here;
    };
    const int64_t o_items = take(static_cast<int64_t>(p->items.size()) * sizeof(TreeItem));
    const int64_t o_woff = take(static_cast<int64_t>(p->worker_off.size()) * 4);
    const int64_t o_merge = take(static_cast<int64_t>(p->merge.size()) * sizeof(TreeMerge));
    const int64_t o_lo = take(static_cast<int64_t>(p->row_lo.size()) * 8);
    const int64_t o_hi = take(static_cast<int64_t>(p->row_hi.size()) * 8);
    const int64_t o_err = take(4);
    const int64_t o_ticket = take(8);
    const int64_t head_bytes = at;
    const int64_t o_po = take(static_cast<int64_t>(p->n_slots) * p->rows_item * p->shape.D * 4);
    const int64_t o_pl = take(static_cast<int64_t>(p->n_slots) * p->rows_item * 4);
    std::vector<unsigned char> img(static_cast<size_t>(head_bytes), 0);
    auto put = [&](int64_t off, const void *src, size_t bytes) {
        if (bytes) std::memcpy(img.data() + off, src, bytes);
    };
    put(o_items, p->items.data(), p->items.size() * sizeof(TreeItem));
    put(o_woff, p->worker_off.data(), p->worker_off.size() * 4);
    put(o_merge, p->merge.data(), p->merge.size() * sizeof(TreeMerge));
    put(o_lo, p->row_lo.data(), p->row_lo.size() * 8);
    put(o_hi, p->row_hi.data(), p->row_hi.size() * 8);
    if (cudaMalloc(&p->dev_base, static_cast<size_t>(at)) != cudaSuccess) {
        cudaGetLastError();
        p->dev_base = nullptr;
        return TG_ENOMEM;
    }
    TG_TRY(cudaMemcpy(p->dev_base, img.data(), img.size(), cudaMemcpyHostToDevice));
    // the call returns once pageable memory is staged; a stream that does not wait for the default one
    // must find the plan complete
    TG_TRY(cudaStreamSynchronize(cudaStreamLegacy));
    unsigned char *d = static_cast<unsigned char *>(p->dev_base);
    p->dev_bytes = at;
    p->d_items = reinterpret_cast<TreeItem *>(d + o_items);
    p->d_worker_off = reinterpret_cast<int32_t *>(d + o_woff);
    p->d_merge = reinterpret_cast<TreeMerge *>(d + o_merge);
    p->d_row_lo = reinterpret_cast<int64_t *>(d + o_lo);
    p->d_row_hi = reinterpret_cast<int64_t *>(d + o_hi);
    p->d_err = reinterpret_cast<uint32_t *>(d + o_err);
    p->d_ticket = reinterpret_cast<uint32_t *>(d + o_ticket);
    p->d_part_o = reinterpret_cast<float *>(d + o_po);
    p->d_part_lse = reinterpret_cast<float *>(d + o_pl);
    return TG_OK;
}

void tree_free(tg_tree_plan *p) {
    if (p->dev_base) {
        DeviceScope scope;
        scope.enter(p->device);
        cudaFree(p->dev_base);
    }
    delete p;
}

struct TreeFree {
    void operator()(tg_tree_plan *p) const { tree_free(p); }
};

int tree_plan_create(const tg_shape *s, const int32_t *kv_cap, int32_t max_draft, const int32_t *group_of_head,
                     const int64_t *group_off, int32_t n_groups, int32_t num_workers, int32_t host_only, int32_t device,
                     int32_t wait_limit_us, tg_tree_plan **out) {
    if (!out) return TG_EINVAL;
    *out = nullptr;
    if (!s || s->B < 0 || s->Hkv < 1 || s->Hq < s->Hkv || s->Hq % s->Hkv != 0 || s->num_pages < 0 || max_draft < 1 ||
        !group_of_head || !group_off || n_groups < 1 || num_workers < 0 || wait_limit_us < 0 || device < -1)
        return TG_EINVAL;
    const int32_t G = s->Hq / s->Hkv;
    const int64_t BH = static_cast<int64_t>(s->B) * s->Hkv;
    if (s->page != 16 || (s->D != 64 && s->D != 128) || (G != 1 && G != 2 && G != 4 && G != 8) ||
        max_draft > TG_MAX_DRAFT || BH * 8 > INT32_MAX || s->num_pages > (INT32_MAX / 16))
        return TG_EUNSUPPORTED;
    if (BH > 0 && !kv_cap) return TG_EINVAL;
    int64_t pages = 0;
    for (int64_t i = 0; i < BH; ++i) {
        if (kv_cap[i] < 0) return TG_EINVAL;
        if (kv_cap[i] > TG_MAX_HEAD_TOKENS) return TG_EUNSUPPORTED;
        pages += (kv_cap[i] + 15) / 16;
    }
    if (pages > 0 && s->num_pages < 1) return TG_EINVAL;  // reserved tokens need a pool: a bad page id reads its page 0
    // costs times workers stay in 64 bits
    if (pages > (1ll << 40) || num_workers > 65536) return TG_EUNSUPPORTED;
    for (int32_t g = 0; g < n_groups; ++g)
        if (group_off[g] < 0 || group_off[g + 1] < group_off[g]) return TG_EINVAL;
    for (int32_t h = 0; h < s->Hkv; ++h)
        if (group_of_head[h] < 0 || group_of_head[h] >= n_groups) return TG_EINVAL;

    std::unique_ptr<tg_tree_plan, TreeFree> p(new tg_tree_plan);
    p->shape = *s;
    p->G = G;
    p->max_draft = max_draft;
    p->tiles = max_draft * G > kRows ? 2 : 1;
    p->m = max_draft * G <= kRows / 2 ? kRows / 2 : kRows;
    p->rows_item = p->tiles == 2 ? 2 * kRows : max_draft * G;
    p->q_rows = p->tiles == 2 ? kRows : max_draft * G;
    // The narrow kernel, whose items cost more and whose tokens cost less, from the mean pages of a head
    // on at which it measured faster (128 or 256 sequences of 32/8 heads, 4 and 12 rows, 1 s loops, us
    // narrow : wide by mean pages):  8: 98 : 84 and 99 : 87   23: 121 : 137 and 124 : 135
    // 45: 171 : 183 and 174 : 183   90: 141 : 145 and 142 : 148   180: 261 : 266 and 268 : 270;
    // one sequence, 16 rows, 30000 tokens at 30 to 90 %: 28 : 38. (A variant of 32 rows measured 298 : 281
    // at 180 pages and 166 : 144 at 23, with 32 rows in use, and 889 : 864 on the serving layer with 20.)
    const int32_t rows = max_draft * G;
    if (s->D == 128 && rows <= kNarrowRows && pages >= BH * 16) {
        p->narrow = true;
        p->smem_bytes = NarrowLayout::kBytes;
    } else if (s->D == 128) {
        p->smem_bytes = p->m == 64 ? TreeLayout<128, 1, 64>::kBytes : p->tiles == 1 ? TreeLayout<128, 1, 128>::kBytes : TreeLayout<128, 2, 128>::kBytes;
    } else {
        p->smem_bytes = p->m == 64 ? TreeLayout<64, 1, 64>::kBytes : p->tiles == 1 ? TreeLayout<64, 1, 128>::kBytes : TreeLayout<64, 2, 128>::kBytes;
    }
    p->host_only = host_only != 0;
    p->any_pages = pages > 0;
    if (wait_limit_us > 0) p->wait_ns = static_cast<uint64_t>(wait_limit_us) * 1000ull;
    for (int32_t h = 0; h < s->Hkv; ++h) {
        p->row_lo.push_back(group_off[group_of_head[h]]);
        p->row_hi.push_back(group_off[group_of_head[h] + 1]);
    }
    int sms = 148;
    p->device = device;
    if (!p->host_only) {
        if (device < 0) TG_TRY(cudaGetDevice(&p->device));
        const int rc = device_num_sms(p->device, &sms);
        if (rc != TG_OK) return rc;
    }
    // one resident wave: two CTAs per SM of the wide kernel with one tile, else one
    const int32_t resident = sms * (p->tiles == 1 && !p->narrow ? 2 : 1);
    build_items(p.get(), kv_cap, num_workers > 0 ? num_workers : resident);
    if (!p->host_only) {
        const int rc = tree_device_init(p.get());
        if (rc != TG_OK) return rc;
    }
    *out = p.release();
    return TG_OK;
}

typedef void (*TreeFn)(TreeArgs, CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap);

int launch_tree(const tg_tree_plan *p, TreeFn fn, int threads, const TreeArgs &a, const CUtensorMap *tm, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p->n_workers));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = static_cast<size_t>(p->smem_bytes);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    TG_TRY(cudaLaunchKernelEx(&cfg, fn, a, tm[0], tm[1], tm[2], tm[3], tm[4]));
    return TG_OK;
}

template <int D>
TreeFn wide_fn(const tg_tree_plan *p, bool cap) {
    if (p->m == 64) return cap ? tree_kernel<D, 1, 64, true> : tree_kernel<D, 1, 64, false>;
    if (p->tiles == 1) return cap ? tree_kernel<D, 1, 128, true> : tree_kernel<D, 1, 128, false>;
    return cap ? tree_kernel<D, 2, 128, true> : tree_kernel<D, 2, 128, false>;
}

int launch_tree_kernel(const tg_tree_plan *p, const TreeArgs &a, const CUtensorMap *tm, bool cap, cudaStream_t stream) {
    if (p->narrow)
        return launch_tree(p, cap ? tree_narrow_kernel<true> : tree_narrow_kernel<false>, NarrowLayout::kThreads, a, tm, stream);
    const int threads = p->tiles == 1 ? TreeLayout<128, 1, 128>::kThreads : TreeLayout<128, 2, 128>::kThreads;
    return launch_tree(p, p->shape.D == 128 ? wide_fn<128>(p, cap) : wide_fn<64>(p, cap), threads, a, tm, stream);
}

template <int D>
int launch_tree_merge(const tg_tree_plan *p, const TreeMergeArgs &a, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p->merge.size()), static_cast<unsigned>((p->rows_item + kMergeWarps - 1) / kMergeWarps));
    cfg.blockDim = dim3(kMergeWarps * 32);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    TG_TRY(cudaLaunchKernelEx(&cfg, tree_merge_kernel<D>, a));
    return TG_OK;
}

}  // namespace
}  // namespace tg

using namespace tg;

extern "C" int tg_tree_plan_create(const tg_shape *shape, const int32_t *kv_cap, int32_t max_draft,
                                   const int32_t *group_of_head, const int64_t *group_off, int32_t n_groups,
                                   int32_t num_workers, int32_t host_only, int32_t device, int32_t wait_limit_us,
                                   tg_tree_plan **out) {
    return no_throw([&] {
        return tree_plan_create(shape, kv_cap, max_draft, group_of_head, group_off, n_groups, num_workers, host_only,
                                device, wait_limit_us, out);
    });
}

extern "C" void tg_tree_plan_destroy(tg_tree_plan *p) {
    if (p) tree_free(p);
}

extern "C" int tg_tree_plan_items(const tg_tree_plan *p, int32_t *n_items, int32_t *n_workers, int32_t *n_merge,
                                  int32_t *rows, int64_t *device_bytes, int32_t *items, int32_t *worker_off) {
    if (!p) return TG_EINVAL;
    if (rows) *rows = p->narrow ? kNarrowRows : p->m * p->tiles;
    if (n_items) *n_items = static_cast<int32_t>(p->items.size());
    if (n_workers) *n_workers = p->n_workers;
    if (n_merge) *n_merge = static_cast<int32_t>(p->merge.size());
    if (device_bytes) *device_bytes = p->dev_bytes;
    if (items && !p->items.empty()) std::memcpy(items, p->items.data(), p->items.size() * sizeof(TreeItem));
    if (worker_off) std::memcpy(worker_off, p->worker_off.data(), p->worker_off.size() * 4);
    return TG_OK;
}

extern "C" int tg_tree_plan_status(tg_tree_plan *p, tg_stream stream) {
    if (!p || p->host_only) return TG_EINVAL;
    DeviceScope scope;
    TG_TRY(scope.enter(p->device));
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    uint32_t err = 0;
    TG_TRY(cudaMemcpyAsync(&err, p->d_err, 4, cudaMemcpyDeviceToHost, st));
    TG_TRY(cudaMemsetAsync(p->d_err, 0, 4, st));
    TG_TRY(cudaStreamSynchronize(st));
    if (err & kErrTimeout) {  // a stopped call may have left its tickets part-counted
        TG_TRY(cudaMemsetAsync(p->d_ticket, 0, 8, st));
        TG_TRY(cudaStreamSynchronize(st));
        return TG_ETIMEOUT;
    }
    return err ? TG_EBADPAGE : TG_OK;
}

extern "C" int tg_tree_decode(tg_tree_plan *p, int64_t n_tokens, const int32_t *draft_off, const void *q,
                              int64_t q_stride, const void *k_draft, int64_t k_stride, const void *v_draft,
                              int64_t v_stride, const uint64_t *tree_mask, const void *k_pages, const void *v_pages,
                              const int32_t *page_table, const int64_t *head_page_off, const int32_t *head_kv_len,
                              float scale, float softcap, void *out, float *lse, tg_stream stream) {
    if (!p || p->host_only || n_tokens < 0 || n_tokens > INT32_MAX / 2) return TG_EINVAL;
    const tg_shape &s = p->shape;
    if (s.B == 0 || n_tokens == 0) return TG_OK;
    const int64_t qw = static_cast<int64_t>(s.Hq) * s.D, kw = static_cast<int64_t>(s.Hkv) * s.D;
    if (!draft_off || !q || !k_draft || !v_draft || !tree_mask || (p->any_pages && !page_table) || !head_page_off || !head_kv_len || !out ||
        !lse || !al16(q) || !al16(k_draft) || !al16(v_draft) || !al16(k_pages) || !al16(v_pages) || !al16(out) ||
        q_stride < qw || k_stride < kw || v_stride < kw || q_stride % 8 != 0 || k_stride % 8 != 0 || v_stride % 8 != 0 ||
        !std::isfinite(scale) || !std::isfinite(softcap) || softcap < 0.f || (s.num_pages > 0 && (!k_pages || !v_pages)))
        return TG_EINVAL;
    int cur = 0;
    TG_TRY(cudaGetDevice(&cur));
    if (cur != p->device) return TG_EINVAL;
    // without a pool no head reserves a page, so none is read; the maps still need an address
    const void *kp = s.num_pages > 0 ? k_pages : q, *vp = s.num_pages > 0 ? v_pages : q;
    const int64_t pool = s.num_pages > 0 ? s.num_pages : 1;
    CUtensorMap tm[5];
    int rc = token_map(&tm[0], q, s.D, s.Hq, n_tokens, q_stride, p->G, p->q_rows / p->G);
    if (rc == TG_OK) rc = pool_map(&tm[1], kp, s.D, pool);
    if (rc == TG_OK) rc = pool_map(&tm[2], vp, s.D, pool);
    if (rc == TG_OK) rc = draft_map(&tm[3], k_draft, s.D, s.Hkv, n_tokens, k_stride);
    if (rc == TG_OK) rc = draft_map(&tm[4], v_draft, s.D, s.Hkv, n_tokens, v_stride);
    if (rc != TG_OK) return rc;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    TreeArgs a{};
    a.items = p->d_items;
    a.worker_off = p->d_worker_off;
    a.n_items = static_cast<int32_t>(p->items.size());
    a.ticket = p->d_ticket;
    a.G = p->G;
    a.g_shift = p->G == 1 ? 0 : p->G == 2 ? 1 : p->G == 4 ? 2 : 3;
    a.Hq = s.Hq;
    a.Hkv = s.Hkv;
    a.max_draft = p->max_draft;
    a.q_rows = p->q_rows;
    a.rows_item = p->rows_item;
    a.n_tokens = n_tokens;
    a.num_pages = s.num_pages;
    a.scale_log2 = scale * kLog2e;
    if (softcap > 0.f) {
        a.cap2 = softcap * kLog2e;
        // finite, twice log2 e times it too, so that a score of zero stays one under the tiniest cap
        a.cap_x_signed = std::min(std::max(scale / softcap, -1e38f), 1e38f);
        a.cap_x = std::fabs(a.cap_x_signed);
        double k = static_cast<double>(scale) / softcap;
        for (int i = 0; i < 4; ++i, k *= (static_cast<double>(scale) / softcap) * (static_cast<double>(scale) / softcap))
            a.cap_p[i] = static_cast<float>(static_cast<double>(softcap) * 1.4426950408889634 * kTanh[i] * k);
        for (float c : a.cap_p)
            if (!std::isfinite(c)) a.cap_x = INFINITY;  // a tiny cap: the general form for all scores
    }
    a.v_draft = static_cast<const __nv_bfloat16 *>(v_draft);
    a.v_stride = v_stride;
    a.mask = reinterpret_cast<const unsigned long long *>(tree_mask);
    a.draft_off = draft_off;
    a.table = page_table;
    a.head_off = head_page_off;
    a.row_lo = p->d_row_lo;
    a.row_hi = p->d_row_hi;
    a.kv_len = head_kv_len;
    a.out = static_cast<__nv_bfloat16 *>(out);
    a.lse = lse;
    a.part_o = p->d_part_o;
    a.part_lse = p->d_part_lse;
    a.err = p->d_err;
    a.wait_ns = p->wait_ns;
    rc = launch_tree_kernel(p, a, tm, softcap > 0.f, st);
    if (rc != TG_OK || p->merge.empty()) return rc;
    TreeMergeArgs g{};
    g.merge = p->d_merge;
    g.draft_off = draft_off;
    g.G = p->G;
    g.Hq = s.Hq;
    g.Hkv = s.Hkv;
    g.max_draft = p->max_draft;
    g.rows_item = p->rows_item;
    g.n_tokens = n_tokens;
    g.part_o = p->d_part_o;
    g.part_lse = p->d_part_lse;
    g.out = static_cast<__nv_bfloat16 *>(out);
    g.lse = lse;
    return s.D == 128 ? launch_tree_merge<128>(p, g, st) : launch_tree_merge<64>(p, g, st);
}
