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
    int32_t bh, first_slot, nsplit, row0, cap, pad[3];
};

}  // namespace tg

struct tg_tree_plan {
    tg_shape shape{};
    int32_t G = 0, max_draft = 0, tiles = 1;
    bool host_only = true;
    int device = 0;
    uint64_t wait_ns = 4000000000ull;
    int32_t n_workers = 0;
    int32_t rows_item = 0;   // query rows of an item at most
    int32_t q_rows = 0;      // rows of one Q box (multiple of 8)
    int32_t n_slots = 0;
    std::vector<tg::TreeItem> items;
    std::vector<int32_t> worker_off;
    std::vector<tg::TreeMerge> merge;
    std::vector<int32_t> slot_page;  // first page of each slot's item
    std::vector<int64_t> row_lo, row_hi;  // bounds of each KV head's group table

    void *dev_base = nullptr;
    int64_t dev_bytes = 0;
    tg::TreeItem *d_items = nullptr;
    int32_t *d_worker_off = nullptr;
    tg::TreeMerge *d_merge = nullptr;
    int32_t *d_slot_page = nullptr;
    int64_t *d_row_lo = nullptr, *d_row_hi = nullptr;
    float *d_part_o = nullptr, *d_part_lse = nullptr;
    uint32_t *d_err = nullptr;
};

namespace tg {
namespace {

constexpr int kRows = 128;      // rows of a tile = tensor-memory lanes
constexpr int kBlock = 64;      // tokens of a block (4 pages)
constexpr int kHdr = 16;        // block headers kept
constexpr int kCutPages = 4;    // heads are cut at whole blocks
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

// Block header flags.
constexpr int32_t kFirst = 1, kLast = 2, kDraft = 4, kStop = 8;

struct alignas(16) BlockHdr {
    int32_t flags;
    int32_t nv;     // valid tokens of the block
    int32_t nrow;   // valid query rows of the item
    int32_t bh;
    int32_t tok0;   // the sequence's first drafted token
    int32_t row0;
    int32_t slot;
    int32_t pad;
    unsigned long long bad;  // drafted tokens whose V row holds an infinity or NaN
    unsigned long long pad2;
};
static_assert(sizeof(BlockHdr) == 48, "BlockHdr layout");

template <int D, int TILES>
struct TreeLayout {
    static constexpr int kHalves = D / 64;             // 128-byte column halves
    static constexpr int kEntry = kBlock * D * 2;      // K or V of a block
    static constexpr int kQTile = kRows * D * 2;
    static constexpr int kEntries = TILES == 1 ? (D == 128 ? 5 : 10) : (D == 128 ? 9 : 20);
    static constexpr int kQ = 0;
    static constexpr int kRing = TILES * kQTile;
    static constexpr int kHdrs = kRing + kEntries * kEntry;
    static constexpr int kBars = kHdrs + kHdr * static_cast<int>(sizeof(BlockHdr));
    // full[E], empty[E], q_full[2], q_empty[2], per tile: s_full[2], p_full[2], o_done[2], drain
    static constexpr int kNumBars = 2 * kEntries + 4 + 7 * TILES;
    static constexpr int kBytes = kBars + 8 * kNumBars + 16;
    static constexpr int kThreads = 32 * (5 * TILES + 1);
    static constexpr uint32_t kCols = 256u * TILES;    // tensor-memory columns
};

struct TreeArgs {
    const TreeItem *items;
    const int32_t *worker_off;
    int32_t G, Hq, Hkv, max_draft, q_rows, rows_item;
    int64_t n_tokens, num_pages;
    float scale_log2;       // scale * log2 e
    float cap2, cap_in;     // softcap * log2 e; 2 log2 e * scale / softcap
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
    uint32_t *err;
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

// ------------------------------------------------------------------------------------------
// Tree kernel: a persistent CTA per worker walks the worker's items (equal shares of the reserved
// pages, cut ahead of time). Per CTA and tile of 128 query rows:
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
// TILES = 1 (up to 128 rows): two CTAs per SM, so one's softmax and output overlap the other's
// products. TILES = 2 (up to 256 rows): one CTA per SM whose tiles share the K and V ring; wider
// drafts (G = 8) take several row blocks.
// What masked places hold cannot leak: scores are selected, not added to; V rows past the valid
// tokens are zeroed in shared memory before the product (0 * NaN); and an infinity or NaN in a
// drafted V row is taken out of the product and added back only for the rows that attend to it.
// ------------------------------------------------------------------------------------------
template <int D, int TILES, bool CAP>
__global__ void __launch_bounds__(TreeLayout<D, TILES>::kThreads, TILES == 1 ? 2 : 1)
    tree_kernel(const __grid_constant__ TreeArgs a, const __grid_constant__ CUtensorMap tm_q,
                const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                const __grid_constant__ CUtensorMap tm_kd, const __grid_constant__ CUtensorMap tm_vd) {
    using TL = TreeLayout<D, TILES>;
    using namespace ptx;
    constexpr unsigned FULL = 0xffffffffu;
    constexpr int NE = TL::kEntries;
    constexpr int KS = D / 16;
    extern __shared__ __align__(1024) unsigned char smem[];
    const uint32_t sbase = smem_addr(smem);
    BlockHdr *hdrs = reinterpret_cast<BlockHdr *>(smem + TL::kHdrs);
    const uint32_t bar0 = sbase + TL::kBars;
    const uint32_t full = bar0, empty = bar0 + 8 * NE, q_full = bar0 + 16 * NE, q_empty = q_full + 16;
    const uint32_t s_full = q_empty + 16, p_full = s_full + 16 * TILES, o_done = p_full + 16 * TILES,
                   drain = o_done + 16 * TILES;
    volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(smem + TL::kBars + 8 * TL::kNumBars);
    volatile int32_t *abort_flag = reinterpret_cast<volatile int32_t *>(tmem_slot + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // Q of the next item is loaded beside the current one's when two boxes fit
    const int nq = TILES == 1 && a.q_rows <= kRows / 2 ? 2 : 1;
    const uint32_t q_half = static_cast<uint32_t>(a.q_rows) * 128u;      // bytes of one column half of a box
    const uint32_t q_box = q_half * TL::kHalves;

    if (threadIdx.x == 0) {
        for (int e = 0; e < NE; ++e) {
            mbar_init(full + 8 * e, 1);
            mbar_init(empty + 8 * e, TILES);
        }
        for (int k = 0; k < 2; ++k) {
            mbar_init(q_full + 8 * k, 1);
            mbar_init(q_empty + 8 * k, TILES);
        }
        for (int k = 0; k < 2 * TILES; ++k) {
            mbar_init(s_full + 8 * k, 1);
            mbar_init(p_full + 8 * k, 4);
            mbar_init(o_done + 8 * k, 1);
        }
        for (int t = 0; t < TILES; ++t) mbar_init(drain + 8 * t, 1);
        *abort_flag = (sbase & 1023u) ? 1 : 0;  // swizzled tiles need 1024-byte alignment
        if (sbase & 1023u) atomicOr(a.err, kErrPlan);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 4 * TILES) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_addr(const_cast<uint32_t *>(tmem_slot))), "r"(TL::kCols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
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
        const int32_t i0 = a.worker_off[blockIdx.x], i1 = a.worker_off[blockIdx.x + 1];
        auto fetch = [&](int32_t i) {
            ItemState s;
            s.it = a.items[i];
            const int32_t b = s.it.bh / a.Hkv;
            s.tok0 = a.draft_off[b];
            s.nb = a.draft_off[b + 1] - s.tok0;
            s.len = a.kv_len[s.it.bh];
            s.off = a.head_off[s.it.bh];
            return s;
        };
        ItemState nx{};
        if (i0 < i1) nx = fetch(i0);
        int32_t blk = 0, qn = 0, entries = 0;
        bool stop = *abort_flag != 0;
        auto wait_entry = [&](int32_t e) {
            int32_t bad = 0;
            if (lane == 0 && (!mbar_wait(empty + 8 * (e % NE), (static_cast<uint32_t>(e / NE) & 1u) ^ 1u, a.wait_ns) || *abort_flag)) {
                timed_out();
                bad = 1;
            }
            return __shfl_sync(FULL, bad, 0) == 0;
        };
        for (int32_t i = i0; i < i1 && !stop; ++i) {
            ItemState s = nx;
            if (i + 1 < i1) nx = fetch(i + 1);
            const int32_t b = s.it.bh / a.Hkv, h = s.it.bh - b * a.Hkv;
            // a bad sequence or head is skipped whole: nothing of it is read
            uint32_t err = 0;
            if (s.nb < 0 || s.nb > a.max_draft || s.tok0 < 0 || static_cast<int64_t>(s.tok0) + s.nb > a.n_tokens) err |= kErrPlan;
            if (s.len < 0 || s.len > s.it.cap) err |= kErrPlan;
            const int32_t pages = (s.len + 15) / 16;
            if (!err && pages > 0 && (s.off < a.row_lo[h] || s.off + pages > a.row_hi[h])) err |= kErrBadRow;
            if (err) {
                if (lane == 0) atomicOr(a.err, err);
                continue;
            }
            const int32_t nrow = min(s.nb * a.G - s.it.row0, a.rows_item);
            if (nrow <= 0) continue;
            const int32_t np = max(0, min(s.it.page_end, pages) - s.it.page_begin);
            const int32_t nc = (np + 3) / 4, nblk = nc + s.it.draft;
            if (nblk == 0) continue;
            const int32_t *row = a.table + s.off + s.it.page_begin;
            int32_t ids = lane < np ? __ldg(row + lane) : -1;
            int32_t ids_next = 32 + lane < np ? __ldg(row + 32 + lane) : -1;
            for (int32_t j = 0; j < nblk && !stop; ++j, ++blk) {
                const bool is_draft = j == nc;
                int32_t nv, boxes;
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
                // lane 2 p + half loads half-page p of K, then of V
                const int pg = lane >> 1, hf = lane & 1;
                int64_t pid = is_draft ? 0 : __shfl_sync(FULL, ids, (4 * j + (pg & 3)) & 31);
                const bool mine = pg < boxes && hf < TL::kHalves && lane < 8;
                if (!is_draft && mine && (pid < 0 || pid >= a.num_pages)) {
                    atomicOr(a.err, kErrBadPage);
                    pid = 0;  // a page of the pool; the row is flagged as unspecified
                }
                const uint32_t bytes = static_cast<uint32_t>(boxes) * 16u * D * 2u;
                const int32_t y = is_draft ? s.tok0 + 16 * pg : static_cast<int32_t>(pid * 16);
                for (int kv = 0; kv < 2; ++kv) {
                    const int32_t e = 2 * blk + kv;
                    if (!wait_entry(e)) {
                        stop = true;
                        break;
                    }
                    const uint32_t fb = full + 8 * (e % NE);
                    if (lane == 0) {
                        if (kv == 0) {
                            BlockHdr *hd = hdrs + (blk % kHdr);
                            hd->flags = (j == 0 ? kFirst : 0) | (j == nblk - 1 ? kLast : 0) | (is_draft ? kDraft : 0);
                            hd->nv = nv;
                            hd->nrow = nrow;
                            hd->bh = s.it.bh;
                            hd->tok0 = s.tok0;
                            hd->row0 = s.it.row0;
                            hd->slot = s.it.slot;
                            hd->bad = 0ull;
                        }
                        mbar_expect_tx(fb, bytes);
                    }
                    __syncwarp();
                    if (mine) {
                        const uint32_t dst = sbase + TL::kRing + (e % NE) * TL::kEntry + hf * (kBlock * 128) + pg * 2048;
                        if (is_draft) tma_3d(dst, kv ? &tm_vd : &tm_kd, hf * 64, h, y, fb);
                        else tma_2d(dst, kv ? &tm_v : &tm_k, hf * 64, y, fb);
                    }
                    __syncwarp();
                    entries = e + 1;
                }
                if (j == 0 && !stop) {
                    // the item's query rows, into the box that the item before last has left
                    const int qb = qn % nq;
                    int32_t bad = 0;
                    if (lane == 0) {
                        if (!mbar_wait(q_empty + 8 * qb, (static_cast<uint32_t>(qn / nq) & 1u) ^ 1u, a.wait_ns) || *abort_flag) {
                            timed_out();
                            bad = 1;
                        } else {
                            mbar_expect_tx(q_full + 8 * qb, q_box * TILES);
#pragma unroll
                            for (int t = 0; t < TILES; ++t)
#pragma unroll
                                for (int qh = 0; qh < TL::kHalves; ++qh)
                                    tma_3d(sbase + TL::kQ + t * TL::kQTile + qb * q_box + qh * q_half, &tm_q, qh * 64, h * a.G,
                                           s.tok0 + (s.it.row0 + t * kRows) / a.G, q_full + 8 * qb);
                        }
                    }
                    if (__shfl_sync(FULL, bad, 0)) stop = true;
                    else ++qn;
                }
            }
        }
        const bool ended = !stop && wait_entry(2 * blk);
        if (ended) {  // the end marker, in the entry that the oldest copy has left
            if (lane == 0) {
                hdrs[blk % kHdr].flags = kStop;
                mbar_arrive(full + 8 * ((2 * blk) % NE));
            }
        }
        // no copy may be in flight when the CTA exits
        const uint64_t lim = a.wait_ns < kDrainNs ? a.wait_ns : kDrainNs;
        if (lane == 0) {
            for (int32_t e = max(0, entries - NE + (ended ? 1 : 0)); e < entries; ++e)
                mbar_wait(full + 8 * (e % NE), static_cast<uint32_t>(e / NE) & 1u, lim);
            for (int32_t k = max(0, qn - nq); k < qn; ++k)
                mbar_wait(q_full + 8 * (k % nq), static_cast<uint32_t>(k / nq) & 1u, lim);
        }
        __syncwarp();
    } else if (warp >= 4 * TILES) {
        // ================================ MMA warps ================================
        // S(blk) is issued before PV(blk - 1), so the next scores are ready when the softmax has
        // finished a block. P(blk) lies over S(blk) in its buffer; S(blk + 2), which reuses it, is
        // issued by this thread after PV(blk), and the MMAs of one thread run in issue order.
        const int t = warp - 4 * TILES;
        if (lane == 0) {
            constexpr uint32_t id_s = idesc_bf16(kBlock, kRows, 0), id_o = idesc_bf16(D, kRows, 1);
            const uint32_t tm = tmem + 256 * t, t_o = tm + 128;
            bool ok = *abort_flag == 0;
            int32_t qn = 0;
            int32_t p_flags = 0, p_nv = 0;
            bool p_on = false;
            for (int32_t blk = 0; ok; ++blk) {
                const int32_t e = 2 * blk;
                ok = mbar_wait(full + 8 * (e % NE), static_cast<uint32_t>(e / NE) & 1u, a.wait_ns) && !*abort_flag;
                if (!ok) break;
                fence_after();
                const volatile BlockHdr *hd = hdrs + (blk % kHdr);
                const int32_t flags = hd->flags, nv = hd->nv;
                const bool on = !(flags & kStop) && hd->nrow > t * kRows;
                if (!(flags & kStop)) {
                    const int qb = qn % nq;
                    if (flags & kFirst) {
                        ok = mbar_wait(q_full + 8 * qb, static_cast<uint32_t>(qn / nq) & 1u, a.wait_ns) && !*abort_flag;
                        if (!ok) break;
                        fence_after();
                    }
                    if (on) {
                        const uint32_t q = sbase + TL::kQ + t * TL::kQTile + qb * q_box;
                        const uint32_t k = sbase + TL::kRing + (e % NE) * TL::kEntry;
#pragma unroll
                        for (int ks = 0; ks < KS; ++ks) {
                            const uint32_t hf = ks / 4, o = (ks % 4) * 32;
                            mma_ss(tm + 64 * (blk & 1), sdesc(q + hf * q_half + o, 16, 1024),
                                   sdesc(k + hf * (kBlock * 128) + o, 16, 1024), id_s, ks > 0);
                        }
                        mma_commit(s_full + 8 * (2 * t + (blk & 1)));
                        mma_commit(empty + 8 * (e % NE));
                        if (flags & kLast) mma_commit(q_empty + 8 * qb);
                    } else {
                        mbar_arrive(s_full + 8 * (2 * t + (blk & 1)));
                        mbar_arrive(empty + 8 * (e % NE));
                        if (flags & kLast) mbar_arrive(q_empty + 8 * qb);
                    }
                    if (flags & kLast) ++qn;
                }
                if (blk > 0) {
                    const int32_t pb = blk - 1, pe = 2 * pb + 1;
                    ok = mbar_wait(p_full + 8 * (2 * t + (pb & 1)), static_cast<uint32_t>(pb >> 1) & 1u, a.wait_ns) &&
                         mbar_wait(full + 8 * (pe % NE), static_cast<uint32_t>(pe / NE) & 1u, a.wait_ns) && !*abort_flag;
                    if (!ok) break;
                    fence_after();
                    if (p_on) {
                        const uint32_t v = sbase + TL::kRing + (pe % NE) * TL::kEntry;
                        const int nk = (p_nv + 15) / 16;
                        for (int k = 0; k < nk; ++k)
                            mma_ts(t_o, tm + 64 * (pb & 1) + 8 * k, sdesc(v + k * 2048, kBlock * 128, 1024), id_o,
                                   k > 0 || !(p_flags & kFirst));
                        mma_commit(o_done + 8 * (2 * t + (pb & 1)));
                        mma_commit(empty + 8 * (pe % NE));
                    } else {
                        mbar_arrive(o_done + 8 * (2 * t + (pb & 1)));
                        mbar_arrive(empty + 8 * (pe % NE));
                    }
                }
                if (flags & kStop) {
                    mbar_arrive(s_full + 8 * (2 * t + (blk & 1)));
                    break;
                }
                p_flags = flags;
                p_nv = nv;
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
        const int i = kRows * t + 32 * qd + lane;  // row of the item
        const uint32_t lanes = static_cast<uint32_t>(32 * qd) << 16;
        const uint32_t t_s = tmem + lanes + 256 * t, t_o = t_s + 128;
        float m = -INFINITY, le = 0.f;
        unsigned long long mask = 0ull;
        bool ok = *abort_flag == 0;
        for (int32_t blk = 0; ok; ++blk) {
            const int bf = blk & 1;
            ok = mbar_wait(s_full + 8 * (2 * t + bf), static_cast<uint32_t>(blk >> 1) & 1u, a.wait_ns) && !*abort_flag;
            if (!__all_sync(FULL, ok)) { ok = false; break; }
            fence_after();
            BlockHdr *hd = hdrs + (blk % kHdr);
            const volatile BlockHdr *vh = hd;
            const int32_t flags = vh->flags;
            if (flags & kStop) break;
            const int32_t nv = vh->nv, nrow = vh->nrow;
            const bool valid = i < nrow;
            if (kRows * t + 32 * qd >= nrow) {  // no row of this warp
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full + 8 * (2 * t + bf));
                continue;
            }
            if (flags & kFirst) {
                m = -INFINITY;
                le = 0.f;
                mask = valid ? __ldg(a.mask + vh->tok0 + (vh->row0 + i) / a.G) : 0ull;
            }
            // places of this block that count: the valid tokens; of the draft, those of the mask
            unsigned long long sees = nv >= 64 ? ~0ull : (1ull << nv) - 1ull;
            if (flags & kDraft) sees &= mask;
            // V rows between the valid tokens and the end of their 16-row box: zeros (stale rows may
            // hold NaN, which a zero probability does not silence); an infinity or NaN in a drafted
            // V row leaves the product too (added back below for the rows that see it)
            if (qd == 0 && ((nv & 15) || (flags & kDraft))) {
                const int32_t ve = 2 * blk + 1;
                ok = mbar_wait(full + 8 * (ve % NE), static_cast<uint32_t>(ve / NE) & 1u, a.wait_ns) && !*abort_flag;
                if (!__all_sync(FULL, ok)) { ok = false; break; }
                const uint32_t v = sbase + TL::kRing + (ve % NE) * TL::kEntry;
                const int32_t end = (nv + 15) & ~15;
                for (int32_t c = lane; c < (end - nv) * 8 * TL::kHalves; c += 32) {
                    const int32_t r = nv + c / (8 * TL::kHalves), q = c % (8 * TL::kHalves);
                    asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};"
                                 ::"r"(v + (q >> 3) * (kBlock * 128) + r * 128 + (q & 7) * 16), "r"(0u) : "memory");
                }
                if (flags & kDraft) {
                    for (int32_t r = lane; r < nv; r += 32) {
                        uint32_t seen = 0u;
#pragma unroll
                        for (int q = 0; q < 8 * TL::kHalves; ++q) {
                            const uint32_t addr = v + (q >> 3) * (kBlock * 128) + r * 128 + (((q & 7) ^ (r & 7)) << 4);
                            uint4 x;
                            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                         : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(addr) : "memory");
                            if (any_nonfinite(x.x) | any_nonfinite(x.y) | any_nonfinite(x.z) | any_nonfinite(x.w)) seen |= 1u << q;
                        }
                        if (seen) {
                            atomicOr(&hd->bad, 1ull << r);
                            __threadfence_block();
                            for (int q = 0; q < 8 * TL::kHalves; ++q)
                                if (seen >> q & 1u) {
                                    const uint32_t addr = v + (q >> 3) * (kBlock * 128) + r * 128 + (((q & 7) ^ (r & 7)) << 4);
                                    for (int w = 0; w < 8; ++w) {
                                        uint16_t x;
                                        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(x) : "r"(addr + 2 * w) : "memory");
                                        if ((x & 0x7F80u) == 0x7F80u)
                                            asm volatile("st.shared.u16 [%0], %1;" ::"r"(addr + 2 * w), "h"(static_cast<uint16_t>(0)) : "memory");
                                    }
                                }
                        }
                    }
                }
                fence_async_smem();
                __syncwarp();
            }
            uint32_t sr[64];
            tmem_ld64(t_s + 64 * bf, sr);
            tmem_wait_ld();
            if (CAP) {
                // c tanh(x) in log2 units, tanh(x) = 1 - 2 / (1 + 2^(2 x log2 e)): absolute error of
                // a few 2^-24 c, and the limits +-c at the ends
#pragma unroll
                for (int c = 0; c < 64; ++c) {
                    const float e = ex2(__uint_as_float(sr[c]) * a.cap_in);
                    sr[c] = __float_as_uint(a.cap2 * fmaf(-2.f, rcp(1.f + e), 1.f));
                }
            }
            float sl2 = CAP ? 1.f : a.scale_log2;
            const bool whole = sees == ~0ull;
            const bool all_whole = __all_sync(FULL, whole);
            float mr[8];
#pragma unroll
            for (int c = 0; c < 8; ++c) mr[c] = -INFINITY;
            if (!all_whole) {
                // a score that does not count becomes -inf, so that its probability is zero; the
                // scale goes in first (it may be zero or negative)
                const uint32_t lo = static_cast<uint32_t>(sees), hi = static_cast<uint32_t>(sees >> 32);
#pragma unroll
                for (int c = 0; c < 64; ++c) {
                    const bool on = ((c < 32 ? lo : hi) >> (c & 31)) & 1u;
                    sr[c] = __float_as_uint(on ? __uint_as_float(sr[c]) * sl2 : -INFINITY);
                }
                sl2 = 1.f;
            }
#pragma unroll
            for (int c = 0; c < 64; ++c) mr[c & 7] = fmaxf(mr[c & 7], __uint_as_float(sr[c]) * sl2);
            const float mx = fmaxf(fmaxf(fmaxf(mr[0], mr[1]), fmaxf(mr[2], mr[3])),
                                   fmaxf(fmaxf(mr[4], mr[5]), fmaxf(mr[6], mr[7])));
            const bool up = mx > m + 8.f;
            if (__any_sync(FULL, up)) {
                const float mn = up ? mx : m;
                const float c0 = !up ? 1.f : (m == -INFINITY ? 0.f : ex2(m - mn));
                if (!(flags & kFirst)) {
                    // O holds the products up to PV(blk - 1): wait for it, then scale in place
                    ok = mbar_wait(o_done + 8 * (2 * t + (bf ^ 1)), static_cast<uint32_t>((blk - 1) >> 1) & 1u, a.wait_ns) && !*abort_flag;
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
            // p = 2^(s - m), bf16 for the product (its operand type; half a step is 2^-9 of p), fp32
            // for the sum; m stays -inf while nothing counted: p = 0 then
            const float nm = m == -INFINITY ? 0.f : -m;
            float ls[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            uint32_t pw[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) {
                const float p0 = ex2(fmaf(__uint_as_float(sr[2 * e]), sl2, nm));
                const float p1 = ex2(fmaf(__uint_as_float(sr[2 * e + 1]), sl2, nm));
                ls[e & 3] += p0;
                ls[4 + (e & 3)] += p1;
                pw[e] = pack_bf16(p0, p1);
            }
            le += ((ls[0] + ls[1]) + (ls[2] + ls[3])) + ((ls[4] + ls[5]) + (ls[6] + ls[7]));
            tmem_st32(t_s + 64 * bf, pw);
            tmem_wait_st();
            fence_before();
            __syncwarp();
            const int32_t tok0 = vh->tok0, bh = vh->bh, slot = vh->slot, row0 = vh->row0;
            if (lane == 0) mbar_arrive(p_full + 8 * (2 * t + bf));
            if (!(flags & kLast)) continue;

            // ---- the item's rows: out = O / le, lse = (m + log2 le) ln 2 ----
            ok = mbar_wait(o_done + 8 * (2 * t + bf), static_cast<uint32_t>(blk >> 1) & 1u, a.wait_ns) && !*abort_flag;
            if (!__all_sync(FULL, ok)) { ok = false; break; }
            fence_after();
            const float inv = le > 0.f ? 1.f / le : (le == 0.f ? 0.f : le);
            const unsigned long long bad = (flags & kDraft) ? *const_cast<volatile unsigned long long *>(&hd->bad) & sees : 0ull;
            const int32_t b = bh / a.Hkv, h = bh - b * a.Hkv, r = row0 + i;
            const int64_t orow = valid ? (static_cast<int64_t>(tok0 + r / a.G) * a.Hq + h * a.G + r % a.G) : 0;
#pragma unroll 1
            for (int ch = 0; ch < D / 32; ++ch) {
                uint32_t o[32];
                tmem_ld32(t_o + 32 * ch, o);
                tmem_wait_ld();
                float f[32];
#pragma unroll
                for (int c = 0; c < 32; ++c) f[c] = __uint_as_float(o[c]) * inv;
                if (bad) {
                    for (unsigned long long left = bad; left; left &= left - 1) {
                        const int j = __ffsll(static_cast<long long>(left)) - 1;
                        const __nv_bfloat16 *vr = a.v_draft + (static_cast<int64_t>(tok0) + j) * a.v_stride + h * D + 32 * ch;
#pragma unroll
                        for (int c = 0; c < 32; ++c) {
                            const float x = __bfloat162float(vr[c]);
                            if (!isfinite(x)) f[c] += x;
                        }
                    }
                }
                if (!valid) continue;
                if (slot < 0) {
                    uint4 *dst = reinterpret_cast<uint4 *>(a.out + orow * D + 32 * ch);
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        dst[c] = make_uint4(pack_bf16(f[8 * c], f[8 * c + 1]), pack_bf16(f[8 * c + 2], f[8 * c + 3]),
                                            pack_bf16(f[8 * c + 4], f[8 * c + 5]), pack_bf16(f[8 * c + 6], f[8 * c + 7]));
                } else {
                    float4 *dst = reinterpret_cast<float4 *>(a.part_o + (static_cast<int64_t>(slot) * a.rows_item + i) * D + 32 * ch);
#pragma unroll
                    for (int c = 0; c < 8; ++c) dst[c] = make_float4(f[4 * c], f[4 * c + 1], f[4 * c + 2], f[4 * c + 3]);
                }
            }
            if (valid) {
                const float l = le == 0.f ? -INFINITY : (m + lg2(le)) * kLn2;
                if (slot < 0) a.lse[orow] = l;
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
// Merge of the split heads: a warp per query row, its parts in order (page ranges ascending), by
// log-sum-exp. A part whose pages hold no token yet was not written and is left out; the last part
// holds the drafted tokens and always counts.
// ------------------------------------------------------------------------------------------
struct TreeMergeArgs {
    const TreeMerge *merge;
    const int32_t *slot_page, *draft_off, *kv_len;
    int32_t G, Hq, Hkv, max_draft, rows_item;
    int64_t n_tokens;
    const float *part_o, *part_lse;
    __nv_bfloat16 *out;
    float *lse;
};
constexpr int kMergeWarps = 8;

template <int D>
__global__ void __launch_bounds__(kMergeWarps * 32) tree_merge_kernel(const __grid_constant__ TreeMergeArgs a) {
    constexpr int E = D / 32;  // elements per lane
    ptx::grid_wait();
    ptx::grid_launch();
    const TreeMerge mg = a.merge[blockIdx.x];
    const int lane = threadIdx.x & 31;
    const int32_t i = blockIdx.y * kMergeWarps + (threadIdx.x >> 5);
    const int32_t b = mg.bh / a.Hkv, h = mg.bh - b * a.Hkv;
    const int32_t tok0 = a.draft_off[b], nb = a.draft_off[b + 1] - tok0, len = a.kv_len[mg.bh];
    if (nb < 0 || nb > a.max_draft || tok0 < 0 || static_cast<int64_t>(tok0) + nb > a.n_tokens || len < 0 || len > mg.cap) return;
    const int32_t r = mg.row0 + i;
    if (i >= a.rows_item || r >= nb * a.G) return;
    const int32_t pages = (len + 15) / 16;
    float m = -INFINITY, l = 0.f, o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
    for (int32_t j = 0; j < mg.nsplit; ++j) {
        const int32_t slot = mg.first_slot + j;
        if (j + 1 < mg.nsplit && a.slot_page[slot] >= pages) continue;
        const float pl = a.part_lse[static_cast<int64_t>(slot) * a.rows_item + i] * kLog2e;
        if (pl == -INFINITY) continue;
        const float *po = a.part_o + (static_cast<int64_t>(slot) * a.rows_item + i) * D + lane * E;
        const float mn = fmaxf(m, pl);
        const float c0 = m == -INFINITY ? 0.f : exp2f(m - mn), c1 = exp2f(pl - mn);
        l = l * c0 + c1;
        m = mn;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = o[e] * c0 + c1 * po[e];
    }
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

// bf16 tensor map of 1 + `rank` dimensions, boxes of 64 columns, 128-byte swizzle, zeros outside.
int make_map(CUtensorMap *tm, const void *base, int rank, const cuuint64_t *dims, const cuuint64_t *strides,
             const cuuint32_t *box) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) {
        set_cuda_error("cuTensorMapEncodeTiled unavailable", 0);
        return TG_ECUDA;
    }
    const cuuint32_t one[3] = {1, 1, 1};
    const CUresult r = fn(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, static_cast<cuuint32_t>(rank), const_cast<void *>(base),
                          dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) {
        set_cuda_error("cuTensorMapEncodeTiled", static_cast<int>(cudaErrorInvalidValue));
        return TG_ECUDA;
    }
    return TG_OK;
}

int pool_map(CUtensorMap *tm, const void *base, int32_t D, int64_t pages) {
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(pages) * 16};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(D) * 2};
    const cuuint32_t box[2] = {64, 16};
    return make_map(tm, base, 2, dims, strides, box);
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

constexpr int kItemCost = 8;  // pages' worth of an item's fixed work (draft block, Q, output)

// Work list: every (head, row block) is a run of pages plus a fixed cost; the runs are laid end to
// end and cut into n_workers equal shares at whole blocks (no share below kMinShare pages).
constexpr int kMinShare = 16;

void build_items(tg_tree_plan *p, const int32_t *cap, int32_t num_workers) {
    const tg_shape &s = p->shape;
    const int64_t BH = static_cast<int64_t>(s.B) * s.Hkv;
    const int32_t rows = p->max_draft * p->G;
    const int32_t rblocks = (rows + p->rows_item - 1) / p->rows_item;
    int64_t total = 0;
    for (int64_t i = 0; i < BH; ++i) total += (cap[i] + 15) / 16 + kItemCost;
    total *= rblocks;
    const int64_t nw = std::max<int64_t>(1, std::min<int64_t>(num_workers, total / kMinShare));
    p->worker_off.assign(1, 0);
    int64_t done = 0;  // cost laid out so far
    int64_t w = 1;     // the current worker's share ends at total * w / nw
    for (int64_t i = 0; i < BH; ++i)
        for (int32_t rb = 0; rb < rblocks; ++rb) {
            const int32_t pages = (cap[i] + 15) / 16;
            const int32_t first_slot = p->n_slots;
            const size_t first = p->items.size();
            int32_t at = 0;
            for (;;) {
                while (w < nw && done + kItemCost >= total * w / nw) {  // the share is full
                    p->worker_off.push_back(static_cast<int32_t>(p->items.size()));
                    ++w;
                }
                int64_t room = w < nw ? total * w / nw - done - kItemCost : INT_MAX;
                room = std::max<int64_t>(kCutPages, room / kCutPages * kCutPages);
                int32_t end = static_cast<int32_t>(std::min<int64_t>(pages, at + room));
                if (pages - end < 2 * kCutPages) end = pages;  // no sliver of a head for the next worker
                TreeItem it{};
                it.bh = static_cast<int32_t>(i);
                it.page_begin = at;
                it.page_end = end;
                it.row0 = rb * p->rows_item;
                it.draft = end == pages;
                it.cap = cap[i];
                it.slot = -1;
                p->items.push_back(it);
                done += (end - at) + (at == 0 ? kItemCost : 0);
                at = end;
                if (at == pages) break;
            }
            const int32_t n = static_cast<int32_t>(p->items.size() - first);
            if (n > 1) {
                for (int32_t j = 0; j < n; ++j) {
                    p->items[first + j].slot = first_slot + j;
                    p->slot_page.push_back(p->items[first + j].page_begin);
                }
                p->n_slots += n;
                TreeMerge mg{};
                mg.bh = static_cast<int32_t>(i);
                mg.first_slot = first_slot;
                mg.nsplit = n;
                mg.row0 = rb * p->rows_item;
                mg.cap = cap[i];
                p->merge.push_back(mg);
            }
        }
    while (static_cast<int64_t>(p->worker_off.size()) < nw) p->worker_off.push_back(static_cast<int32_t>(p->items.size()));
    p->worker_off.push_back(static_cast<int32_t>(p->items.size()));
    p->n_workers = static_cast<int32_t>(p->worker_off.size()) - 1;
}

template <int D, int TILES, bool CAP>
int set_smem() {
    TG_TRY(cudaFuncSetAttribute(tree_kernel<D, TILES, CAP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                TreeLayout<D, TILES>::kBytes));
    return TG_OK;
}
template <int D, int TILES>
int set_smem_both() {
    const int rc = set_smem<D, TILES, false>();
    return rc != TG_OK ? rc : set_smem<D, TILES, true>();
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
    const int rc = p->shape.D == 128 ? (p->tiles == 1 ? set_smem_both<128, 1>() : set_smem_both<128, 2>())
                                     : (p->tiles == 1 ? set_smem_both<64, 1>() : set_smem_both<64, 2>());
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
    const int64_t o_spage = take(static_cast<int64_t>(p->slot_page.size()) * 4);
    const int64_t o_lo = take(static_cast<int64_t>(p->row_lo.size()) * 8);
    const int64_t o_hi = take(static_cast<int64_t>(p->row_hi.size()) * 8);
    const int64_t o_err = take(4);
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
    put(o_spage, p->slot_page.data(), p->slot_page.size() * 4);
    put(o_lo, p->row_lo.data(), p->row_lo.size() * 8);
    put(o_hi, p->row_hi.data(), p->row_hi.size() * 8);
    if (cudaMalloc(&p->dev_base, static_cast<size_t>(at)) != cudaSuccess) {
        cudaGetLastError();
        p->dev_base = nullptr;
        return TG_ENOMEM;
    }
    TG_TRY(cudaMemcpy(p->dev_base, img.data(), img.size(), cudaMemcpyHostToDevice));
    unsigned char *d = static_cast<unsigned char *>(p->dev_base);
    p->dev_bytes = at;
    p->d_items = reinterpret_cast<TreeItem *>(d + o_items);
    p->d_worker_off = reinterpret_cast<int32_t *>(d + o_woff);
    p->d_merge = reinterpret_cast<TreeMerge *>(d + o_merge);
    p->d_slot_page = reinterpret_cast<int32_t *>(d + o_spage);
    p->d_row_lo = reinterpret_cast<int64_t *>(d + o_lo);
    p->d_row_hi = reinterpret_cast<int64_t *>(d + o_hi);
    p->d_err = reinterpret_cast<uint32_t *>(d + o_err);
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
    for (int64_t i = 0; i < BH; ++i) {
        if (kv_cap[i] < 0) return TG_EINVAL;
        if (kv_cap[i] > TG_MAX_HEAD_TOKENS) return TG_EUNSUPPORTED;
    }
    for (int32_t g = 0; g < n_groups; ++g)
        if (group_off[g] < 0 || group_off[g + 1] < group_off[g]) return TG_EINVAL;
    for (int32_t h = 0; h < s->Hkv; ++h)
        if (group_of_head[h] < 0 || group_of_head[h] >= n_groups) return TG_EINVAL;

    std::unique_ptr<tg_tree_plan, TreeFree> p(new tg_tree_plan);
    p->shape = *s;
    p->G = G;
    p->max_draft = max_draft;
    p->tiles = max_draft * G > kRows ? 2 : 1;
    p->rows_item = p->tiles == 2 ? 2 * kRows : max_draft * G;
    p->q_rows = p->tiles == 2 ? kRows : (max_draft * G + 7) / 8 * 8;
    p->host_only = host_only != 0;
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
    // one resident wave: two CTAs per SM with one tile, one CTA with two
    const int32_t resident = sms * (p->tiles == 1 ? 2 : 1);
    build_items(p.get(), kv_cap, num_workers > 0 ? num_workers : resident);
    if (!p->host_only) {
        const int rc = tree_device_init(p.get());
        if (rc != TG_OK) return rc;
    }
    *out = p.release();
    return TG_OK;
}

template <int D, int TILES, bool CAP>
int launch_tree(const tg_tree_plan *p, const TreeArgs &a, const CUtensorMap *tm, cudaStream_t stream) {
    using TL = TreeLayout<D, TILES>;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p->n_workers));
    cfg.blockDim = dim3(TL::kThreads);
    cfg.dynamicSmemBytes = TL::kBytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    TG_TRY(cudaLaunchKernelEx(&cfg, tree_kernel<D, TILES, CAP>, a, tm[0], tm[1], tm[2], tm[3], tm[4]));
    return TG_OK;
}

template <int D>
int launch_tree_d(const tg_tree_plan *p, const TreeArgs &a, const CUtensorMap *tm, bool cap, cudaStream_t stream) {
    if (p->tiles == 1) return cap ? launch_tree<D, 1, true>(p, a, tm, stream) : launch_tree<D, 1, false>(p, a, tm, stream);
    return cap ? launch_tree<D, 2, true>(p, a, tm, stream) : launch_tree<D, 2, false>(p, a, tm, stream);
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
                                  int64_t *device_bytes, int32_t *items, int32_t *worker_off) {
    if (!p) return TG_EINVAL;
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
    if (err & kErrTimeout) return TG_ETIMEOUT;
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
    if (!draft_off || !q || !k_draft || !v_draft || !tree_mask || !page_table || !head_page_off || !head_kv_len || !out ||
        !lse || !al16(q) || !al16(k_draft) || !al16(v_draft) || !al16(k_pages) || !al16(v_pages) || !al16(out) ||
        q_stride < qw || k_stride < kw || v_stride < kw || q_stride % 8 != 0 || k_stride % 8 != 0 || v_stride % 8 != 0 ||
        !(scale == scale) || !(softcap >= 0.f) || (s.num_pages > 0 && (!k_pages || !v_pages)))
        return TG_EINVAL;
    int cur = 0;
    TG_TRY(cudaGetDevice(&cur));
    if (cur != p->device) return TG_EINVAL;
    // a pool of no page is never read; its map still needs an address
    const void *kp = s.num_pages > 0 ? k_pages : q, *vp = s.num_pages > 0 ? v_pages : q;
    const int64_t pool = s.num_pages > 0 ? s.num_pages : 1;
    CUtensorMap tm[5];
    int rc = token_map(&tm[0], q, s.D, s.Hq, n_tokens, q_stride, p->G, p->q_rows / p->G);
    if (rc == TG_OK) rc = pool_map(&tm[1], kp, s.D, pool);
    if (rc == TG_OK) rc = pool_map(&tm[2], vp, s.D, pool);
    if (rc == TG_OK) rc = token_map(&tm[3], k_draft, s.D, s.Hkv, n_tokens, k_stride, 1, 16);
    if (rc == TG_OK) rc = token_map(&tm[4], v_draft, s.D, s.Hkv, n_tokens, v_stride, 1, 16);
    if (rc != TG_OK) return rc;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    TreeArgs a{};
    a.items = p->d_items;
    a.worker_off = p->d_worker_off;
    a.G = p->G;
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
        a.cap_in = 2.f * kLog2e * scale / softcap;
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
    rc = s.D == 128 ? launch_tree_d<128>(p, a, tm, softcap > 0.f, st) : launch_tree_d<64>(p, a, tm, softcap > 0.f, st);
    if (rc != TG_OK || p->merge.empty()) return rc;
    TreeMergeArgs g{};
    g.merge = p->d_merge;
    g.slot_page = p->d_slot_page;
    g.draft_off = draft_off;
    g.kv_len = head_kv_len;
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
