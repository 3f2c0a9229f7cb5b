// Moving retained tokens between pages: page copies (a forked sequence's own copies of pages it
// will write, a tier copied for a new reader) and the compaction of a prompt's rows to the budget
// pages of each head.
//
// Sources: "Tangram" explainer, 三大机制 1 (Budget Reservation: a head holds only its budget after
// compression, in pages reserved at admission) and RadixAttention lesson, Phase 17 · 06 (a node's
// pages are shared until a request departs from them; the partial page is the reader's own).
//
// Both kernels only move bytes: each row is read once and written once, 16 bytes a lane.
#include <cuda_runtime.h>
#include <climits>
#include <cstdint>

#include "tg.h"
#include "tg_internal.h"
#include "tg_ptx.cuh"

namespace tg {
namespace {

constexpr int kCopyWarps = 8;
constexpr int kCopyVec = 8;     // 16-byte vectors of a lane in flight
constexpr int kCompactWarps = 8;

struct CopyArgs {
    const int32_t *src, *dst, *rows;
    int64_t n, num_pages;
    uint4 *pool[2];
    float *scale[2];
    int32_t row_vec;  // 16-byte vectors per row
    int32_t *n_bad;
};

// One warp per (pair, K or V): a page's first `rows` rows are one contiguous run of bytes in the
// pool, copied kCopyVec vectors a lane at a time (a whole bf16 page of D = 128 is one round). Bound:
// DRAM: 554 MB of INT8 pages with their scales read and written in 94.5 us, 5.86 TB/s; few pages: the
// load's and the store's latency (the tails of a fork 1.8 us, 2.6 us with one warp for K and V).
__global__ void __launch_bounds__(kCopyWarps * 32) copy_pages_kernel(const __grid_constant__ CopyArgs a) {
    const int64_t w = static_cast<int64_t>(blockIdx.x) * kCopyWarps + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    const int64_t i = w >> 1;
    const int side = static_cast<int>(w & 1);
    ptx::grid_wait();
    if (i >= a.n) return;
    const int64_t s = a.src[i], d = a.dst[i];
    const int32_t rows = a.rows ? a.rows[i] : 16;
    if (s < 0 || s >= a.num_pages || d < 0 || d >= a.num_pages || rows < 0 || rows > 16) {
        if (side == 0 && lane == 0) atomicAdd(a.n_bad, 1);
        return;
    }
    if (s == d) return;
    const int total = rows * a.row_vec;
    const uint4 *from = a.pool[side] + s * 16 * a.row_vec;
    uint4 *to = a.pool[side] + d * 16 * a.row_vec;
    float sc = 0.f;
    const bool has = a.scale[side] && lane < rows;
    if (has) sc = a.scale[side][s * 16 + lane];
    for (int v0 = 0; v0 < total; v0 += 32 * kCopyVec) {
        uint4 x[kCopyVec];
#pragma unroll
        for (int j = 0; j < kCopyVec; ++j)
            if (v0 + j * 32 + lane < total) x[j] = from[v0 + j * 32 + lane];
#pragma unroll
        for (int j = 0; j < kCopyVec; ++j)
            if (v0 + j * 32 + lane < total) to[v0 + j * 32 + lane] = x[j];
    }
    if (has) a.scale[side][d * 16 + lane] = sc;
}

struct CompactArgs {
    int32_t BH, row_vec;
    int64_t n_keep, src_pages, num_pages;
    const uint4 *k_src, *v_src;
    uint4 *k_dst, *v_dst;
    const int32_t *src_table, *table, *src_len, *budget;
    const int64_t *src_off, *off, *keep_off;
    const int32_t *keep;
    int32_t *kv_len, *n_bad;
};

// Number of rows head bh keeps, or -1 when its list is not usable (out of order, outside keep,
// longer than its budget).
__device__ __forceinline__ int64_t kept_rows(const CompactArgs &a, int32_t bh) {
    const int64_t b = a.keep_off[bh], e = a.keep_off[bh + 1];
    return b < 0 || e < b || e > a.n_keep || e - b > max(0, a.budget[bh]) ? -1 : e - b;
}

// The head that entry i of keep is taken for: the last one whose list starts at or before i, by bisection
// of keep_off (the same few cached words for every lane). With offsets out of order a list may have
// entries that another head is found for, or share some with another list. [from, to) is the run of
// entries around i that bisect the same way: a list that lies in the run of its first entry is found by
// every entry of it, and any of its entries can tell. The others are copied by their head's warp.
struct Owner {
    int32_t head;
    int64_t from, to;
    __device__ __forceinline__ Owner(const CompactArgs &a, int64_t i) : head(0), from(LLONG_MIN), to(LLONG_MAX) {
        for (int32_t hi = a.BH; hi - head > 1;) {
            const int32_t mid = (head + hi) >> 1;
            const int64_t at = a.keep_off[mid];
            if (at <= i) {
                head = mid;
                from = max(from, at);
            } else {
                hi = mid;
                to = min(to, at);
            }
        }
    }
    __device__ __forceinline__ bool owns(int64_t first, int64_t m) const { return from <= first && first + m <= to; }
};

// Pool rows of head bh's token `to` and of its source, entry i of keep; false when either is out of bounds.
__device__ __forceinline__ bool kept_row(const CompactArgs &a, int32_t bh, int64_t i, int64_t to, int64_t &src, int64_t &dst) {
    const int32_t from = a.keep[i];
    int64_t sp = -1;
    const int64_t dp = a.table[a.off[bh] + to / 16];
    if (from >= 0 && from < a.src_len[bh]) sp = a.src_table[a.src_off[bh] + from / 16];
    if (sp < 0 || sp >= a.src_pages || dp < 0 || dp >= a.num_pages) return false;
    src = sp * 16 + from % 16;
    dst = dp * 16 + to % 16;
    return true;
}

// One warp: the whole list of head bh, a row at a time.
__device__ __noinline__ void compact_apart(const CompactArgs &a, int32_t bh, int lane) {
    const int64_t first = a.keep_off[bh], m = kept_rows(a, bh);
    for (int64_t to = 0; to < m; ++to) {
        int64_t src, dst;
        if (!kept_row(a, bh, first + to, to, src, dst)) {
            if (lane == 0) atomicAdd(a.n_bad, 1);
            continue;
        }
        for (int c = lane; c < a.row_vec; c += 32) {
            a.k_dst[dst * a.row_vec + c] = a.k_src[src * a.row_vec + c];
            a.v_dst[dst * a.row_vec + c] = a.v_src[src * a.row_vec + c];
        }
    }
}

// One warp per TPW entries of the keep list, whatever heads they belong to, so heads of very
// different budgets cost the same per row. Lane l finds entry l's head, its source and destination
// rows; then the warp copies the K rows and the V rows 16 bytes a lane, the rows' addresses by shuffle. Bound: DRAM
// (figures at the launch); short lists: the search's dependent loads, then one round of copies.
template <int TPW>
__global__ void __launch_bounds__(kCompactWarps * 32) compact_kernel(const __grid_constant__ CompactArgs a) {
    constexpr unsigned FULL = 0xffffffffu;
    const int lane = threadIdx.x & 31;
    const int64_t gtid = static_cast<int64_t>(blockIdx.x) * (kCompactWarps * 32) + threadIdx.x;
    ptx::grid_wait();
    bool apart = false;  // this thread's head is not found by its entries
    if (gtid < a.BH) {
        const int64_t m = kept_rows(a, static_cast<int32_t>(gtid));
        if (m > 0) {
            const int64_t first = a.keep_off[gtid];
            const Owner o(a, first);
            apart = o.head != gtid || !o.owns(first, m);
        }
        a.kv_len[gtid] = m < 0 ? 0 : static_cast<int32_t>(m);
        if (m < 0) atomicAdd(a.n_bad, 1);
    }
    const int64_t i = (gtid >> 5) * TPW + lane;  // keep-list entry of this lane
    int64_t src = -1, dst = -1;
    if (lane < TPW && i < a.n_keep) {
        const Owner o(a, i);
        const int32_t lo = o.head;
        const int64_t first = a.keep_off[lo];
        const int64_t m = kept_rows(a, lo);
        if (first <= i && i - first < m && o.owns(first, m)) {
            if (!kept_row(a, lo, i, i - first, src, dst)) atomicAdd(a.n_bad, 1);
        }
    }
    for (uint32_t rest = __ballot_sync(FULL, apart); rest; rest &= rest - 1)
        compact_apart(a, static_cast<int32_t>(gtid - lane) + __ffs(static_cast<int>(rest)) - 1, lane);
    if (!__any_sync(FULL, src >= 0)) return;
    // vector v of the warp's rows: row v / row_vec, K first, then V
    const int per = TPW * a.row_vec;
    for (int v0 = 0; v0 < 2 * per; v0 += 32 * kCopyVec) {
        uint4 x[kCopyVec];
        uint4 *to[kCopyVec];
#pragma unroll
        for (int j = 0; j < kCopyVec; ++j) {
            const int v = v0 + j * 32 + lane;
            const bool is_v = v >= per;
            const int u = is_v ? v - per : v;
            const int r = u / a.row_vec, c = u - r * a.row_vec;
            const int64_t s = __shfl_sync(FULL, src, r & 31), d = __shfl_sync(FULL, dst, r & 31);
            to[j] = nullptr;
            if (v < 2 * per && s >= 0) {
                x[j] = (is_v ? a.v_src : a.k_src)[s * a.row_vec + c];
                to[j] = (is_v ? a.v_dst : a.k_dst) + d * a.row_vec + c;
            }
        }
#pragma unroll
        for (int j = 0; j < kCopyVec; ++j)
            if (to[j]) *to[j] = x[j];
    }
}

bool al16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <class A>
int launch(void (*kern)(A), const A &a, int64_t ctas, int threads, tg_stream stream, const char *what) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, a);
    if (e != cudaSuccess) {
        set_cuda_error(what, static_cast<int>(e));
        return TG_ECUDA;
    }
    return TG_OK;
}

}  // namespace
}  // namespace tg

using namespace tg;

extern "C" int tg_copy_pages(int64_t num_pages, int32_t row_bytes, int64_t n_copies, const int32_t *src_page,
                             const int32_t *dst_page, const int32_t *rows, void *k_pool, void *v_pool, float *k_scale,
                             float *v_scale, int32_t *n_bad, tg_stream stream) {
    if (num_pages < 0 || row_bytes < 1 || n_copies < 0 || n_copies > INT32_MAX) return TG_EINVAL;
    if (row_bytes % 16 != 0 || row_bytes > 4096) return TG_EUNSUPPORTED;
    if (n_copies == 0) return TG_OK;
    if (!src_page || !dst_page || !k_pool || !v_pool || !n_bad || !al16(k_pool) || !al16(v_pool) ||
        !k_scale != !v_scale)
        return TG_EINVAL;
    CopyArgs a{};
    a.src = src_page;
    a.dst = dst_page;
    a.rows = rows;
    a.n = n_copies;
    a.num_pages = num_pages;
    a.pool[0] = static_cast<uint4 *>(k_pool);
    a.pool[1] = static_cast<uint4 *>(v_pool);
    a.scale[0] = k_scale;
    a.scale[1] = v_scale;
    a.row_vec = row_bytes / 16;
    a.n_bad = n_bad;
    return launch(copy_pages_kernel, a, (2 * n_copies + kCopyWarps - 1) / kCopyWarps, kCopyWarps * 32, stream,
                  "copy_pages_kernel");
}

extern "C" int tg_compact_kv(const tg_shape *s, int64_t src_num_pages, const void *k_src, const void *v_src,
                             const int32_t *src_table, const int64_t *src_head_off, const int32_t *src_len,
                             const int64_t *keep_off, const int32_t *keep_idx, int64_t n_keep, void *k_pages,
                             void *v_pages, const int32_t *page_table, const int64_t *head_page_off,
                             const int32_t *head_budget, int32_t *head_kv_len, int32_t *n_bad, tg_stream stream) {
    if (!s || s->B < 0 || s->Hkv < 1 || s->page != 16 || s->D < 8 || s->D % 8 != 0 || s->num_pages < 0 ||
        static_cast<int64_t>(s->B) * s->Hkv > INT32_MAX || src_num_pages < 0 || n_keep < 0 ||
        n_keep > static_cast<int64_t>(INT32_MAX) * 64)
        return TG_EINVAL;
    if (s->D > 2048) return TG_EUNSUPPORTED;
    const int32_t BH = s->B * s->Hkv;
    if (BH == 0) return TG_OK;
    if (!keep_off || !head_budget || !head_kv_len || !n_bad) return TG_EINVAL;
    if (n_keep > 0 && (!k_src || !v_src || !src_table || !src_head_off || !src_len || !keep_idx || !k_pages ||
                       !v_pages || !page_table || !head_page_off))
        return TG_EINVAL;
    if (!al16(k_src) || !al16(v_src) || !al16(k_pages) || !al16(v_pages)) return TG_EINVAL;
    CompactArgs a{};
    a.BH = BH;
    a.row_vec = s->D / 8;
    a.n_keep = n_keep;
    a.src_pages = src_num_pages;
    a.num_pages = s->num_pages;
    a.k_src = static_cast<const uint4 *>(k_src);
    a.v_src = static_cast<const uint4 *>(v_src);
    a.k_dst = static_cast<uint4 *>(k_pages);
    a.v_dst = static_cast<uint4 *>(v_pages);
    a.src_table = src_table;
    a.table = page_table;
    a.src_len = src_len;
    a.budget = head_budget;
    a.src_off = src_head_off;
    a.off = head_page_off;
    a.keep_off = keep_off;
    a.keep = keep_idx;
    a.kv_len = head_kv_len;
    a.n_bad = n_bad;
    // 32 entries a warp (1.3 M kept rows of D = 128: 224 us, 6.0 TB/s, against 272 us with 8); lists too
    // short to give every SM 16 such warps go 8 entries a warp (17 000 rows: 5.2 us against 9.5 us)
    const bool few = n_keep < 148 * 16 * 32;
    const int64_t threads = few ? (n_keep + 7) / 8 * 32 : n_keep;
    const int64_t most = threads > BH ? threads : BH;
    return launch(few ? compact_kernel<8> : compact_kernel<32>, a,
                  (most + kCompactWarps * 32 - 1) / (kCompactWarps * 32), kCompactWarps * 32, stream, "compact_kernel");
}
