// Memory-safety and allocation-failure drive of tg_fork and tg_tree_masks (host code), built with
// AddressSanitizer and UndefinedBehaviorSanitizer by tests/test_spec_sanitizers.py; the device hooks
// that the planner in the same file references are stubbed. Random reservations, forks of forks and
// releases: while a fork is armed its k-th allocation throws, for k = 0, 1, ... until it completes;
// every failing call must return TG_ENOMEM and leave reference counts, free pages and the known
// sequences as they were. Page accounting is exact throughout.
#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <map>
#include <new>
#include <random>
#include <vector>

#include "tg.h"
#include "tg_internal.h"

namespace tg {
int device_init_plan(tg_plan *) { return TG_EUNSUPPORTED; }
void device_free_plan(tg_plan *) {}
int device_num_sms(int, int *n) {
    *n = 148;
    return TG_OK;
}
void set_cuda_error(const char *, int) {}
}  // namespace tg

static bool g_armed = false, g_hit = false;
static long g_left = -1;
static void *take(std::size_t n) {
    if (g_armed && g_left-- == 0) {
        g_hit = true;
        throw std::bad_alloc();
    }
    void *p = std::malloc(n ? n : 1);
    if (!p) throw std::bad_alloc();
    return p;
}
void *operator new(std::size_t n) { return take(n); }
void *operator new[](std::size_t n) { return take(n); }
void operator delete(void *p) noexcept { std::free(p); }
void operator delete[](void *p) noexcept { std::free(p); }
void operator delete(void *p, std::size_t) noexcept { std::free(p); }
void operator delete[](void *p, std::size_t) noexcept { std::free(p); }

#define CHECK(x)                                                     \
    do {                                                             \
        if (!(x)) {                                                  \
            std::fprintf(stderr, "line %d: %s\n", __LINE__, #x);     \
            std::abort();                                            \
        }                                                            \
    } while (0)

static std::mt19937_64 g_rng;
static int64_t uni(int64_t lo, int64_t hi) { return lo + static_cast<int64_t>(g_rng() % static_cast<uint64_t>(hi - lo + 1)); }

static long drive(uint64_t seed) {
    g_rng.seed(seed);
    const int32_t pages = 400, H = static_cast<int32_t>(uni(1, 4));
    long injected = 0;
    tg_alloc *a = nullptr;
    CHECK(tg_alloc_create(pages, 16, seed, &a) == TG_OK);
    struct Live {
        std::vector<int32_t> kv, ids;
    };
    std::map<int32_t, Live> live;
    auto refs = [&] {
        std::vector<int32_t> r;
        for (int32_t p = 0; p < pages; ++p) r.push_back(tg_alloc_refcount(a, p));
        return r;
    };
    auto exact = [&] {
        std::vector<int32_t> want(pages, 0);
        for (auto &kv : live)
            for (int32_t id : kv.second.ids) ++want[id];
        CHECK(refs() == want);
        CHECK(tg_alloc_free_pages(a) == std::count(want.begin(), want.end(), 0));
    };
    int32_t next = 0;
    for (int step = 0; step < 120; ++step, ++next) {
        const int64_t what = uni(0, 9);
        if (live.empty() || what < 3) {
            Live l;
            int64_t cap = 0;
            for (int32_t h = 0; h < H; ++h) {
                l.kv.push_back(static_cast<int32_t>(uni(0, 120)));
                cap += (l.kv.back() + 15) / 16;
            }
            l.ids.resize(static_cast<size_t>(cap));
            int64_t n = 0;
            const int rc = tg_reserve(a, next, H, l.kv.data(), 0, nullptr, l.ids.data(), cap, nullptr, &n);
            CHECK(rc == TG_OK || rc == TG_ENOSPC);
            if (rc == TG_OK) live[next] = l;
        } else if (what < 8) {
            auto it = live.begin();
            std::advance(it, uni(0, static_cast<int64_t>(live.size()) - 1));
            Live l;
            std::vector<int32_t> held, shared;
            int64_t cap = 0, copies = 0;
            for (int32_t h = 0; h < H; ++h) {
                held.push_back(static_cast<int32_t>(uni(0, it->second.kv[h])));
                shared.push_back(static_cast<int32_t>(uni(0, held.back() / 16)));
                l.kv.push_back(held.back() + static_cast<int32_t>(uni(0, 40)));
                cap += (l.kv.back() + 15) / 16;
                copies += (held.back() + 15) / 16 - shared.back();
            }
            l.ids.resize(static_cast<size_t>(cap));
            std::vector<int32_t> src(copies), dst(copies), rows(copies), count(H);  // exactly as large as needed
            int64_t n = 0, m = 0;
            const auto before = refs();
            const int64_t free_before = tg_alloc_free_pages(a);
            for (long k = 0;; ++k) {
                g_left = k;
                g_hit = false;
                g_armed = true;
                const int rc = tg_fork(a, it->first, next, H, held.data(), l.kv.data(), shared.data(), l.ids.data(), cap,
                                       count.data(), src.data(), dst.data(), rows.data(), copies, &m, &n);
                g_armed = false;
                if (!g_hit) {
                    CHECK(rc == TG_OK || rc == TG_ENOSPC);
                    if (rc == TG_OK) {
                        CHECK(n == cap && m == copies);
                        live[next] = l;
                    }
                    break;
                }
                ++injected;
                CHECK(rc == TG_ENOMEM && refs() == before && tg_alloc_free_pages(a) == free_before);
                CHECK(tg_release(a, next) == TG_ENOTFOUND);
            }
            // a buffer one too small is refused
            if (cap > 0) {
                int64_t z = 0;
                CHECK(tg_fork(a, it->first, 100000, H, held.data(), l.kv.data(), shared.data(), l.ids.data(), cap - 1, nullptr,
                              src.data(), dst.data(), rows.data(), copies, &z, nullptr) == TG_EINVAL);
            }
        } else {
            auto it = live.begin();
            std::advance(it, uni(0, static_cast<int64_t>(live.size()) - 1));
            CHECK(tg_release(a, it->first) == TG_OK);
            live.erase(it);
        }
        exact();
    }
    tg_alloc_destroy(a);

    const int32_t B = static_cast<int32_t>(uni(0, 6));
    std::vector<int32_t> off(1, 0), parent;
    for (int32_t b = 0; b < B; ++b) {
        const int32_t n = static_cast<int32_t>(uni(0, 64));
        for (int32_t j = 0; j < n; ++j) parent.push_back(static_cast<int32_t>(uni(-1, j - 1)));
        off.push_back(off.back() + n);
    }
    std::vector<uint64_t> mask(parent.size());
    CHECK(tg_tree_masks(B, off.data(), parent.data(), mask.data()) == TG_OK);
    for (int32_t b = 0; b < B; ++b)
        for (int32_t j = 0; j < off[b + 1] - off[b]; ++j) {
            uint64_t want = 0;
            for (int32_t k = j; k >= 0; k = parent[off[b] + k]) want |= 1ull << k;
            CHECK(mask[off[b] + j] == want);
        }
    return injected;
}

int main() {
    long injected = 0;
    for (uint64_t s = 1; s <= 40; ++s) injected += drive(s);
    CHECK(injected > 100);
    std::printf("%ld injected failures\n", injected);
    return 0;
}
