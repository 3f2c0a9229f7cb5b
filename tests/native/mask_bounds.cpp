// tg_tree_masks with offsets out of order, built with AddressSanitizer by tests/test_spec_contract.py:
// the call must refuse them before it reads a parent, since the array holds draft_off[B] of them only
// where the offsets ascend.
#include <cstdint>
#include <cstdio>
#include <cstdlib>
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

static void refused(std::vector<int32_t> off) {
    off.shrink_to_fit();
    const int32_t B = static_cast<int32_t>(off.size()) - 1, n = off[B] > 0 ? off[B] : 0;
    std::vector<int32_t> parent(static_cast<size_t>(n), -1);
    std::vector<uint64_t> mask(static_cast<size_t>(n), 7);
    if (tg_tree_masks(B, off.data(), parent.data(), mask.data()) != TG_EINVAL) std::abort();
    for (uint64_t m : mask)
        if (m != 7) std::abort();
}

int main() {
    refused({0, 5, 3});
    refused({0, 40, 40, 4});
    refused({0, 2, 66, 130, 1});
    refused({0, 1, 2147483647, 3});
    refused({0, 64, 0});
    refused({0, 8, 8, -2147483647});
    std::puts("refused");
    return 0;
}
