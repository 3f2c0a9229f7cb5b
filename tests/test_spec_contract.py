"""What the header promises of the speculative step's host side, at its edges (CPU)."""
import numpy as np
import pytest

import non_uniform_paged_flash_b200 as tg


def _plan(cap, T=4, Hq=8, Hkv=2, D=128, pages=1 << 20, workers=0):
    B = np.asarray(cap).size // Hkv
    return tg.tg_tree_plan_create(tg.make_shape(B, Hq, Hkv, D, pages), cap, T, np.zeros(Hkv, np.int32), [0, 1 << 20],
                                  num_workers=workers, host_only=True)


@pytest.mark.parametrize("cap,ok", [([0, 0], True), ([0, 1], False), ([40, 0], False)])
def test_plan_needs_a_pool_for_reserved_tokens(cap, ok):
    """Heads that reserve tokens need pages to hold them: with an empty pool there is no page a bad
    page id could be replaced by."""
    if ok:
        assert tg.tg_tree_plan_items(_plan(cap, pages=0))["n_items"] == 2
        return
    with pytest.raises(tg.TGError) as e:
        _plan(cap, pages=0)
    assert e.value.status == tg.TG_EINVAL
