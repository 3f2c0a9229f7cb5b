"""What the header promises of the speculative step at its edges (one B200): results that depend on
nothing but what they are a function of, bit for bit."""
import pytest
import torch

import non_uniform_paged_flash_b200 as tg
from tests.test_gpu_tree import Batch

pytestmark = pytest.mark.gpu


def bits(bt, rows, **kw):
    bt.out.fill_(7)
    bt.lse.fill_(7)
    bt.run(**kw)
    torch.cuda.synchronize()
    assert tg.tg_tree_plan_status(bt.plan) == tg.TG_OK
    return bt.out[rows].clone(), bt.lse[rows].clone()


def same(a, b):
    return torch.equal(a[0].view(torch.int16), b[0].view(torch.int16)) and torch.equal(a[1].view(torch.int32), b[1].view(torch.int32))


# ---- tree attention, kernel of few rows: every row's base is its own ----

@pytest.mark.parametrize("G,nd", [(4, [2, 4]), (1, [5, 16]), (2, [1, 8])])
def test_other_sequences_queries_leave_a_sequence_alone(G, nd):
    """The rows behind a short draft hold the next sequence's queries: however far their scores go, the
    sequence's own bits stay."""
    bt = Batch(31, G, 128, 2, [100, 33, 260, 17], nd, few=True)
    first = slice(0, nd[0])
    a = bits(bt, first)
    bt.q[nd[0]:] *= 40
    assert same(a, bits(bt, first))


@pytest.mark.parametrize("G,T", [(4, 4), (1, 9), (2, 7)])
@pytest.mark.parametrize("factor", [60.0, 1e30])
def test_finite_masked_drafted_keys_leave_their_non_readers_alone(G, T, factor):
    """A drafted key far from the others moves the base of the rows that attend to it and no other."""
    masks = [1 << j for j in range(T)]
    masks = [m | (2 if j in (3, T - 1) else 0) for j, m in enumerate(masks)]
    others = [t for t in range(T) if not masks[t] >> 1 & 1]
    bt = Batch(32, G, 128, 2, [300, 17], [T], masks=masks, few=True)
    a = bits(bt, others)
    bt.k[1] = (bt.k[1].float() * factor).clamp(-1e37, 1e37).bfloat16()
    assert same(a, bits(bt, others))
