"""What the header promises of the speculative step at its edges (one B200): results that depend on
nothing but what they are a function of, bit for bit."""
import numpy as np
import pytest
import torch

import non_uniform_paged_flash_b200 as tg
from tests import _spec as sp
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


# ---- tree attention: only the scores that count choose the arithmetic, under a cap above all ----

FORMS = [(4, 128, [3, 4, 1], True), (4, 128, [3, 4, 1], False), (4, 64, [3, 4, 1], False), (1, 128, [20, 9, 3], False),
         (8, 128, [12, 9, 3], False), (8, 128, [30, 9, 3], False)]


@pytest.mark.parametrize("G,D,nd,few", FORMS)
@pytest.mark.parametrize("cap", [30.0, 0.0])
def test_scores_ignore_stale_rows(G, D, nd, few, cap):
    """Whatever the pages' rows past a head's tokens hold, small, far or NaN: the same bits."""
    got = []
    for stale in (1e-3, 1e4, float("nan")):
        bt = Batch(33, G, D, 2, [1, 17, 63, 66, 0, 129], nd, stale=stale, cap_extra=40, few=few)
        got.append(bits(bt, slice(None), softcap=cap))
        bt.check(softcap=cap)
    assert same(got[0], got[1]) and same(got[0], got[2])


@pytest.mark.parametrize("G,D,nd,few", FORMS)
@pytest.mark.parametrize("cap", [30.0, 0.0])
def test_scores_ignore_earlier_items(G, D, nd, few, cap):
    """One worker takes a long head and then short ones: what the long one left in shared memory does not
    reach them."""
    bt = Batch(34, G, D, 1, [700, 10, 3], nd, few=few, workers=1)
    rest = slice(nd[0], sum(nd))
    a = bits(bt, rest, softcap=cap)
    rows = torch.from_numpy(sp.head_rows(bt.ids, bt.off, 0, 700)).cuda()
    for x in ("kp", "vp"):
        bt.dev[x].view(-1, D)[rows] *= 1000
    assert same(a, bits(bt, rest, softcap=cap))


@pytest.mark.parametrize("G,D,nd,few", FORMS)
@pytest.mark.parametrize("cap", [30.0, 0.0])
def test_scores_ignore_other_sequences_queries(G, D, nd, few, cap):
    bt = Batch(35, G, D, 2, [100, 33, 260, 17, 0, 5], nd, few=few)
    first = slice(0, nd[0])
    a = bits(bt, first, softcap=cap)
    bt.q[nd[0]:] *= 100
    assert same(a, bits(bt, first, softcap=cap))


@pytest.mark.parametrize("G,D,T,few", [(4, 128, 4, True), (1, 128, 9, True), (4, 128, 9, False), (4, 64, 9, False),
                                       (8, 128, 33, False)])
@pytest.mark.parametrize("value", [40.0, 1e30, float("inf"), float("nan")])
@pytest.mark.parametrize("cap", [30.0, 0.0])
def test_scores_ignore_masked_drafted_keys(G, D, T, few, value, cap):
    masks = [1 << j for j in range(T)]
    masks = [m | (2 if j in (3, T - 1) else 0) for j, m in enumerate(masks)]
    others = [t for t in range(T) if not masks[t] >> 1 & 1]
    bt = Batch(36, G, D, 1, [37], [T], masks=masks, few=few)
    a = bits(bt, others, softcap=cap)
    bt.k[1] = value
    assert same(a, bits(bt, others, softcap=cap))


@pytest.mark.parametrize("G,D,nd,few", FORMS)
@pytest.mark.parametrize("cap", [15.0, 30.0])
def test_capped_scores_near_and_far(G, D, nd, few, cap):
    """Small and large scores side by side: rows of both kinds in a warp, tokens of both kinds in a row."""
    bt = Batch(37, G, D, 2, [100, 33, 260, 64, 129, 5], nd, few=few)
    bt.q[::2] *= 20
    bt.dev["kp"][::3] *= 8
    bt.run(softcap=cap)
    bt.check(softcap=cap)


@pytest.mark.parametrize("T,few", [(4, False), (16, False), (40, False), (4, True)])
def test_capped_repeats_are_bit_equal(T, few):
    """Dynamic items, scores on both sides of the forms' border."""
    rng = np.random.default_rng(2)
    bt = Batch(38, 4, 128, 2, rng.integers(0, 2000, size=40), [T, 2, 3, 1] * 5, workers=20, few=few)
    bt.q[::3] *= 8
    a = bits(bt, slice(None), softcap=15.0)
    for _ in range(10):
        assert same(a, bits(bt, slice(None), softcap=15.0))


# ---- compaction: a head's length never counts rows that were not written ----

@pytest.mark.parametrize("koff,budget", [([0, 10, 5, 15], [20] * 3), ([0, 4, 2, 50, 130], [40] * 4),
                                         ([0, 10, 5, 7, 12, 40, 40, 60], [40] * 7), ([0, 10, 10, 15, 120], [20, 0, 5, 105]),
                                         ([100, 120, 0, 20, 10, 30], [25] * 5), ([-3, 5, 9], [9, 9])]
                         + [(None, seed) for seed in range(12)])
@pytest.mark.parametrize("D", [64, 512])
def test_compact_offsets_in_any_order(koff, budget, D):
    """Each head's own offsets decide about its list, whatever the others are: in order, within the keep
    list and within the budget, all of it is written and counted, though another list may name the same
    entries; else none of it."""
    rng = np.random.default_rng(0 if koff else budget)
    if koff is None:
        BH = int(rng.integers(1, 80))
        koff = np.sort(rng.integers(0, 121, size=BH + 1))
        for _ in range(int(rng.integers(0, 5))):
            koff[rng.integers(0, BH + 1)] = rng.integers(-30, 180)
        budget = rng.integers(0, 121, size=BH)
    BH, koff, budget = len(koff) - 1, np.asarray(koff, np.int64), np.asarray(budget, np.int32)
    n_keep = 120
    keep = rng.integers(0, 200, size=n_keep).astype(np.int32)
    sids, soff, spool = sp.tables(rng, np.full(BH, 13))
    ids, off, pool = sp.tables(rng, -(-budget.astype(np.int64) // 16))
    ks, vs = (sp.bf16(rng, spool, 16, D).cuda() for _ in range(2))
    kd, vd = (sp.bf16(rng, pool, 16, D).cuda() for _ in range(2))
    exp = [kd.cpu().view(-1, D).clone(), vd.cpu().view(-1, D).clone()]
    n = torch.full((BH,), 9, dtype=torch.int32, device="cuda")
    bad = torch.zeros(1, dtype=torch.int32, device="cuda")
    cu = lambda a, t=None: torch.from_numpy(np.ascontiguousarray(a if t is None else a.astype(t))).cuda()
    tg.tg_compact_kv(tg.make_shape(1, BH, BH, D, pool), ks, vs, cu(sids), cu(soff), cu(np.full(BH, 200), np.int32), cu(koff),
                     cu(keep), kd, vd, cu(ids if ids.size else np.zeros(1, np.int32)), cu(off), cu(budget), n, bad)
    m = np.diff(koff)
    usable = (koff[:-1] >= 0) & (m >= 0) & (koff[1:] <= n_keep) & (m <= budget)
    assert n.cpu().tolist() == np.where(usable, m, 0).tolist() and int(bad) == int((~usable).sum())
    for i in np.flatnonzero(usable):
        to, frm = sp.head_rows(ids, off, i, int(m[i])), sp.head_rows(sids, soff, i, 200)[keep[koff[i]:koff[i + 1]]]
        for e, x in zip(exp, (ks, vs)):
            e[to] = x.cpu().view(-1, D)[frm]
    assert torch.equal(kd.cpu().view(-1, D), exp[0]) and torch.equal(vd.cpu().view(-1, D), exp[1])


# ---- caps at the ends of their range ----

@pytest.mark.parametrize("softcap", [1e-45, 1e-40, 1e-37, 1e30])
@pytest.mark.parametrize("D,few", [(64, False), (128, False), (128, True)])
def test_caps_near_the_ends_of_fp32(softcap, D, few):
    """A cap too small to divide by, and one too large to matter, with scores of zero among them."""
    bt = Batch(39, 4, D, 2, [100, 33, 0, 17], [4, 3], few=few)
    bt.q[::2] = 0
    bt.run(softcap=softcap)
    bt.check(softcap=softcap)
