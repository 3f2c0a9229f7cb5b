"""Tree attention of drafted tokens over the ragged paged cache against a plain 64-bit form: head
layouts, draft widths, lengths around page and block ends, split and unsplit plans, capped scores,
masked places that hold NaN or infinities, rows that see nothing, and the ways a caller may run it.
Tolerances are the roundings the kernel makes (see _spec.tree_reference)."""
import math

import numpy as np
import pytest
import torch

import non_uniform_paged_flash_b200 as tg
from tests import _spec as sp

pytestmark = pytest.mark.gpu


class Batch:
    """A random ragged batch on the GPU with its plan."""

    def __init__(self, seed, G, D, Hkv, lens, nd, max_draft=None, cap_extra=0, workers=0, q_scale=1.5, stale=0.0,
                 extra_rows=0, masks=None, fused=True, few=False):
        rng = np.random.default_rng(seed)
        if few:  # one more sequence, long enough for the kernel of few rows
            units = np.size(lens) // Hkv + 1
            lens = np.concatenate([np.ravel(lens), np.full(Hkv, 20 * 16 * units - 7)])
            nd = np.concatenate([nd, [1]])
            max_draft = max_draft or int(np.max(nd))
            if masks is not None:
                masks = list(masks) + [1]
        self.G, self.D, self.Hkv, self.Hq = G, D, Hkv, G * Hkv
        self.lens = np.asarray(lens, np.int64).reshape(-1)
        self.B = self.lens.size // Hkv
        cap = self.lens + cap_extra
        self.ids, self.off, self.pool = sp.tables(rng, -(-cap // 16))
        self.nd = np.asarray(nd, np.int64)
        self.doff = np.concatenate([[0], np.cumsum(self.nd)]).astype(np.int32)
        self.N = int(self.doff[-1]) + extra_rows
        self.k_pages, self.v_pages = (sp.bf16(rng, self.pool, 16, D) for _ in range(2))
        self.mask = sp.random_masks(rng, self.nd) if masks is None else np.asarray(masks, np.uint64)
        self.mask = np.concatenate([self.mask, np.full(extra_rows, 2**64 - 1, np.uint64)])
        qkv = sp.bf16(rng, self.N, self.Hq + 2 * Hkv, D)
        qkv[:, :self.Hq] *= q_scale
        dev = qkv.cuda()
        self.q, self.k, self.v = dev[:, :self.Hq], dev[:, self.Hq:self.Hq + Hkv], dev[:, self.Hq + Hkv:]
        if not fused:
            self.q, self.k, self.v = (x.contiguous() for x in (self.q, self.k, self.v))
        self.cap = cap
        if stale:  # rows of the pool that hold no retained token
            held = np.zeros(self.pool * 16, bool)
            for i in range(self.lens.size):
                held[sp.head_rows(self.ids, self.off, i, int(self.lens[i]))] = True
            for pages in (self.k_pages, self.v_pages):
                pages.view(-1, D)[torch.from_numpy(~held)] = stale
        self.shape = tg.make_shape(self.B, self.Hq, Hkv, D, self.pool)
        self.plan = tg.tg_tree_plan_create(self.shape, cap, max_draft or max(1, int(self.nd.max(initial=1))),
                                           np.zeros(Hkv, np.int32), [0, max(1, self.ids.size)], num_workers=workers,
                                           wait_limit_us=1000000)
        self.rows = tg.tg_tree_plan_items(self.plan)["rows"]
        assert not few or self.rows == 16
        self.scale = 1 / math.sqrt(D)
        self.dev = dict(kp=self.k_pages.cuda(), vp=self.v_pages.cuda(),
                        table=torch.from_numpy(self.ids if self.ids.size else np.zeros(1, np.int32)).cuda(),
                        off=torch.from_numpy(self.off).cuda(),
                        n=torch.from_numpy(self.lens.astype(np.int32)).cuda(),
                        doff=torch.from_numpy(self.doff).cuda(),
                        mask=torch.from_numpy(self.mask.view(np.int64)).cuda())
        self.out = torch.full((self.N, self.Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((self.N, self.Hq), 7.0, device="cuda")

    def run(self, softcap=0.0, scale=None, stream=None):
        d = self.dev
        tg.tg_tree_decode(self.plan, d["doff"], self.q, self.k, self.v, d["mask"], d["kp"], d["vp"], d["table"],
                          d["off"], d["n"], self.scale if scale is None else scale, softcap, self.out, self.lse,
                          stream=stream)

    def reference(self, softcap=0.0, scale=None):
        rows = [sp.head_rows(self.ids, self.off, i, int(self.lens[i])) for i in range(self.lens.size)]
        K, V = self.dev["kp"].cpu().view(-1, self.D), self.dev["vp"].cpu().view(-1, self.D)
        return sp.tree_reference(self.q.cpu(), self.k.cpu(), self.v.cpu(), self.mask, self.doff,
                                 [K[r] for r in rows], [V[r] for r in rows], self.G,
                                 self.scale if scale is None else scale, softcap)

    def check(self, softcap=0.0, scale=None):
        torch.cuda.synchronize()
        assert tg.tg_tree_plan_status(self.plan) == tg.TG_OK
        out, lse, to, tl = self.reference(softcap, scale)
        n = int(self.doff[-1])
        o, l = self.out.double().cpu(), self.lse.double().cpu()
        empty = torch.isinf(lse[:n])
        assert torch.equal(torch.isinf(l[:n]), empty) and bool((o[:n][empty] == 0).all())
        far_o = ((o[:n] - out[:n]).abs() / to[:n])[~empty]
        far_l = ((l[:n] - lse[:n]).abs() / tl[:n])[~empty]
        assert not far_o.numel() or (float(far_o.max()) <= 1 and float(far_l.max()) <= 1), \
            (float(far_o.max()), float(far_l.max()))
        assert bool((o[n:] == 7).all()) and bool((l[n:] == 7).all())   # rows behind the last sequence


LENGTHS = [0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 300]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("T", [1, 5, 16, 33, 64])
def test_shapes(D, G, T):
    """Every head layout with one row to 512 rows (one tile, two tiles, several row blocks)."""
    rng = np.random.default_rng(100 * D + 10 * G + T)
    lens = rng.choice(LENGTHS, size=6)
    nd = [T, int(rng.integers(0, T + 1)), max(1, T // 2)]
    bt = Batch(D + G + T, G, D, 2, lens, nd, max_draft=T)
    bt.run()
    bt.check()


@pytest.mark.parametrize("G,T", [(1, 1), (1, 3), (1, 16), (2, 8), (2, 5), (4, 1), (4, 3), (4, 4), (8, 1), (8, 2)])
def test_shapes_of_few_rows(G, T):
    """The same for the kernel of few rows: lengths of none to several blocks beside a
    long one, ragged drafts."""
    rng = np.random.default_rng(10 * G + T)
    bt = Batch(G + T, G, 128, 2, rng.choice(LENGTHS, size=8), [T, 0, max(1, T // 2), int(rng.integers(0, T + 1))], max_draft=T,
               few=True)
    bt.run()
    bt.check()


@pytest.mark.parametrize("workers", [1, 3, 0])
@pytest.mark.parametrize("few", [False, True])
def test_lengths_and_splits(workers, few):
    """Lengths around page and block ends, whole and split heads (merged in order)."""
    lens = LENGTHS + [700, 1023]
    bt = Batch(5, 4, 128, 2, lens, [3, 0, 4, 1, 2, 4 if few else 16, 2], workers=workers, few=few)
    bt.run()
    bt.check()


def test_split_heads_of_long_rows():
    bt = Batch(6, 4, 128, 1, [5000, 17], [6, 3], workers=40, q_scale=4.0)
    assert tg.tg_tree_plan_items(bt.plan)["n_merge"] >= 1
    bt.run()
    bt.check()


@pytest.mark.parametrize("G,T,D,few", [(G, T, D, False) for G, T in [(4, 4), (4, 8), (4, 16), (4, 40), (1, 3)] for D in (64, 128)]
                         + [(4, 4, 128, True), (1, 3, 128, True), (2, 7, 128, True)])
@pytest.mark.parametrize("rising", [True, False])
def test_scores_far_from_the_first(G, T, D, few, rising):
    """Scores that climb by hundreds over a head's tokens (every block moves the running base), or that
    fall from a first token far above the rest; drafted keys above all of them."""
    bt = Batch(23, G, D, 2, [700, 130, 64, 0], [T, max(1, T // 2)], q_scale=6.0, few=few)
    bt.q.copy_(bt.q.abs())
    for i, n in enumerate(bt.lens):
        rows = torch.from_numpy(sp.head_rows(bt.ids, bt.off, i, int(n))).cuda()
        t = torch.arange(int(n), device="cuda")
        size = 0.05 + 4.0 * (t / max(1, int(n) - 1) if rising else (t == 0))
        k = bt.dev["kp"].view(-1, D)
        k[rows] = (k[rows].float().abs() * size[:, None]).bfloat16()
    bt.k.copy_(bt.k.abs() * 5)
    bt.run()
    bt.check()


def test_two_tiles_split():
    bt = Batch(7, 4, 128, 1, [900], [64], workers=9)
    assert tg.tg_tree_plan_items(bt.plan)["n_merge"] == 1
    bt.run()
    bt.check()


@pytest.mark.parametrize("D,T,few", [(64, 5, False), (64, 40, False), (128, 5, False), (128, 40, False), (128, 3, True),
                                     (128, 4, True)])
def test_softcap(D, T, few):
    bt = Batch(8, 4, D, 2, [100, 33, 0, 17], [T, 3], max_draft=T, q_scale=12.0, few=few)
    bt.run(softcap=15.0)
    bt.check(softcap=15.0)


@pytest.mark.parametrize("scale", [0.0, -0.05, 0.5])
@pytest.mark.parametrize("few", [False, True])
def test_scales(scale, few):
    bt = Batch(9, 2, 128, 2, [50, 20, 129, 3], [5, 8], few=few)
    bt.run(scale=scale)
    bt.check(scale=scale)


@pytest.mark.parametrize("few", [False, True])
def test_stale_rows_and_foreign_drafts_do_not_leak(few):
    """NaN in every pool row that is not retained, in K and V; NaN behind the last sequence."""
    bt = Batch(10, 4, 128, 2, [1, 17, 63, 66, 0, 129], [3, 4, 1], stale=float("nan"), extra_rows=4, cap_extra=40, few=few)
    n = int(bt.doff[-1])
    for x in (bt.k, bt.v, bt.q):
        x[n:] = float("nan")
    bt.run()
    bt.check()


@pytest.mark.parametrize("D,G,T,few", [(128, 4, 9, False), (64, 1, 40, False), (128, 8, 33, False), (128, 1, 9, True),
                                       (128, 1, 13, True)])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_masked_drafted_values_do_not_leak(D, G, T, few, value):
    """A drafted token whose K and V hold NaN or an infinity: the tokens that do not attend to it are
    as without it; those that do hold what 64 bits give in V's places."""
    masks = [1 << j for j in range(T)]
    masks = [m | (2 if j in (3, T - 1) else 0) for j, m in enumerate(masks)]   # token 1's other readers
    bt = Batch(11, G, D, 1, [37], [T], masks=masks, few=few)
    bt.v[1, 0, 5] = value
    bt.v[1, 0, D - 1] = value
    bt.run()
    torch.cuda.synchronize()
    assert tg.tg_tree_plan_status(bt.plan) == tg.TG_OK
    out, lse, to, tl = bt.reference()
    o, l = bt.out.double().cpu(), bt.lse.double().cpu()
    fine = torch.isfinite(out)
    assert torch.equal(torch.isfinite(o), fine) and int((~fine).sum()) == 3 * G * 2
    assert torch.equal(torch.isnan(o), torch.isnan(out)) and torch.equal(o[torch.isinf(out)], out[torch.isinf(out)])
    to = torch.where(torch.isfinite(to), to, torch.zeros(()).double())
    assert bool(((o - out).abs()[fine] <= to[fine]).all()) and bool(((l - lse).abs() <= tl).all())
    # K as well: only its readers' rows may change
    clean = o.clone()
    bt.k[1] = value
    bt.run()
    torch.cuda.synchronize()
    o = bt.out.double().cpu()
    others = [t for t in range(T) if not masks[t] >> 1 & 1]
    assert torch.equal(o[others], clean[others])


@pytest.mark.parametrize("few", [False, True])
def test_rows_that_see_nothing(few):
    """No cache and an empty mask: out 0, lse -inf; mask bits past the draft are ignored."""
    bt = Batch(12, 4, 128, 2, [0, 20, 0, 0], [4, 3], masks=[0, 2, 0xF0, 3, 2**64 - 1, 0, 0xFFF8], few=few)
    bt.run()
    bt.check()
    assert bool(torch.isinf(bt.lse[0, :4]).all()) and bool(torch.isfinite(bt.lse[0, 4:]).all())


@pytest.mark.parametrize("T", [4, 20])
def test_growing_heads_use_one_plan(T):
    """Reserved pages that hold nothing yet are skipped, also as whole parts of a split head."""
    bt = Batch(13, 4, 128, 2, [40, 0, 3, 500], [2, T], cap_extra=1900, workers=60)
    assert bt.rows == (16 if T == 4 else 128)
    for n in ([40, 0, 3, 500], [0, 0, 0, 0], [41, 900, 17, 1400]):
        bt.lens = np.asarray(n, np.int64)
        bt.dev["n"].copy_(torch.tensor(n, dtype=torch.int32))
        bt.run()
        bt.check()


def test_no_drafts_and_no_sequences():
    bt = Batch(14, 4, 128, 2, [40, 7], [0], max_draft=4, extra_rows=3)
    bt.run()
    bt.check()
    shape = tg.make_shape(0, 4, 2, 128, 0)
    plan = tg.tg_tree_plan_create(shape, [], 4, [0, 0], [0, 0])
    z = torch.zeros(0, 4, 128, dtype=torch.bfloat16, device="cuda")
    i32, i64 = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int64, device="cuda")
    tg.tg_tree_decode(plan, i32, z, z[:, :2], z[:, :2], i64, z, z, i32, i64, i32, 1.0, 0.0, z,
                      torch.zeros(0, device="cuda"))


@pytest.mark.parametrize("D", [64, 128])
def test_no_pages_at_all(D):
    """Heads without any reserved token attend to the draft alone; there is no table then."""
    bt = Batch(15, 2, D, 2, [0, 0], [5])
    bt.dev["table"] = torch.zeros(0, dtype=torch.int32, device="cuda")
    bt.run()
    bt.check()


@pytest.mark.parametrize("softcap", [1e-9, 1e-3, 1e9])
@pytest.mark.parametrize("few", [False, True])
def test_extreme_caps(softcap, few):
    bt = Batch(24, 4, 128, 2, [100, 33, 0, 17], [4, 3], few=few)
    bt.run(softcap=softcap)
    bt.check(softcap=softcap)


def test_contiguous_inputs_give_the_same_bits():
    a, b = (Batch(16, 4, 128, 2, [100, 40, 3, 260], [7, 12], fused=f) for f in (True, False))
    a.run()
    b.run()
    torch.cuda.synchronize()
    assert torch.equal(a.out, b.out) and torch.equal(a.lse, b.lse)


def test_other_stream_and_graph_replay():
    """On a side stream, and captured once and replayed after inputs and lengths changed in place."""
    bt = Batch(17, 4, 128, 2, [300, 40, 3, 260], [7, 12], cap_extra=100, workers=24)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        bt.run()
    s.synchronize()
    bt.check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bt.run()
    bt.q.neg_()
    bt.lens = bt.lens + 65
    bt.dev["n"] += 65
    bt.out.fill_(7)
    bt.lse.fill_(7)
    g.replay()
    bt.check()


@pytest.mark.parametrize("few", [False, True])
def test_two_plans_on_two_streams(few):
    bts = [Batch(18 + i, 4, 128, 2, [900, 40, 3, 260], [4, 3], workers=30, few=few) for i in range(2)]
    torch.cuda.synchronize()
    ss = [torch.cuda.Stream() for _ in bts]
    for _ in range(5):
        for bt, s in zip(bts, ss):
            bt.run(stream=s)
    torch.cuda.synchronize()
    for bt in bts:
        bt.check()


@pytest.mark.parametrize("few", [False, True])
def test_repeats_are_bit_equal(few):
    """Dynamic items go to whichever worker comes first; the results do not depend on it."""
    rng = np.random.default_rng(1)
    bt = Batch(20, 4, 128, 2, rng.integers(0, 2000, size=40), [4, 2, 3, 1] * 5, workers=20, few=few)
    info = tg.tg_tree_plan_items(bt.plan)
    assert info["worker_off"][-1] < info["n_items"]
    bt.run()
    torch.cuda.synchronize()
    o, l = bt.out.clone(), bt.lse.clone()
    for _ in range(10):
        bt.run()
    torch.cuda.synchronize()
    assert torch.equal(o, bt.out) and torch.equal(l, bt.lse)


@pytest.mark.parametrize("few", [False, True])
def test_device_side_refusals(few):
    """A page outside the pool, a length above the reserved one, a row outside its table and a draft
    wider than the plan are reported and skipped; the other sequences are right."""
    def case(change):
        bt = Batch(21, 4, 128, 2, [100, 40, 3, 260], [3, 4], few=few)
        change(bt)
        bt.run()
        torch.cuda.synchronize()
        assert tg.tg_tree_plan_status(bt.plan) == tg.TG_EBADPAGE
        assert tg.tg_tree_plan_status(bt.plan) == tg.TG_OK   # read and cleared
        out, lse, to, tl = bt.reference()
        good = slice(0, 3)   # sequence 0's tokens; the change is in sequence 1
        assert bool(((bt.out.double().cpu() - out).abs()[good] <= to[good]).all())

    def bad_page(bt):
        bt.dev["table"][int(bt.off[3])] = bt.pool

    def negative_page(bt):
        bt.dev["table"][int(bt.off[3])] = -1

    def too_long(bt):
        bt.dev["n"][3] += 1

    def negative(bt):
        bt.dev["n"][2] = -1

    def bad_row(bt):
        bt.dev["off"][3] = bt.ids.size   # past the table

    def wide(bt):
        bt.dev["doff"][2:] += 1   # sequence 1 drafts one token more than the plan allows

    for change in (bad_page, negative_page, too_long, negative, bad_row, wide):
        case(change)


def test_argument_refusals():
    bt = Batch(22, 4, 128, 2, [100, 40], [7])
    d = bt.dev
    good = dict(plan=bt.plan, draft_off=d["doff"], q=bt.q, k_draft=bt.k, v_draft=bt.v, tree_mask=d["mask"],
                k_pages=d["kp"], v_pages=d["vp"], page_table=d["table"], head_page_off=d["off"], head_kv_len=d["n"],
                scale=1.0, softcap=0.0, out=bt.out, lse=bt.lse)
    for name, bad in (("q", bt.q.float()), ("q", bt.q.transpose(0, 1)), ("q", bt.q[:, :4]), ("k_draft", bt.k[:5]),
                      ("tree_mask", d["mask"].int()), ("draft_off", d["doff"][:1]), ("head_kv_len", d["n"].long()),
                      ("out", bt.out[:5]), ("lse", bt.lse.bfloat16()), ("k_pages", d["kp"][:1]), ("q", bt.q.cpu()),
                      ("head_page_off", d["off"].int()), ("out", bt.out.transpose(0, 1))):
        with pytest.raises(ValueError):
            tg.tg_tree_decode(**{**good, name: bad})
    for kw in (dict(softcap=-1.0), dict(softcap=float("nan")), dict(scale=float("nan")), dict(scale=float("inf")),
               dict(softcap=float("inf"))):
        with pytest.raises(tg.TGError) as e:
            tg.tg_tree_decode(**{**good, **kw})
        assert e.value.status == tg.TG_EINVAL
    odd = torch.zeros(7 * 48 * 128 + 8, dtype=torch.bfloat16, device="cuda")[1:1 + 7 * 8 * 128].view(7, 8, 128)
    with pytest.raises(tg.TGError):   # not 16-byte aligned
        tg.tg_tree_decode(**{**good, "q": odd})
    host = tg.tg_tree_plan_create(bt.shape, bt.cap, 7, [0, 0], [0, bt.ids.size], host_only=True)
    with pytest.raises(tg.TGError):
        tg.tg_tree_decode(**{**good, "plan": host})
