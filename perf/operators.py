"""Measured cases of the speculative-step operators: query / key norm with rotary positions,
attention of a drafted token tree over the ragged paged cache, the append of the accepted path,
and the page copy and compaction beside them.

One case is one call. The plain forms are elementary torch operations in 32 bits (angles in 64);
with `own` set, run() makes the library's calls on the same state.
"""
import math

import numpy as np
import torch

own = False

PAGE = 16
MB = 1e6


# ------------------------------------------------------------------------------------------
# Cases
# ------------------------------------------------------------------------------------------

def listed():
    return [
        # One conversation verifying a small tree on a tiny MHA layer (8 heads of 64): the call's
        # latency is what counts.
        dict(name="tree tiny mha", op="tree", B=1, Hq=8, Hkv=8, D=64, T=7, lo=512, hi=700, r_lo=0.5, r_hi=0.9,
             softcap=0.0, shape=11),
        # A GQA layer's batch (64 sequences, 32/8 heads of 128, contexts of 2048 to 8192 at budgets of
        # 10 to 90 %) verifying trees of up to 16 tokens.
        dict(name="tree gqa", op="tree", B=64, Hq=32, Hkv=8, D=128, T=16, lo=2048, hi=8192, r_lo=0.1, r_hi=0.9,
             softcap=0.0, shape=12),
        # The multi-turn serving layer (256 sequences, contexts of 4096 to 32768 at 5 to 50 %), short drafts.
        dict(name="tree serving", op="tree", B=256, Hq=32, Hkv=8, D=128, T=5, lo=4096, hi=32768, r_lo=0.05, r_hi=0.5,
             softcap=0.0, shape=13),
        # Few long conversations with the widest trees (up to 64 drafted tokens) and capped scores.
        dict(name="tree wide capped", op="tree", B=13, Hq=32, Hkv=8, D=128, T=64, lo=8192, hi=32768, r_lo=0.3,
             r_hi=0.9, softcap=30.0, shape=14),
        # A verification step's projections: 64 sequences x 16 drafted tokens, whole head rotated by halves.
        dict(name="rope step", op="rope", N=1024, Hq=32, Hkv=8, D=128, rot=128, interleaved=False, far=32768),
        # A prompt's projections: an odd number of tokens at far positions, interleaved pairs of part of the head.
        dict(name="rope prompt", op="rope", N=32001, Hq=32, Hkv=8, D=128, rot=64, interleaved=True, far=1000000),
        # The accepted paths of the GQA layer's batch: up to 6 tokens a sequence.
        dict(name="path gqa", op="path", B=64, Hkv=8, D=128, T=16, P=6, lo=2048, hi=8192, r_lo=0.1, r_hi=0.9,
             sink=4, shape=12),
        # Long accepted chains on a large batch of MHA heads of 64.
        dict(name="path chain", op="path", B=256, Hkv=16, D=64, T=32, P=29, lo=200, hi=1500, r_lo=0.2, r_hi=0.9,
             sink=4, shape=15),
        # Forking: the tail pages of one sequence's 8 heads into 8 children (partial rows).
        dict(name="copy fork tails", op="copy", pages=20000, copies=64, D=128, bits=16, partial=True),
        # Copying a long INT8 tier (codes and scales) for a new reader that will write its own.
        dict(name="copy int8 tier", op="copy", pages=180000, copies=65537, D=128, bits=8, partial=False),
        # A prompt's rows compacted to their budgets: one sequence of 8 heads.
        dict(name="compact one prompt", op="compact", B=1, Hkv=8, D=128, lo=8001, hi=8001, r_lo=0.05, r_hi=0.5,
             shape=16),
        # A batch of prompts compacted to their budgets.
        dict(name="compact batch", op="compact", B=32, Hkv=8, D=128, lo=4096, hi=16384, r_lo=0.1, r_hi=0.9, shape=17),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "rope", "path", "copy", "compact"])
    shape = rng.randrange(1 << 20)
    if op == "rope":
        D = rng.choice([64, 96, 128, 256])
        inter = rng.random() < 0.5
        rot = rng.randrange(0, D + 1, 2) if inter else rng.randrange(0, D + 1, 16)
        Hq, Hkv = rng.choice([(6, 6), (40, 8), (20, 20), (7, 1)])
        N = min(_log(rng, 1, 32000), int(32001 * 40 * 128 / ((Hq + Hkv) * D)))
        return dict(op=op, N=N, Hq=Hq, Hkv=Hkv, D=D, rot=rot, interleaved=inter, far=_log(rng, 1000, 1000000))
    if op == "copy":
        bits = rng.choice([16, 8, 4])
        copies = _log(rng, 1, 16000)
        return dict(op=op, pages=2 * copies + rng.randrange(1, 5000), copies=copies, D=rng.choice([64, 128]),
                    bits=bits, partial=rng.random() < 0.5)
    hi = _log(rng, 40, 20000)
    lo = max(1, int(hi * rng.uniform(0.3, 1.0)))
    r_lo = rng.uniform(0.05, 0.5)
    r_hi = rng.uniform(r_lo, 1.0)
    Hq, Hkv, D = rng.choice([(8, 8, 64), (32, 8, 128), (32, 4, 128), (16, 16, 128), (16, 8, 64)])
    most = 1.0e9 if op == "tree" else 0.5e9   # bytes of K/V held at most
    B = min(_log(rng, 1, 200), max(1, int(most / (hi * (1 if op == "compact" else r_hi) * Hkv * D * 4))))
    base = dict(op=op, B=B, Hkv=Hkv, D=D, lo=lo, hi=hi, r_lo=r_lo, r_hi=r_hi, shape=shape)
    if op == "tree":
        T = _log(rng, 1, 64)
        return dict(base, Hq=Hq, T=T, softcap=rng.choice([0.0, 0.0, 20.0, 50.0]))
    if op == "path":
        T = _log(rng, 1, 64)
        return dict(base, T=T, P=rng.randint(1, T), sink=rng.choice([0, 4, 64]))
    return base


# ------------------------------------------------------------------------------------------
# Shapes: functions of the case alone, so that work() knows them
# ------------------------------------------------------------------------------------------

def _heads(c):
    """Context lengths [B] and retained budgets [B][Hkv] of the case's batch."""
    r = np.random.RandomState(c["shape"])
    L = r.randint(c["lo"], c["hi"] + 1, size=c["B"]).astype(np.int64)
    rank = r.permutation(c["Hkv"])
    ratio = c["r_lo"] + (c["r_hi"] - c["r_lo"]) * rank / max(1, c["Hkv"] - 1)
    ratio = np.clip(ratio[None, :] + r.uniform(-0.02, 0.02, size=(c["B"], c["Hkv"])), 0.001, 1.0)
    budget = np.maximum(1, np.minimum(L[:, None], np.round(ratio * L[:, None]))).astype(np.int64)
    return L, budget, r


def _tree_shape(c):
    """Budgets, lengths (every fifth head is still growing), drafted tokens of each sequence and
    the mask bits: token j of a sequence has a parent among its earlier tokens (or the cache) and
    attends to itself and to its ancestors."""
    _, budget, r = _heads(c)
    n = budget.copy()
    grow = n.reshape(-1)[::5]
    n.reshape(-1)[::5] = np.maximum(0, grow - r.randint(0, 3 * c["T"] + 1, size=grow.shape))
    nd = r.randint((c["T"] + 1) // 2, c["T"] + 1, size=c["B"]).astype(np.int64)
    bits = np.zeros((c["B"], c["T"]), dtype=np.uint64)
    for j in range(c["T"]):
        parent = r.randint(max(-1, j - 5), j, size=c["B"]) if j else np.full(c["B"], -1)
        up = np.where(parent >= 0, bits[np.arange(c["B"]), np.maximum(parent, 0)], np.uint64(0))
        bits[:, j] = up | np.uint64(1 << j)
    return budget, n, nd, bits


def _path_shape(c):
    _, budget, r = _heads(c)
    n = budget.copy()
    grow = n.reshape(-1)[::5]
    n.reshape(-1)[::5] = np.maximum(0, grow - r.randint(0, 2 * c["P"] + 1, size=grow.shape))
    nd = r.randint(c["P"], c["T"] + 1, size=c["B"]).astype(np.int64)
    plen = r.randint(0, c["P"] + 1, size=c["B"]).astype(np.int64)
    plen[0] = c["P"]
    # an accepted path: ascending drafted tokens
    path = np.stack([np.sort(r.permutation(int(m))[:c["P"]]) for m in nd])
    return budget, n, nd, plen, path


def _tables(counts, seed, spare):
    """Page ids of every head's row (a permutation of the pool), the flat table and its offsets."""
    need = int(counts.sum())
    pool = need + spare
    ids = np.random.RandomState(seed % (1 << 31)).permutation(pool)[:need].astype(np.int32)
    off = np.zeros(counts.size, dtype=np.int64)
    off[1:] = np.cumsum(counts.reshape(-1))[:-1]
    return ids, off, pool


def _cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _bf16(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.bfloat16)


# ------------------------------------------------------------------------------------------
# prepare
# ------------------------------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return {"tree": _prepare_tree, "rope": _prepare_rope, "path": _prepare_path, "copy": _prepare_copy,
            "compact": _prepare_compact}[case["op"]](case, seed, g)


def _prepare_tree(c, seed, g):
    budget, n, nd, bits = _tree_shape(c)
    B, Hq, Hkv, D = c["B"], c["Hq"], c["Hkv"], c["D"]
    counts = -(-budget // PAGE)
    ids, off, pool = _tables(counts, seed, max(1, int(counts.sum()) // 9))
    doff = np.zeros(B + 1, dtype=np.int32)
    doff[1:] = np.cumsum(nd)
    N = int(doff[-1])
    mask = np.concatenate([bits[b, :nd[b]] for b in range(B)]).view(np.int64)
    # q, k and v are slices of one fused projection, as a layer hands them over; keys and queries
    # carry a spread of scales so that some heads attend sharply
    qkv = _bf16(g, N, Hq + 2 * Hkv, D)
    st = dict(case=c, q=qkv[:, :Hq] * 1.5, k=qkv[:, Hq:Hq + Hkv], v=qkv[:, Hq + Hkv:], mask=_cuda(mask),
              draft_off=_cuda(doff), k_pages=_bf16(g, pool, PAGE, D), v_pages=_bf16(g, pool, PAGE, D),
              table=_cuda(ids), off=_cuda(off), kv_len=_cuda(n.reshape(-1).astype(np.int32)),
              scale=1.0 / math.sqrt(D), n_max=int(n.max()), nd=nd,
              out=torch.empty(N, Hq, D, dtype=torch.bfloat16, device="cuda"),
              lse=torch.empty(N, Hq, dtype=torch.float32, device="cuda"))
    if own:
        import non_uniform_paged_flash_b200 as tg
        shape = tg.make_shape(B, Hq, Hkv, D, pool)
        st["plan"] = tg.tg_tree_plan_create(shape, budget.reshape(-1), c["T"], np.zeros(Hkv, np.int32),
                                            np.array([0, ids.size], np.int64))
    return st


def _prepare_rope(c, seed, g):
    N, Hq, Hkv, D, rot = c["N"], c["Hq"], c["Hkv"], c["D"], c["rot"]
    qkv = _bf16(g, N, Hq + 2 * Hkv, D)
    start = torch.randint(0, c["far"], (1,), generator=g, device="cuda")
    pos = (start + torch.arange(N, device="cuda") % c["far"]).to(torch.int32)
    # base 10000, positions interpolated by 4 (a context four times the trained one)
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(1, rot)) / 4.0
    return dict(case=c, q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hkv], wq=1 + 0.1 * _bf16(g, D), wk=1 + 0.1 * _bf16(g, D),
                pos=pos, inv=inv.cuda(), eps=1e-6, rot_scale=1.0,
                q_out=torch.empty(N, Hq, D, dtype=torch.bfloat16, device="cuda"),
                k_out=torch.empty(N, Hkv, D, dtype=torch.bfloat16, device="cuda"))


def _prepare_path(c, seed, g):
    budget, n, nd, plen, path = _path_shape(c)
    B, Hkv, D = c["B"], c["Hkv"], c["D"]
    counts = -(-budget // PAGE)
    ids, off, pool = _tables(counts, seed, max(1, int(counts.sum()) // 9))
    doff = np.zeros(B + 1, dtype=np.int32)
    doff[1:] = np.cumsum(nd)
    N = int(doff[-1])
    ring = np.maximum(1, budget - np.minimum(c["sink"], budget - 1))
    cursor = np.where(n == budget, np.random.RandomState(seed % (1 << 31)).randint(0, 1 << 20, n.shape) % ring, 0)
    kv = _bf16(g, N, 2 * Hkv, D)
    BH = B * Hkv
    return dict(case=c, k=kv[:, :Hkv], v=kv[:, Hkv:], draft_off=_cuda(doff), path=_cuda(path.astype(np.int32)),
                path_len=_cuda(plen.astype(np.int32)), k_pages=_bf16(g, pool, PAGE, D),
                v_pages=_bf16(g, pool, PAGE, D), table=_cuda(ids), off=_cuda(off),
                budget=_cuda(budget.reshape(-1).astype(np.int32)), kv_len=_cuda(n.reshape(-1).astype(np.int32)),
                cursor=_cuda(cursor.reshape(-1).astype(np.int32)),
                kv_len_out=torch.empty(BH, dtype=torch.int32, device="cuda"),
                cursor_out=torch.empty(BH, dtype=torch.int32, device="cuda"),
                slot_out=torch.empty(BH, c["P"], dtype=torch.int32, device="cuda"))


def _prepare_copy(c, seed, g):
    perm = torch.randperm(c["pages"], generator=g, device="cuda").to(torch.int32)
    m = c["copies"]
    # children share sources (a fork copies one tail page to each); targets are fresh pages
    pick = torch.randint(0, max(1, c["pages"] - m), (m,), generator=g, device="cuda")
    st = dict(case=c, src=perm[m:][pick].contiguous(), dst=perm[:m].contiguous(), rows=None, ks=None, vs=None,
              n_bad=torch.zeros(1, dtype=torch.int32, device="cuda"))
    if c["partial"]:
        st["rows"] = torch.randint(1, PAGE + 1, (m,), generator=g, device="cuda").to(torch.int32)
    if c["bits"] == 16:
        st["k"], st["v"] = _bf16(g, c["pages"], PAGE, c["D"]), _bf16(g, c["pages"], PAGE, c["D"])
        return st
    width, dt, lo, hi = (c["D"], torch.int8, -127, 128) if c["bits"] == 8 else (c["D"] // 2, torch.uint8, 0, 256)
    for name in ("k", "v"):
        st[name] = torch.randint(lo, hi, (c["pages"], PAGE, width), generator=g, device="cuda", dtype=dt)
        st[name + "s"] = torch.rand(c["pages"], PAGE, generator=g, device="cuda") * 0.02 + 0.005
    return st


def _prepare_compact(c, seed, g):
    L, budget, _ = _heads(c)
    B, Hkv, D = c["B"], c["Hkv"], c["D"]
    r = np.random.RandomState(seed % (1 << 31))
    full = np.repeat(L[:, None], Hkv, axis=1)
    src_ids, src_off, src_pool = _tables(-(-full // PAGE), seed, 3)
    ids, off, pool = _tables(-(-budget // PAGE), seed + 1, max(1, int(budget.sum()) // 150))
    keep_off = np.zeros(B * Hkv + 1, dtype=np.int64)
    keep_off[1:] = np.cumsum(budget.reshape(-1))
    # the rows a compression rule kept: the first 4, the last ones, and a random rest, ascending
    keep = np.concatenate([np.sort(r.permutation(int(l))[:int(m)])
                           for l, m in zip(full.reshape(-1), budget.reshape(-1))]).astype(np.int32)
    return dict(case=c, k_src=_bf16(g, src_pool, PAGE, D), v_src=_bf16(g, src_pool, PAGE, D),
                src_table=_cuda(src_ids), src_off=_cuda(src_off),
                src_len=_cuda(full.reshape(-1).astype(np.int32)), keep_off=_cuda(keep_off), keep=_cuda(keep),
                k_pages=_bf16(g, pool, PAGE, D), v_pages=_bf16(g, pool, PAGE, D), table=_cuda(ids), off=_cuda(off),
                budget=_cuda(budget.reshape(-1).astype(np.int32)),
                kv_len=torch.empty(B * Hkv, dtype=torch.int32, device="cuda"),
                n_bad=torch.zeros(1, dtype=torch.int32, device="cuda"))


# ------------------------------------------------------------------------------------------
# run
# ------------------------------------------------------------------------------------------

def run(state):
    if own:
        return _OWN[state["case"]["op"]](state)
    return _PLAIN[state["case"]["op"]](state)


def _own_tree(s):
    import non_uniform_paged_flash_b200 as tg
    tg.tg_tree_decode(s["plan"], s["draft_off"], s["q"], s["k"], s["v"], s["mask"], s["k_pages"], s["v_pages"],
                      s["table"], s["off"], s["kv_len"], s["scale"], s["case"]["softcap"], s["out"], s["lse"])
    return s["out"], s["lse"]


def _own_rope(s):
    import non_uniform_paged_flash_b200 as tg
    tg.tg_qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], s["eps"], s["pos"], s["inv"], s["q_out"], s["k_out"],
                       interleaved=s["case"]["interleaved"], rot_scale=s["rot_scale"])
    return s["q_out"], s["k_out"]


def _own_path(s):
    import non_uniform_paged_flash_b200 as tg
    c = s["case"]
    shape = tg.make_shape(c["B"], c["Hkv"], c["Hkv"], c["D"], s["k_pages"].shape[0])
    tg.tg_append_path_sink_recent(shape, c["sink"], s["draft_off"], s["path"], s["path_len"], s["k"], s["v"],
                                  s["k_pages"], s["v_pages"], s["table"], s["off"], s["budget"], s["kv_len"],
                                  s["cursor"], s["kv_len_out"], s["cursor_out"], s["slot_out"])
    return s["k_pages"], s["v_pages"], s["kv_len_out"], s["cursor_out"], s["slot_out"]


def _own_copy(s):
    import non_uniform_paged_flash_b200 as tg
    tg.tg_copy_pages(s["src"], s["dst"], s["rows"], s["k"], s["v"], s["n_bad"], k_scale=s["ks"], v_scale=s["vs"])
    return _copy_outputs(s)


def _own_compact(s):
    import non_uniform_paged_flash_b200 as tg
    c = s["case"]
    shape = tg.make_shape(c["B"], c["Hkv"], c["Hkv"], c["D"], s["k_pages"].shape[0])
    tg.tg_compact_kv(shape, s["k_src"], s["v_src"], s["src_table"], s["src_off"], s["src_len"], s["keep_off"],
                     s["keep"], s["k_pages"], s["v_pages"], s["table"], s["off"], s["budget"], s["kv_len"],
                     s["n_bad"])
    return s["k_pages"], s["v_pages"], s["kv_len"], s["n_bad"]


def _copy_outputs(s):
    # codes are whole numbers, each with its row's scale beside it
    return [t for t in (s["k"], s["v"], s["ks"], s["vs"], s["n_bad"]) if t is not None]


def _attention(s, dt):
    """Rows padded to the longest head and to the widest draft, in the type dt."""
    c = s["case"]
    B, Hq, Hkv, D, T = c["B"], c["Hq"], c["Hkv"], c["D"], c["T"]
    G = Hq // Hkv
    t = torch.arange(s["n_max"], device="cuda")
    held = t < s["kv_len"].long()[:, None]                                       # [BH, n]
    page = s["table"].long()[torch.where(held, s["off"][:, None] + t // PAGE, 0)]
    row = torch.where(held, page * PAGE + t % PAGE, 0)
    K = s["k_pages"].view(-1, D)[row].to(dt).view(B, Hkv, -1, D)
    V = s["v_pages"].view(-1, D)[row].to(dt).view(B, Hkv, -1, D)
    held = held.view(B, Hkv, 1, -1)
    j = torch.arange(T, device="cuda")
    first = s["draft_off"].long()[:-1, None]
    drafted = j < (s["draft_off"].long()[1:, None] - first)                      # [B, T]
    tok = torch.where(drafted, first + j, 0)
    q = s["q"][tok].to(dt).view(B, T, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, T * G, D)
    kd = s["k"][tok].to(dt).permute(0, 2, 1, 3)
    vd = s["v"][tok].to(dt).permute(0, 2, 1, 3)
    sees = ((s["mask"][tok][:, :, None] >> j) & 1).bool() & drafted[:, None, :]     # [B, T, T]
    sees = sees.repeat_interleave(G, dim=1)[:, None]
    sc = torch.cat([q @ K.transpose(2, 3), q @ kd.transpose(2, 3)], dim=3) * s["scale"]
    del K, kd
    if c["softcap"] > 0:
        sc = c["softcap"] * torch.tanh(sc / c["softcap"])
    n = s["n_max"]
    sc[..., :n].masked_fill_(~held, -math.inf)
    sc[..., n:].masked_fill_(~sees, -math.inf)
    top = sc.amax(dim=3, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    sc = sc.sub_(top).exp_()
    tot = sc.sum(dim=3, keepdim=True)
    o = (sc[..., :n] @ V + sc[..., n:] @ vd) / torch.where(tot > 0, tot, torch.ones_like(tot))
    lse = (torch.log(tot) + top).squeeze(3)
    o = o.view(B, Hkv, T, G, D).permute(0, 2, 1, 3, 4).reshape(B, T, Hq, D)
    lse = lse.view(B, Hkv, T, G).permute(0, 2, 1, 3).reshape(B, T, Hq)
    return o[drafted], lse[drafted]


def _plain_tree(s):
    o, lse = _attention(s, torch.float32)
    return o.to(torch.bfloat16), lse


def _turned(x, w, s, dt):
    """One side of the norm and rotation, in the type dt (angles in 64 bits)."""
    c = s["case"]
    x = x.to(dt)
    x = x * torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + s["eps"]) * w.to(dt)
    r = c["rot"]
    ang = s["pos"].double()[:, None] * s["inv"]
    cos, sin = (ang.cos() * s["rot_scale"]).to(dt)[:, None], (ang.sin() * s["rot_scale"]).to(dt)[:, None]
    if c["interleaved"]:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], dim=-1).flatten(-2)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], dim=-1)
    return torch.cat([turned, x[..., r:]], dim=-1)


def _plain_rope(s):
    return tuple(_turned(s[x], s["w" + x], s, torch.float32).to(torch.bfloat16) for x in ("q", "k"))


def _path_slots(s):
    """Slot of every accepted token under the sink + recent rule, -1 for those past the path and
    those that a later token of the same path replaces; new lengths and cursors."""
    c = s["case"]
    P = c["P"]
    bud, n, cur = s["budget"].long(), s["kv_len"].long(), s["cursor"].long()
    m = s["path_len"].long().repeat_interleave(c["Hkv"])
    keep = torch.minimum(torch.full_like(bud, c["sink"]), bud - 1).clamp(min=0)
    ring = bud - keep
    i = torch.arange(P, device="cuda")
    at = n[:, None] + i
    over = at - bud[:, None]
    slot = torch.where(over < 0, at, keep[:, None] + (cur[:, None] + over) % ring[:, None])
    slot = torch.where(i < m[:, None], slot, -1)
    later = ((slot[:, :, None] == slot[:, None, :]) & (i[None, :] > i[:, None])).any(dim=2)
    slot = torch.where(later, -1, slot)
    n_new = torch.minimum(bud, n + m)
    cur_new = torch.where(n + m > bud, (cur + n + m - bud) % ring, cur)
    return slot, n_new.int(), cur_new.int()


def _plain_path(s):
    c = s["case"]
    slot, n_new, cur_new = _path_slots(s)
    bh, i = (slot >= 0).nonzero(as_tuple=True)
    at = slot[bh, i]
    page, row = s["table"].long()[s["off"][bh] + at // PAGE], at % PAGE
    b, h = bh // c["Hkv"], bh % c["Hkv"]
    tok = s["draft_off"].long()[b] + s["path"].long()[b, i]
    s["k_pages"][page, row] = s["k"][tok, h]
    s["v_pages"][page, row] = s["v"][tok, h]
    return s["k_pages"], s["v_pages"], n_new, cur_new, slot.int()


def _plain_copy(s):
    src, dst = s["src"].long(), s["dst"].long()
    for t in (s["k"], s["v"], s["ks"], s["vs"]):
        if t is None:
            continue
        if s["rows"] is None:
            t[dst] = t[src]
        else:
            i, r = (torch.arange(PAGE, device="cuda") < s["rows"][:, None]).nonzero(as_tuple=True)
            t[dst[i], r] = t[src[i], r]
    return _copy_outputs(s)


def _compact_rows(s):
    n = s["keep_off"][1:] - s["keep_off"][:-1]
    i = torch.arange(s["keep"].numel(), device="cuda")
    bh = torch.repeat_interleave(n, output_size=s["keep"].numel())
    to = i - s["keep_off"][bh]
    frm = s["keep"].long()
    src = s["src_table"].long()[s["src_off"][bh] + frm // PAGE] * PAGE + frm % PAGE
    dst = s["table"].long()[s["off"][bh] + to // PAGE] * PAGE + to % PAGE
    return n, src, dst


def _plain_compact(s):
    D = s["case"]["D"]
    n, src, dst = _compact_rows(s)
    s["k_pages"].view(-1, D)[dst] = s["k_src"].view(-1, D)[src]
    s["v_pages"].view(-1, D)[dst] = s["v_src"].view(-1, D)[src]
    return s["k_pages"], s["v_pages"], n.int(), s["n_bad"]


_PLAIN = dict(tree=_plain_tree, rope=_plain_rope, path=_plain_path, copy=_plain_copy, compact=_plain_compact)
_OWN = dict(tree=_own_tree, rope=_own_rope, path=_own_path, copy=_own_copy, compact=_own_compact)


# ------------------------------------------------------------------------------------------
# work and exact
# ------------------------------------------------------------------------------------------

def work(case):
    c = case
    if c["op"] == "tree":
        _, n, nd, bits = _tree_shape(c)
        G, D, N = c["Hq"] // c["Hkv"], c["D"], int(nd.sum())
        held = int(n.sum())
        seen = sum(bin(int(x)).count("1") for b in range(c["B"]) for x in bits[b, :nd[b]])
        pairs = int((n.sum(axis=1) * nd).sum()) * G + seen * c["Hq"]
        return {"bytes": held * D * 4 + N * (c["Hq"] * (4 * D + 4) + c["Hkv"] * 4 * D + 8)
                + int((-(-n // PAGE)).sum()) * 4 + n.size * 12 + 4 * (c["B"] + 1),
                "flops": 4 * D * pairs}
    if c["op"] == "rope":
        heads = c["N"] * (c["Hq"] + c["Hkv"])
        return {"bytes": heads * c["D"] * 4 + c["N"] * 4 + c["rot"] * 4 + 4 * c["D"],
                "flops": heads * (4 * c["D"] + 3 * c["rot"])}
    if c["op"] == "path":
        _, n, _, plen, _ = _path_shape(c)
        return {"bytes": int(plen.sum()) * c["Hkv"] * c["D"] * 8 + n.size * (20 + 8 + 4 * c["P"]) + 8 * c["B"],
                "flops": 0}
    if c["op"] == "copy":
        row = {16: 2 * c["D"], 8: c["D"] + 4, 4: c["D"] // 2 + 4}[c["bits"]]
        rows = c["copies"] * (8.5 if c["partial"] else PAGE)
        return {"bytes": int(rows * row * 4 + c["copies"] * (12 if c["partial"] else 8)), "flops": 0}
    _, budget, _ = _heads(c)
    return {"bytes": int(budget.sum()) * (c["D"] * 8 + 4) + budget.size * 40, "flops": 0}


def exact(case, seed):
    """From the definitions in 64 bits, row by row of the batch, apart from the plain forms."""
    s = prepare(case, seed)
    c = case
    if c["op"] == "tree":
        return _exact_tree(s)
    if c["op"] == "rope":
        return tuple(_exact_rope(s, s[x], s["w" + x]) for x in ("q", "k"))
    if c["op"] == "path":
        return _exact_path(s)
    if c["op"] == "copy":
        old = [None if s[n] is None else s[n].clone() for n in ("k", "v", "ks", "vs")]
        rows = torch.full_like(s["src"], PAGE) if s["rows"] is None else s["rows"]
        r = torch.arange(PAGE, device="cuda").repeat(c["copies"])
        i = torch.arange(c["copies"], device="cuda").repeat_interleave(PAGE)
        i, r = i[r < rows[i]], r[r < rows[i]]
        outs = []
        for o in old:
            if o is not None:
                new = o.clone()
                new[s["dst"].long()[i], r] = o[s["src"].long()[i], r]
                outs.append(new.double() if new.is_floating_point() else new)
        return outs + [s["n_bad"]]
    return _exact_compact(s)


def _exact_tree(s):
    c = s["case"]
    G, D = c["Hq"] // c["Hkv"], c["D"]
    off, n = s["off"].cpu().numpy(), s["kv_len"].cpu().numpy()
    doff = s["draft_off"].cpu().numpy()
    if int(n.sum()) > 20_000_000 or n.size > 6000:
        return None
    N = int(doff[-1])
    out = torch.zeros(N, c["Hq"], D, dtype=torch.float64, device="cuda")
    lse = torch.zeros(N, c["Hq"], dtype=torch.float64, device="cuda")
    slot = torch.arange(PAGE, device="cuda")
    for b in range(c["B"]):
        lo, hi = int(doff[b]), int(doff[b + 1])
        m = hi - lo
        see = ((s["mask"][lo:hi, None] >> torch.arange(m, device="cuda")) & 1) > 0
        for h in range(c["Hkv"]):
            i = b * c["Hkv"] + h
            ids = s["table"][int(off[i]):int(off[i]) + -(-int(n[i]) // PAGE)].long()
            rows = (ids[:, None] * PAGE + slot).reshape(-1)[:int(n[i])]
            K = torch.cat([s["k_pages"].view(-1, D)[rows], s["k"][lo:hi, h]]).double()
            V = torch.cat([s["v_pages"].view(-1, D)[rows], s["v"][lo:hi, h]]).double()
            Q = s["q"][lo:hi, h * G:(h + 1) * G].double()                   # [m, G, D]
            x = torch.einsum("tgd,nd->tgn", Q, K) * s["scale"]
            if c["softcap"] > 0:
                x = c["softcap"] * torch.tanh(x / c["softcap"])
            ok = torch.cat([torch.ones(m, rows.numel(), dtype=torch.bool, device="cuda"), see], dim=1)
            x = x.masked_fill(~ok[:, None], -math.inf)
            l = torch.logsumexp(x, dim=2)
            lse[lo:hi, h * G:(h + 1) * G] = l
            out[lo:hi, h * G:(h + 1) * G] = torch.einsum("tgn,nd->tgd", torch.exp(x - l[..., None]), V)
    return out, lse


def _exact_rope(s, x, w):
    c = s["case"]
    x, r = x.double(), c["rot"]
    y = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / c["D"] + s["eps"]) * w.double()
    z = torch.view_as_complex(torch.stack([y[..., 0:r:2], y[..., 1:r:2]] if c["interleaved"]
                                          else [y[..., :r // 2], y[..., r // 2:r]], dim=-1).contiguous())
    z = z * torch.polar(torch.full((), s["rot_scale"], dtype=torch.float64, device="cuda"),
                        torch.outer(s["pos"].double(), s["inv"]))[:, None]
    if c["interleaved"]:
        y[..., 0:r:2], y[..., 1:r:2] = z.real, z.imag
    else:
        y[..., :r // 2], y[..., r // 2:r] = z.real, z.imag
    return y


def _exact_path(s):
    """The rule one token at a time."""
    c = s["case"]
    bud, n, cur = (s[k].cpu().numpy().astype(np.int64).copy() for k in ("budget", "kv_len", "cursor"))
    plen, path, doff = (s[k].cpu().numpy() for k in ("path_len", "path", "draft_off"))
    heads = np.arange(n.size)
    b = heads // c["Hkv"]
    slots = np.full((n.size, c["P"]), -1, dtype=np.int64)
    keep = np.maximum(0, np.minimum(c["sink"], bud - 1))
    for i in range(c["P"]):
        on = i < plen[b]
        free = n < bud
        at = np.where(free, n, keep + cur % (bud - keep))
        slots[:, :i][(slots[:, :i] == at[:, None]) & on[:, None]] = -1
        slots[:, i] = np.where(on, at, -1)
        cur = np.where(on & ~free, (cur + 1) % (bud - keep), cur)
        n = np.where(on & free, n + 1, n)
    table, off = s["table"].cpu().numpy(), s["off"].cpu().numpy()
    hh, ii = np.nonzero(slots >= 0)
    at = slots[hh, ii]
    flat = torch.from_numpy(table[off[hh] + at // PAGE].astype(np.int64) * PAGE + at % PAGE).cuda()
    tok = torch.from_numpy(doff[b[hh]].astype(np.int64) + path[b[hh], ii]).cuda()
    outs = []
    for pool, new in ((s["k_pages"], s["k"]), (s["v_pages"], s["v"])):
        p = pool.double().view(-1, c["D"])
        p[flat] = new[tok, torch.from_numpy(hh % c["Hkv"]).cuda()].double()
        outs.append(p.view(pool.shape))
    return (*outs, _cuda(n.astype(np.int32)), _cuda(cur.astype(np.int32)), _cuda(slots.astype(np.int32)))


def _exact_compact(s):
    D = s["case"]["D"]
    off, ko = s["off"].cpu().numpy(), s["keep_off"].cpu().numpy()
    so, keep = s["src_off"].cpu().numpy(), s["keep"].cpu().numpy().astype(np.int64)
    st, tb = s["src_table"].cpu().numpy(), s["table"].cpu().numpy()
    src, dst = np.empty(keep.size, np.int64), np.empty(keep.size, np.int64)
    for i in range(off.size):
        a, b = int(ko[i]), int(ko[i + 1])
        to = np.arange(b - a)
        src[a:b] = st[so[i] + keep[a:b] // PAGE].astype(np.int64) * PAGE + keep[a:b] % PAGE
        dst[a:b] = tb[off[i] + to // PAGE].astype(np.int64) * PAGE + to % PAGE
    outs = []
    for pool, frm in ((s["k_pages"], s["k_src"]), (s["v_pages"], s["v_src"])):
        p = pool.double().view(-1, D)
        p[torch.from_numpy(dst).cuda()] = frm.view(-1, D)[torch.from_numpy(src).cuda()].double()
        outs.append(p.view(pool.shape))
    return (*outs, _cuda(np.diff(ko).astype(np.int32)), s["n_bad"])
