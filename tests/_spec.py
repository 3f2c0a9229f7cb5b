"""Plain 64-bit forms of the speculative-step operators and random ragged batches, for the tests."""
from __future__ import annotations

import math

import numpy as np
import torch

PAGE = 16
HALF = 2.0 ** -8          # a rounding to bf16 is off by at most this share of the value


def bf16(rng, *shape, scale=1.0):
    return torch.from_numpy(rng.standard_normal(shape) * scale).to(torch.bfloat16)


def tables(rng, counts, spare=3):
    """Pages of a shuffled pool for every head's row, rows end to end: (ids, offsets, pool pages)."""
    counts = np.asarray(counts, np.int64).reshape(-1)
    pool = int(counts.sum()) + spare
    ids = rng.permutation(pool)[:int(counts.sum())].astype(np.int32)
    off = np.zeros(counts.size, np.int64)
    off[1:] = np.cumsum(counts)[:-1]
    return ids, off, pool


def head_rows(ids, off, i, n):
    """Flat pool rows of head i's first n tokens."""
    t = np.arange(n)
    return ids[off[i] + t // PAGE].astype(np.int64) * PAGE + t % PAGE


def random_masks(rng, nd, forest=True):
    """Ancestor masks of random trees, one per sequence, laid end to end (numpy uint64)."""
    out = []
    for n in nd:
        bits = []
        for j in range(int(n)):
            p = int(rng.integers(-1 if forest else max(-1, j - 1), j)) if j else -1
            bits.append((bits[p] if p >= 0 else 0) | (1 << j))
        out += bits
    return np.array(out, dtype=np.uint64)


def tree_reference(q, k, v, mask, draft_off, k_rows, v_rows, G, scale, softcap):
    """out, lse, and the tolerances of both, in 64 bits. k_rows[i] / v_rows[i]: retained rows of head
    i = b * Hkv + h. A tolerance counts the roundings: P to bf16 (HALF of sum p |v|), the output to
    bf16 (HALF of |out|), and the scores' fp32 sums of D products (at most (D + 2) 2^-23 of the sum of
    their magnitudes, the tensor core may truncate), which move p by as much relatively."""
    N, Hq, D = q.shape
    Hkv = Hq // G
    out = torch.zeros(N, Hq, D, dtype=torch.float64)
    lse = torch.full((N, Hq), -math.inf, dtype=torch.float64)
    tol_o = torch.zeros(N, Hq, D, dtype=torch.float64)
    tol_l = torch.zeros(N, Hq, dtype=torch.float64)
    qd, kd, vd = q.double(), k.double(), v.double()
    for b in range(len(draft_off) - 1):
        lo, hi = int(draft_off[b]), int(draft_off[b + 1])
        for h in range(Hkv):
            K, V = k_rows[b * Hkv + h].double(), v_rows[b * Hkv + h].double()
            for t in range(lo, hi):
                see = [lo + j for j in range(hi - lo) if int(mask[t]) >> j & 1]
                Kt, Vt = torch.cat([K, kd[see, h]]), torch.cat([V, vd[see, h]])
                if Kt.shape[0] == 0:
                    continue
                for g in range(h * G, h * G + G):
                    s = Kt @ qd[t, g] * scale
                    mag = float((Kt.abs() @ qd[t, g].abs()).max()) * abs(scale)
                    ds = (D + 2) * 2.0 ** -23 * mag + 2.0 ** -22 * mag
                    if softcap > 0:
                        s = softcap * torch.tanh(s / softcap)
                        ds += 8 * 2.0 ** -24 * softcap
                    l = torch.logsumexp(s, 0)
                    p = torch.exp(s - l)
                    o = p @ Vt
                    A = p @ Vt.abs()
                    out[t, g], lse[t, g] = o, l
                    n = Kt.shape[0]
                    rel = 2 * ds + n * 2.0 ** -24 + 2.0 ** -20
                    tol_o[t, g] = (HALF + rel) * A + HALF * o.abs() + 1e-30
                    tol_l[t, g] = ds + n * 2.0 ** -24 + 2.0 ** -20 * (1 + l.abs())
    return out, lse, tol_o, tol_l


def rope_reference(x, w, eps, pos, inv, interleaved, rot_scale):
    """y and its tolerance: one rounding to bf16 and fp32 arithmetic on the pair."""
    y = x.double()
    if w is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * w.double()
    r = 2 * len(inv)
    out, mag = y.clone(), y.abs()
    if r:
        ang = pos.double()[:, None] * torch.as_tensor(inv)
        c, s = torch.cos(ang)[:, None] * rot_scale, torch.sin(ang)[:, None] * rot_scale
        i = slice(0, r, 2) if interleaved else slice(0, r // 2)
        j = slice(1, r, 2) if interleaved else slice(r // 2, r)
        a, b = y[..., i], y[..., j]
        out[..., i], out[..., j] = a * c - b * s, a * s + b * c
        both = (a.abs() + b.abs()) * abs(rot_scale)
        mag = mag.clone()
        mag[..., i], mag[..., j] = both, both
    return out, HALF * out.abs() + 2.0 ** -20 * mag + 1e-30


def path_reference(sink, draft_off, path, path_len, budget, kv_len, cursor, Hkv):
    """The sink + recent rule one token at a time: (kept {head: {slot: draft row}}, kv_len, cursor,
    slots [BH, P])."""
    BH, P = len(budget), path.shape[1]
    n, c = np.array(kv_len, np.int64), np.array(cursor, np.int64)
    slots = np.full((BH, P), -1, np.int64)
    kept = [dict() for _ in range(BH)]
    for i in range(BH):
        b = i // Hkv
        if budget[i] < 1:
            continue
        s = max(0, min(sink, budget[i] - 1))
        for t in range(int(path_len[b])):
            if n[i] < budget[i]:
                at = n[i]
                n[i] += 1
            else:
                at = s + c[i] % (budget[i] - s)
                c[i] = (at - s + 1) % (budget[i] - s)
            slots[i][slots[i] == at] = -1
            slots[i, t] = at
            kept[i][int(at)] = int(draft_off[b]) + int(path[b, t])
    return kept, n, c, slots
