"""Plain float64 definitions of the paged-cache operators and the token log probabilities.

Like tp_oracle.py this is test infrastructure: numpy only, loops where a loop is the definition, no
code shared with the kernels.
"""
import math

import numpy as np


def tables(lens, add, free, head, table, page, max_pages, n_pages, rows):
    """Requests one after another.  Returns (table, lens_out, cu_rows, positions, slots, counts)."""
    table = table.copy()
    lens_out, cu = np.array(lens, dtype=np.int64), [0]
    pos, slots = np.zeros(rows, np.int64), np.full(rows, -1, np.int64)
    left = len(free) - head if 0 <= head <= len(free) else 0
    need_sum = taken = refused = 0
    for m, (n, a) in enumerate(zip(lens, add)):
        first, count = cu[-1], max(a, 0)
        cu.append(first + count)
        ok = n >= 0 and a >= 0 and n + a <= max_pages * page and first + count <= rows
        held = -(-n // page)
        need = -(-(n + a) // page) - held if ok else 0
        got = ok and (need == 0 or need_sum + need <= left)
        if got:
            for j in range(need):
                table[m, held + j] = free[head + need_sum + j]
            lens_out[m] = n + a
            taken += need
        else:
            refused += 1
        need_sum += need
        for i in range(count):
            if first + i >= rows:
                break
            pos[first + i] = (n + i + 2 ** 31) % 2 ** 32 - 2 ** 31  # an int32: wraps for a refused length near 2^31
            if got:
                p = table[m, (n + i) // page]
                if 0 <= p < n_pages:
                    slots[first + i] = p * page + (n + i) % page
    return table, lens_out, np.array(cu), pos, slots, np.array([head + taken, cu[-1], refused])


def rope_freqs(rot, theta, scaling="none", factor=1.0, original_len=0, low=1.0, high=4.0, beta_fast=32.0,
               beta_slow=1.0):
    """Radians per position of each pair, and the factor on cos and sin."""
    f = np.array([theta ** (-2.0 * i / rot) for i in range(rot // 2)])
    if scaling == "none":
        return f, 1.0
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "wavelength":
        keep = np.clip((original_len * f / (2 * math.pi) - low) / (high - low), 0, 1)
        return keep * f + (1 - keep) * f / factor, 1.0

    def dim(r):
        return rot * math.log(original_len / (2 * math.pi * r)) / (2 * math.log(theta))
    lo, hi = max(0, math.floor(dim(beta_fast))), min(rot - 1, math.ceil(dim(beta_slow)))
    keep = 1 - np.clip((np.arange(rot // 2) - lo) / max(hi - lo, 1e-3), 0, 1)
    return keep * f + (1 - keep) * f / factor, (0.1 * math.log(factor) + 1 if factor > 1 else 1.0)


def rope(x, pos, freqs, mscale, layout):
    """x [M, heads, hd] turned at pos [M]."""
    y, r = np.array(x, dtype=np.float64), len(freqs)
    ang = np.asarray(pos, np.float64)[:, None] * freqs
    c, s = np.cos(ang) * mscale, np.sin(ang) * mscale
    for i in range(r):
        a, b = (i, i + r) if layout == "half" else (2 * i, 2 * i + 1)
        y[:, :, a] = x[:, :, a] * c[:, i, None] - x[:, :, b] * s[:, i, None]
        y[:, :, b] = x[:, :, b] * c[:, i, None] + x[:, :, a] * s[:, i, None]
    return y


def split_qkv(qkv, t, n_q, n_kv, hd):
    """Shard-major qkv [M, (n_q + 2 n_kv) hd] -> q [M, n_q, hd], k, v [M, n_kv, hd]."""
    x = np.asarray(qkv).reshape(len(qkv), t, (n_q + 2 * n_kv) // t, hd)
    a, b = n_q // t, (n_q + n_kv) // t
    return tuple(y.reshape(len(qkv), -1, hd) for y in (x[:, :, :a], x[:, :, a:b], x[:, :, b:]))


def attention(q, kf, vf, scale, window=0):
    """One request: q [n_q, hd]; kf(g), vf(g): the rows [n, hd] of kv head g, and a truth value for each row
    of whether it counts.  Returns o, lse, and for the error bounds A = sum p |v| and the largest sum |q||k|."""
    n_q, hd = q.shape
    k0, count = kf(0)
    n = len(k0)
    n_kv = kf.n_kv
    o, lse = np.zeros((n_q, hd)), np.full(n_q, -np.inf)
    A, B = np.zeros((n_q, hd)), np.zeros(n_q)
    seen = np.array(count, bool)
    if window:
        seen[: max(0, n - window)] = False
    for h in range(n_q):
        g = h // (n_q // n_kv)
        k, v = kf(g)[0][seen], vf(g)[0][seen]
        if not len(k):
            continue
        s = scale * (k @ q[h])
        top = s.max()
        e = np.exp(s - top)
        lse[h] = top + math.log(e.sum())
        p = e / e.sum()
        o[h], A[h] = p @ v, p @ np.abs(v)
        B[h] = abs(scale) * (np.abs(k) @ np.abs(q[h])).max()
    return o, lse, A, B


def logprobs(x, ids, k):
    """x [M, V] float64.  Returns logprob, rank, entropy, top_logprob, top_id as the header defines them."""
    M, V = x.shape
    lp, rank, ent = np.zeros(M), np.zeros(M, np.int64), np.zeros(M)
    tl, ti = np.zeros((M, k)), np.zeros((M, k), np.int64)
    for m in range(M):
        asked = 0 <= ids[m] < V
        if np.isnan(x[m]).any() or (x[m] == np.inf).any() or (x[m] == -np.inf).all():
            lp[m], rank[m], ent[m] = (np.nan if asked else 0.0), 0, np.nan
            tl[m], ti[m] = np.nan, -1
            continue
        top = x[m].max()
        y = (x[m] - top) - math.log(np.exp(x[m] - top).sum())  # in this order: top may be the type's largest
        p = np.exp(y)
        ent[m] = -np.sum(p[p > 0] * y[p > 0])
        order = np.lexsort((np.arange(V), -x[m]))
        if asked:
            lp[m], rank[m] = y[ids[m]], int(np.nonzero(order == ids[m])[0][0]) + 1
        ti[m], tl[m] = order[:k], y[order[:k]]
    return lp, rank, ent, tl, ti
