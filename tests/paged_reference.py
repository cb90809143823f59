"""The paged-cache operators in 64 bits on the CPU, with the bounds their
results are held to.  Plain numpy, nothing shared with the kernels.

Bounds (u = 2^-24, half a step of fp32; a product sum of n terms in any order
is off by at most n u sum |terms|):
  score    s = scale q.k in log2 units: es = (hd + 4) u scale sum |q k| + 4 u max |s|
           (the sum; scale, its product with log2 e, the difference from the
           maximum and its rounding)
  weight   w = 2^s: relative expm1(es) + 2^-21 (the exponential's own error)
  result   sum_j p_j v_j with p = w / sum w: the weights' errors enter once
           above and once below the line, L + 16 additions and products (and
           the rescalings, one per tile) at u each:
           sum_j p_j |v_j| (e_j + sum_i p_i e_i + 2 (L + 64) u)
  bf16 on the tensor cores: the weights are rounded to bf16 (half a step,
           2^-8) where they multiply the values, not in the sum below the line;
  bf16 result: half a step of the result, 2^-8 |y|.
Row bounds are never below 1e-30.
"""
import numpy as np

U = 2.0 ** -24
HALF_BF16 = 2.0 ** -8


def attend(q, k, v, visible, scale, tensor_core):
    """q [n, nh, hd], k, v [L, nkv, hd], visible bool [n, L] -> y, bound
    [n, nh, hd].  A key that a row does not see is taken out of its sums."""
    n, nh, hd = q.shape
    L, nkv = k.shape[:2]
    y, b = np.zeros((n, nh, hd)), np.full((n, nh, hd), 1e-30)
    rows = visible.any(axis=1)
    if not rows.any():
        return y, b
    seen = visible.any(axis=0)  # keys that some row sees
    k, v, vis, q = k[seen], v[seen], visible[rows][:, seen], q[rows]
    low = HALF_BF16 if tensor_core else 0.0
    for h in range(nh):
        kh, vh = k[:, h // (nh // nkv)], v[:, h // (nh // nkv)]
        s = np.where(vis, scale * (q[:, h] @ kh.T), -np.inf)
        top = np.where(vis, np.abs(s), 0).max(axis=1, keepdims=True)
        es = (hd + 4) * U * scale * (np.abs(q[:, h]) @ np.abs(kh).T) + 4 * U * top
        p = np.exp(s - s.max(axis=1, keepdims=True))
        p /= p.sum(axis=1, keepdims=True)
        e = np.expm1(es) + 2.0 ** -21
        mean_e = (p * e).sum(axis=1, keepdims=True)
        y[rows, h] = p @ vh
        b[rows, h] = (p * (e + mean_e + 2 * (L + 64) * U + low)) @ np.abs(vh) + 1e-30
    return y, b


def _pack(parts, q):
    """The requests' rows one after another; rows of no request are zeros."""
    t = sum(len(y) for y, _ in parts)
    pad = (len(q) - t,) + q.shape[1:]
    return (np.concatenate([y for y, _ in parts] + [np.zeros(pad)]),
            np.concatenate([b for _, b in parts] + [np.full(pad, 1e-30)]))


def prompt(q, k, v, lens, scale, tensor_core=False):
    parts, t = [], 0
    for n in lens:
        vis = np.tril(np.ones((n, n), dtype=bool))
        parts.append(attend(q[t:t + n], k[t:t + n], v[t:t + n], vis, scale, tensor_core))
        t += n
    return _pack(parts, q)


def paged(q, k_cache, v_cache, table, lens, scale, tensor_core=False):
    """lens: (cache rows, new tokens) of each request."""
    nb, nkv, S, hd = k_cache.shape
    parts, t = [], 0
    for r, (L, n) in enumerate(lens):
        j = np.arange(L)
        ids = table[r][j // S]
        ok = (ids >= 0) & (ids < nb)
        ids = np.where(ok, ids, 0)
        k, v = k_cache[ids, :, j % S].copy(), v_cache[ids, :, j % S].copy()
        k[~ok] = v[~ok] = 0.0
        vis = (j[None, :] <= (L - n + np.arange(n))[:, None]) & ok[None, :]
        parts.append(attend(q[t:t + n], k, v, vis, scale, tensor_core))
        t += n
    return _pack(parts, q)


def plan(ctx, new, table, free, S, T):
    """The plan in Python integers: table, cu, kv_lens, positions, slots, used, short."""
    table = table.copy()
    cols = table.shape[1]
    cu, pos, slot, used, short = [0], [], [], 0, False
    for r, (c, n) in enumerate(zip(ctx, new)):
        c, n = max(c, 0), max(n, 0)
        have, need = -(-c // S), -(-(c + n) // S)
        short |= need > cols
        for b in range(min(have, cols), min(need, cols)):
            if used < len(free):
                table[r, b] = free[used]
            else:
                table[r, b] = -1
                short = True
            used += 1
        for p in range(c, c + n):
            b = p // S
            ok = b < cols and table[r, b] >= 0
            pos.append(p)
            slot.append(int(table[r, b]) * S + p % S if ok else -1)
        cu.append(cu[-1] + n)
    short |= cu[-1] > T
    pos, slot = (pos + [-1] * T)[:T], (slot + [-1] * T)[:T]
    kvl = [max(c, 0) + max(n, 0) for c, n in zip(ctx, new)]
    return table, cu, kvl, pos, slot, used, short


def rope(x, pos, cos, sin, n_rot):
    """x [T, heads, hd], the first n_rot heads turned -> y, bound (fp32 products)."""
    y, b = x.copy(), np.zeros_like(x)
    for t, p in enumerate(pos):
        if p < 0 or p >= len(cos):
            y[t] = 0
            continue
        c, s = cos[p], sin[p]
        a, d = x[t, :n_rot, 0::2], x[t, :n_rot, 1::2]
        y[t, :n_rot, 0::2], y[t, :n_rot, 1::2] = a * c - d * s, a * s + d * c
        b[t, :n_rot, 0::2] = 2 * U * (np.abs(a * c) + np.abs(d * s))
        b[t, :n_rot, 1::2] = 2 * U * (np.abs(a * s) + np.abs(d * c))
    return y, b
