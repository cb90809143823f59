"""The 4-bit paged cache in plain numpy: the codes bit for bit, and attention
over them in 64 bits with the bound its results are held to.  Nothing shared
with the kernels.

Quantising is defined in fp32, each step one rounding, so that codes, scales
and zero points are compared for equality.  The rotation's fma is computed in
64 bits (its product is exact there) and rounded once.

Attention (u = 2^-24, half a step of fp32; the tensor cores cut a sum off where
fp32 would round, 2 u a term).  A value is (code - zp) s; the kernels sum codes
and zero points apart, so the errors go by s (code + |zp|), named size:
  score    scale q.k in log2 units: es = scale 2 u (hd + 16) sum |q| size + 4 u top
           plus what the queries' 16-bit parts leave out: 2^-22 of |q| with fp32
           queries (two parts of 11 bits), and for elements far below the row's
           largest 2^-34 of the largest
  weight   relative e = expm1(es) + 2^-21 (the exponential's own error)
  weight times scale, to 16 bits: 2^-11 with bf16 queries, two parts (2^-22)
           with fp32 ones; below fp16's normal range half a step of 2^-24,
           where the largest product of the row is at least 2^4: 2^-29 of it
  tiles    (bf16 queries, head sizes up to 128, many rows a request): keys are
           rounded to fp16, half a step, 2^-11 of every q k in a score (2^-25 of q
           below fp16's normal range), values and weights to bf16, 2^-8 of every
           p v twice in the result
  result   sum_j p_j |v_j| (e_j + sum_i p_i e_i) for the weights above and below
           the line, sum_j p_j size_j 2 (L + 64) u for the sums, sum_j p_j s_j
           code_j (rounding) for the products.
"""
import numpy as np

U = 2.0 ** -24
f32 = np.float32


def chunks(hd):
    n = -(-hd // 32)
    return n if n <= 4 else n + n % 2


def strip_bytes(hd, group):
    return 512 * chunks(hd) + 128 * (-(-hd // group))


def quantise(x, group):
    """x fp32 [..., hd] -> codes [..., hd] uint8, zps, scales [..., G] fp32."""
    x = np.asarray(x, dtype=f32)
    codes = np.zeros(x.shape, dtype=np.uint8)
    zps, scales = [], []
    with np.errstate(all="ignore"):
        for d in range(0, x.shape[-1], group):
            v = x[..., d:d + group]
            bad = ~np.isfinite(v).all(-1, keepdims=True)
            lo, hi = v.min(-1, keepdims=True), v.max(-1, keepdims=True)
            top = np.maximum(np.abs(lo), np.abs(hi))
            s = (hi * f32(2.0 ** -4) - lo * f32(2.0 ** -4)) * f32(16.0 / 15.0)
            s = np.maximum(np.maximum(s, top * f32(2.0 ** -11)), f32(2.0 ** -100))
            bits = np.ascontiguousarray(s).view(np.uint32)
            s = ((bits + np.uint32(0xFFFF)) & np.uint32(0xFFFF0000)).view(f32)
            inv = f32(1.0) / s
            zp = -np.rint(lo * inv)
            c = np.clip(np.rint(v * inv) + zp, 0, 15)
            codes[..., d:d + group] = np.where(bad, 0, c).astype(np.uint8)
            zps.append(np.where(bad, f32(0), zp + f32(0)))
            scales.append(np.where(bad, f32(np.nan), s))
    return codes, np.concatenate(zps, -1), np.concatenate(scales, -1)


def row_bytes(hd, group, r, kcodes, kz, ks, vcodes, vz, vs):
    """Byte offsets in its strip and bytes of row r of one head, from one row's
    codes [hd] and parameters [G]."""
    nc, G = chunks(hd), -(-hd // group)
    out = {}

    def nibble(at, j, code):
        out[at + j // 2] = out.get(at + j // 2, 0) | int(code) << (4 * (j % 2))

    for d in range(32 * nc):
        c, w = divmod(d, 32)
        kc, vc = (kcodes[d], vcodes[d]) if d < hd else (0, 0)
        nibble(((r * 4 + w // 8) * nc + c) * 4, w % 8, kc)
        nibble(256 * nc + (((r // 8 * 8 + w // 4) * 4 + r % 8 // 2) * nc + c) * 4 + 2 * (r % 2), w % 4, vc)
    for first, z, s in ((512 * nc, kz, ks), (512 * nc + 64 * G, vz, vs)):
        for g in range(G):
            word = int(np.float16(z[g]).view(np.uint16)) | int(np.array(s[g], f32).view(np.uint32)) & 0xFFFF0000
            if np.isnan(s[g]):
                word = 0x7FC00000
            for b in range(4):
                out[first + 4 * (r * G + g) + b] = word >> (8 * b) & 255
    return np.array(list(out.keys())), np.array(list(out.values()), dtype=np.uint8)


def put(data, hd, group, S, slot, k, v):
    """Stores rows k, v fp32 [n_kv, hd] in slot of data uint8 [nb, n_kv, bytes]."""
    kq, vq = quantise(k, group), quantise(v, group)
    row = slot % S
    for h in range(data.shape[1]):
        at, b = row_bytes(hd, group, row % 16, kq[0][h], kq[1][h], kq[2][h], vq[0][h], vq[1][h], vq[2][h])
        data[slot // S, h, row // 16 * strip_bytes(hd, group) + at] = b


def unpack(data, hd, group, S):
    """data uint8 [nb, n_kv, bytes] -> two (codes, zps, scales), codes [nb, n_kv,
    S, hd], zps and scales [nb, n_kv, S, G]."""
    nb, nkv, _ = data.shape
    nc, G = chunks(hd), -(-hd // group)
    d = data.reshape(nb, nkv, S // 16, strip_bytes(hd, group))
    r, dim = np.arange(16)[:, None], np.arange(hd)[None, :]
    c, w = dim // 32, dim % 32
    places = ((((r * 4 + w // 8) * nc + c) * 4 + w % 8 // 2),
              256 * nc + (((r // 8 * 8 + w // 4) * 4 + r % 8 // 2) * nc + c) * 4 + 2 * (r % 2) + w % 4 // 2)
    out = []
    for at, first in zip(places, (512 * nc, 512 * nc + 64 * G)):
        byte = d[..., at]
        codes = np.where(dim % 2 == 1, byte >> 4, byte & 15).reshape(nb, nkv, S, hd)
        par = np.ascontiguousarray(d[..., first:first + 64 * G]).view(np.uint32).reshape(nb, nkv, S, G)
        with np.errstate(invalid="ignore"):  # rows that were never stored
            zp = (par & np.uint32(0xFFFF)).astype(np.uint16).view(np.float16).astype(np.float64)
            s = (par & np.uint32(0xFFFF0000)).view(f32).astype(np.float64)
        out.append((codes.astype(np.float64), zp, s))
    return out


def values(part, group):
    codes, zp, s = part
    hd = codes.shape[-1]
    spread = lambda t: np.repeat(t, group, -1)[..., :hd]
    return (codes - spread(zp)) * spread(s)


def rope32(x, pos, cos, sin, n_rot):
    """x fp32 [T, heads, hd] with its first n_rot heads turned as fp32 holds
    them: fma(a, c, -(b s)), fma(a, s, b c)."""
    y = np.array(x, dtype=f32)
    for t, p in enumerate(pos):
        if p < 0 or p >= len(cos):
            y[t] = 0
            continue
        c, s = f32(cos[p]), f32(sin[p])
        a, b = x[t, :n_rot, 0::2], x[t, :n_rot, 1::2]
        d = np.float64
        y[t, :n_rot, 0::2] = (a.astype(d) * c.astype(d) - (b * s).astype(d)).astype(f32)
        y[t, :n_rot, 1::2] = (a.astype(d) * s.astype(d) + (b * c).astype(d)).astype(f32)
    return y


def attend(q, keys, vals, group, visible, scale, q32, tiles=False):
    """q [n, nh, hd]; keys, vals: codes [L, nkv, hd], zps, scales [L, nkv, G];
    visible bool [n, L] -> y, bound [n, nh, hd]."""
    n, nh, hd = q.shape
    L, nkv = keys[0].shape[:2]
    y, b = np.zeros((n, nh, hd)), np.full((n, nh, hd), 1e-30)
    rows = visible.any(axis=1)
    if not rows.any():
        return y, b
    seen = visible.any(axis=0)
    keys, vals = [t[seen] for t in keys], [t[seen] for t in vals]
    vis, q = visible[rows][:, seen], q[rows]
    spread = lambda t: np.repeat(t, group, -1)[..., :hd]
    k, v = values(keys, group), values(vals, group)
    ksize = (keys[0] + np.abs(spread(keys[1]))) * spread(keys[2])
    vsize = (vals[0] + np.abs(spread(vals[1]))) * spread(vals[2])
    vcode = vals[0] * spread(vals[2])
    low = 2.0 ** -22 if q32 else 2.0 ** -11
    for h in range(nh):
        g = h // (nh // nkv)
        qh = np.abs(q[:, h])
        s = np.where(vis, scale * (q[:, h] @ k[:, g].T), -np.inf)
        top = np.where(vis, np.abs(s), 0).max(axis=1, keepdims=True)
        es = scale * (2 * U * (hd + 16) + (2.0 ** -22 if q32 else 0)) * (qh @ ksize[:, g].T) + 4 * U * top
        if tiles:
            es += scale * (2.0 ** -11 * (qh @ np.abs(k[:, g]).T) + 2.0 ** -25 * qh.sum(axis=1, keepdims=True))
        es += scale * 2.0 ** -34 * qh.max(axis=1, keepdims=True) * ksize[:, g].sum(-1)
        p = np.where(vis, np.exp(s - s.max(axis=1, keepdims=True)), 0)
        p /= p.sum(axis=1, keepdims=True)
        e = np.expm1(es) + 2.0 ** -21
        mean_e = (p * e).sum(axis=1, keepdims=True)
        small = 2.0 ** -29 * (p[:, :, None] * spread(vals[2])[None, :, g]).max(axis=1) * 15 * len(k)
        y[rows, h] = p @ v[:, g]
        rounded = p @ np.abs(v[:, g]) * (2 * 2.0 ** -8 + 2.0 ** -16) if tiles else p @ vcode[:, g] * low + small
        b[rows, h] = ((p * (e + mean_e)) @ np.abs(v[:, g]) + p @ vsize[:, g] * (2 * (L + 64) * U) + rounded + 1e-30)
    return y, b


def paged(q, data, group, S, table, lens, scale, q32):
    """lens: (cache rows, new tokens) of each request.  Tiles: requests with more
    than 32 query rows to a key/value head in a call of six or more that has 512
    such rows beyond a token a request (1024 where the average is at most 32), all
    requests of other calls with more than 32 on average."""
    nb, hd = data.shape[0], q.shape[2]
    grp, R = q.shape[1] // data.shape[1], len(lens)
    tc = not q32 and hd <= 128
    both = R >= 6 and (len(q) - R) * grp >= (512 if len(q) * grp > 32 * R else 1024)
    tiles = [tc and (n * grp > 32 if both else len(q) * grp > 32 * R) for _, n in lens]
    kk, vv = unpack(data, hd, group, S)
    parts, t = [], 0
    for r, (L, n) in enumerate(lens):
        j = np.arange(L)
        ids = table[r][j // S]
        ok = (ids >= 0) & (ids < nb)
        ids = np.where(ok, ids, 0)
        rows = [[t_[ids, :, j % S] for t_ in part] for part in (kk, vv)]
        vis = (j[None, :] <= (L - n + np.arange(n))[:, None]) & ok[None, :]
        parts.append(attend(q[t:t + n], *rows, group, vis, scale, q32, tiles[r]))
        t += n
    pad = (len(q) - t,) + q.shape[1:]
    return (np.concatenate([y for y, _ in parts] + [np.zeros(pad)]),
            np.concatenate([b for _, b in parts] + [np.full(pad, 1e-30)]))
