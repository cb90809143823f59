"""The operators of a paged cache held in 4 bits: the sizes they are timed at,
their inputs, their plain form, and their outputs computed in 64 bits.

  append  rotary positions, and keys and values quantised into their pages
          (rope_append with a 4-bit cache); its cache is returned as the values
          that it stands for (kv4_read)
  read    rows of the cache as numbers (kv4_read)
  attend  attention of each request's new tokens (one or many) over its pages
          (attn_paged with a 4-bit cache)

The cache: ``data`` uint8 [blocks, key/value heads, bytes], in strips of 16
rows.  A strip of one head holds, with NC chunks of 32 dimensions and G groups:

  key codes    32-bit words [16 rows][4][NC]; nibble j (low ones first) of word
               (r, t, c) is dimension 32 c + 8 t + j of row r
  value codes  words [2][8][4][NC]; the low half of word (h, g, t, c) belongs to
               row 8 h + 2 t, the high half to the row after it, and nibble j of
               a half is dimension 32 c + 4 g + j
  key scales   words [16][G]: zero point (fp16, a whole number) and scale (bf16)
  value scales the same
  value = (code - zero point) scale

``run`` computes the operators in elementary torch operations, or, where
``own`` is true, through the package's entry points.
"""
import math
import random

import numpy as np
import torch

own = False

BASE = 10000.0  # base of the rotary frequencies

# query heads, key/value heads, head size
SHAPES = ((32, 8, 128), (32, 8, 128), (64, 8, 128), (32, 32, 128), (32, 4, 64), (16, 2, 64), (10, 10, 64),
          (28, 4, 80), (12, 4, 96), (6, 1, 128), (8, 2, 32), (16, 4, 256))
MAX_FLOPS = 6e11  # of a drawn attention case: just below the largest listed ones
MAX_BYTES = 4.4e8


def listed():
    return [
        # the tokens of a small decode batch, from fp32 projections
        dict(name="append_decode_7", op="append", tokens=7, nh=32, nkv=8, hd=128, group=64, x="f32", q="bf16",
             block=16, keep=False, pad=0, shape=21),
        # a padded step of mixed prompts, head size no power of two, fp32 queries
        dict(name="append_mixed_1500", op="append", tokens=1500, nh=28, nkv=4, hd=80, group=32, x="f32", q="f32",
             block=32, keep=True, pad=9, shape=22),
        # a large prompt step
        dict(name="append_prompt_16384", op="append", tokens=16384, nh=32, nkv=8, hd=128, group=64, x="bf16",
             q="bf16", block=64, keep=False, pad=0, shape=23),
        # the context of one short request, to be kept elsewhere
        dict(name="read_one_300", op="read", rows=300, nkv=8, hd=128, group=64, block=16, y="f32", pad=3, shape=31),
        # the contexts of several long requests
        dict(name="read_long_100000", op="read", rows=100000, nkv=8, hd=128, group=64, block=64, y="bf16", pad=0,
             shape=32),
        # one user, one token at a time
        dict(name="decode_one_1500", op="attend", requests=1, ctx_max=1500, ctx_min=1500, chunk_max=1, chunks=0,
             nh=32, nkv=8, hd=128, group=64, dtype="bf16", block=16, shape=41),
        # a full decode batch of ragged contexts
        dict(name="decode_batch_64", op="attend", requests=64, ctx_max=16384, ctx_min=100, chunk_max=1, chunks=0,
             nh=32, nkv=8, hd=128, group=64, dtype="bf16", block=16, shape=42),
        # few users with whole books as context, what a 4-bit cache is for
        dict(name="decode_long_3", op="attend", requests=3, ctx_max=131072, ctx_min=100000, chunk_max=1, chunks=0,
             nh=64, nkv=8, hd=128, group=32, dtype="bf16", block=64, shape=43),
        # fp32 queries, as many key/value heads as query heads
        dict(name="decode_f32_12", op="attend", requests=12, ctx_max=4001, ctx_min=1, chunk_max=1, chunks=0, nh=32,
             nkv=32, hd=128, group=64, dtype="f32", block=32, shape=44),
        # a few tokens a request at once (drafted ones that are checked), small heads
        dict(name="draft_30", op="attend", requests=30, ctx_max=6000, ctx_min=20, chunk_max=5, chunks=30, nh=28,
             nkv=4, hd=80, group=32, dtype="bf16", block=32, shape=45),
        # chunks of prompts beside decoding requests
        dict(name="chunk_mixed_20", op="attend", requests=20, ctx_max=32768, ctx_min=64, chunk_max=2048, chunks=4,
             nh=32, nkv=8, hd=128, group=64, dtype="bf16", block=64, shape=46),
        # one chunk with fp32 queries
        dict(name="chunk_f32_300", op="attend", requests=2, ctx_max=2500, ctx_min=900, chunk_max=300, chunks=1,
             nh=32, nkv=8, hd=128, group=64, dtype="f32", block=128, shape=47),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(("append", "append", "read", "attend", "attend", "attend", "attend"))
    shape = rng.randrange(1 << 30)
    nh, nkv, hd = rng.choice(SHAPES)
    block, group = rng.choice((16, 32, 64, 128, 256)), rng.choice((32, 64))
    if op == "append":
        cap = max(1, int(8e7) // ((nh + 2 * nkv) * hd))
        return dict(op=op, tokens=_log(rng, 1, min(16384, cap)), nh=nh, nkv=nkv, hd=hd, group=group,
                    x=rng.choice(("f32", "bf16")), q=rng.choice(("bf16", "bf16", "f32")), block=block,
                    keep=rng.choice((False, True)), pad=rng.choice((0, 0, 5)), shape=shape)
    if op == "read":
        return dict(op=op, rows=_log(rng, 1, min(100000, int(1e8) // (nkv * hd))), nkv=nkv, hd=hd, group=group,
                    block=block, y=rng.choice(("bf16", "f32")), pad=rng.choice((0, 0, 7)), shape=shape)
    dtype = "f32" if rng.random() < 0.25 else "bf16"
    cap = MAX_FLOPS / 20 if dtype == "f32" else MAX_FLOPS
    while True:
        R = _log(rng, 1, 128)
        chunks = rng.choice((0, 0, 0, R, _log(rng, 1, 8)))
        case = dict(op=op, requests=R, ctx_max=_log(rng, 1, 131072), ctx_min=1,
                    chunk_max=rng.choice((_log(rng, 2, 2048), rng.randint(2, 8))) if chunks else 1,
                    chunks=min(chunks, R), nh=nh, nkv=nkv, hd=hd, group=group, dtype=dtype, block=block, shape=shape)
        w = work(case)
        if w["flops"] <= cap and w["bytes"] <= MAX_BYTES:
            return case


# ------------------------------------------------------------------ sizes

def _paged_lengths(case):
    """(cache length with the new tokens, new tokens) of the requests."""
    r = random.Random(case["shape"])
    out = []
    for i in range(case["requests"]):
        n = 1 if i >= case["chunks"] else _log(r, max(2, case["chunk_max"] // 4), case["chunk_max"])
        lo, hi = case["ctx_min"], case["ctx_max"]
        out.append((n - 1 + r.randint(lo, hi) if r.random() < 0.5 else n - 1 + _log(r, lo, hi), n))
    r.shuffle(out)
    return out


def _blocks(n, size):
    return -(-n // size)


def _chunks(hd):
    """Chunks of 32 dimensions that a strip holds: beyond four, an even number."""
    n = _blocks(hd, 32)
    return n if n <= 4 else n + n % 2


def _strip_bytes(hd, group):
    return 512 * _chunks(hd) + 128 * _blocks(hd, group)


def work(case):
    op = case["op"]
    nkv, hd = case["nkv"], case["hd"]
    row = nkv * (hd + 8 * _blocks(hd, case["group"]))  # bytes of a row's keys and values in the cache
    if op == "append":
        T, nh = case["tokens"], case["nh"]
        bi, bo = (4 if case["x"] == "f32" else 2), (4 if case["q"] == "f32" else 2)
        kept = 2 * nkv * hd * bo if case["keep"] else 0
        stored = 2 * nkv * hd * bo  # the values the cache stands for, read again
        return {"bytes": T * ((nh + 2 * nkv) * hd * bi + nh * hd * bo + kept + 2 * row + stored + hd * 4 + 12),
                "flops": T * (nh + nkv) * hd * 3 + T * nkv * hd * 12}
    if op == "read":
        return {"bytes": case["rows"] * (row + 2 * nkv * hd * (4 if case["y"] == "f32" else 2) + 8),
                "flops": case["rows"] * nkv * hd * 4}
    nh, b = case["nh"], 4 if case["dtype"] == "f32" else 2
    lens = _paged_lengths(case)
    pairs = sum(n * (L - n) + n * (n + 1) // 2 for L, n in lens)
    return {"bytes": sum(L * row + 2 * n * nh * hd * b + 4 * _blocks(L, case["block"]) for L, n in lens),
            "flops": 4 * hd * nh * pairs}


# ------------------------------------------------------------------ the cache's form

def _quantise(x, group):
    """x [..., hd] fp32 -> codes uint8 [..., hd], zero points and scales fp32
    [..., G].  Every step is one rounding in 32 bits, so that the codes are
    defined bit for bit."""
    hd = x.shape[-1]
    codes, zps, scales = torch.empty_like(x, dtype=torch.uint8), [], []
    for d in range(0, hd, group):
        v = x[..., d:d + group]
        lo, hi = v.amin(-1, keepdim=True), v.amax(-1, keepdim=True)
        top = torch.maximum(lo.abs(), hi.abs())
        s = torch.maximum((hi * 0.0625 - lo * 0.0625) * (16.0 / 15.0), top * 2.0 ** -11).clamp_min(2.0 ** -100)
        s = ((s.view(torch.int32) + 0xFFFF) & -65536).view(torch.float32)  # up to the next bf16
        inv = 1.0 / s
        zp = -torch.round(lo * inv)
        c = (torch.round(v * inv) + zp).clamp(0, 15)
        good = top <= 3.4028234663852886e38
        codes[..., d:d + group] = torch.where(good, c, 0.0).to(torch.uint8)
        zps.append(torch.where(good, zp, 0.0))
        scales.append(torch.where(good, s, math.nan))
    return codes, torch.cat(zps, -1), torch.cat(scales, -1)


def _params(zp, s):
    """Zero points and scales as the cache's bytes [..., G * 4]."""
    z = zp.half().view(torch.int16)
    return torch.stack([z, s.bfloat16().view(torch.int16)], -1).flatten(-2).view(torch.uint8)


def _padded(codes, hd):
    return torch.nn.functional.pad(codes, (0, 32 * _chunks(hd) - hd))


def _pack_strips(k, v, group):
    """k, v fp32 [n, heads, rows, hd], rows a multiple of 16 -> uint8 [n, heads, bytes]."""
    n, h, rows, hd = k.shape
    nc = _chunks(hd)
    kc, kz, ks = _quantise(k, group)
    vc, vz, vs = _quantise(v, group)
    kc = _padded(kc, hd).view(n, h, rows // 16, 16, nc, 4, 8).transpose(4, 5)  # row, t, c, j
    vc = _padded(vc, hd).view(n, h, rows // 16, 2, 4, 2, nc, 8, 4).permute(0, 1, 2, 3, 7, 4, 6, 5, 8)
    parts = [(c[..., 0::2] | (c[..., 1::2] << 4)).flatten(3) for c in (kc, vc)]
    parts += [_params(z, s).view(n, h, rows // 16, -1) for z, s in ((kz, ks), (vz, vs))]
    return torch.cat(parts, -1).flatten(2)


def _unpack_strips(data, hd, group):
    """uint8 [n, heads, bytes] -> k, v fp32 [n, heads, rows, hd]."""
    n, h, _ = data.shape
    nc, G = _chunks(hd), _blocks(hd, group)
    d = data.view(n, h, -1, _strip_bytes(hd, group))
    strips = d.shape[2]
    kc, vc = d[..., :256 * nc], d[..., 256 * nc:512 * nc]
    nib = lambda c: torch.stack([c & 15, c >> 4], -1)  # noqa: E731
    kc = nib(kc).view(n, h, strips, 16, 4, nc, 8).transpose(4, 5).reshape(n, h, strips * 16, nc * 32)
    vc = nib(vc).view(n, h, strips, 2, 8, 4, nc, 2, 4).permute(0, 1, 2, 3, 5, 7, 6, 4, 8)
    vc = vc.reshape(n, h, strips * 16, nc * 32)
    out = []
    for c, at in ((kc, 512 * nc), (vc, 512 * nc + 64 * G)):
        p = d[..., at:at + 64 * G].contiguous().view(torch.int16).view(n, h, strips * 16, G, 2)
        zp = p[..., 0].contiguous().view(torch.float16).float()
        s = p[..., 1].contiguous().view(torch.bfloat16).float()
        zp, s = (t.repeat_interleave(group, -1)[..., :hd] for t in (zp, s))
        out.append((c[..., :hd].float() - zp) * s)
    return out


# ------------------------------------------------------------------ inputs

def _dtype(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def _normal(gen, shape, dtype, scale=1.0):
    t = torch.empty(shape, dtype=dtype, device="cuda")
    return t.normal_(0.0, scale, generator=gen)


def _rotary_tables(positions, hd):
    """cos, sin fp32 [positions, hd / 2] of p * BASE^(-2i / hd), angles in 64 bits."""
    inv = BASE ** (-torch.arange(0, hd, 2, dtype=torch.float64, device="cuda") / hd)
    a = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * inv[None, :]
    return torch.cos(a).float(), torch.sin(a).float()


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _prefix(lens):
    return _i32(np.concatenate([[0], np.cumsum(np.asarray(lens, dtype=np.int64))]).astype(np.int32))


def _filled_cache(gen, case, pool):
    """A cache of random rows: channels of unlike spread and offset, as keys have them."""
    nkv, hd, S, group = case["nkv"], case["hd"], case["block"], case["group"]
    gain = torch.exp(0.4 * _normal(gen, (2, nkv, 1, hd), torch.float32))
    mean = _normal(gen, (2, nkv, 1, hd), torch.float32, 0.3)
    data = torch.empty((pool, nkv, S // 16 * _strip_bytes(hd, group)), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 25) // (nkv * S * hd))
    for b in range(0, pool, step):
        n = min(step, pool - b)
        k, v = (_normal(gen, (n, nkv, S, hd), torch.float32) * gain[i] + mean[i] for i in range(2))
        data[b:b + n] = _pack_strips(k, v, group)
    return data


def _runs(case, T, rng, longest):
    """Positions and slots of T tokens in runs of one to a thousand consecutive
    rows, as prompts and single tokens give, and the blocks that they take."""
    S = case["block"]
    pos, slot, n, lens, runs = np.empty(T, np.int32), np.empty(T, np.int64), 0, [], random.Random(case["shape"])
    while n < T:
        L = min(T - n, runs.choice(longest))
        lens.append((n, L, runs.randrange(6000)))
        n += L
    blocks = sum(_blocks(L + p % S, S) for _, L, p in lens) + 8
    perm, b = rng.permutation(blocks), 0
    for n, L, p in lens:
        mine = perm[b:b + _blocks(L + p % S, S)]
        b += len(mine)
        j = p % S + np.arange(L)
        pos[n:n + L] = p + np.arange(L)
        slot[n:n + L] = mine[j // S] * S + j % S
    pad = case["pad"]  # padding rows at the end have neither position nor slot
    return np.concatenate([pos, np.full(pad, -1, np.int32)]), np.concatenate([slot, np.full(pad, -1, np.int64)]), blocks


def _inputs(case, seed):
    """The tensors a program has before the call, from the seed."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rng = np.random.default_rng(seed)
    op, nkv, hd, S = case["op"], case["nkv"], case["hd"], case["block"]
    s = dict(case)
    if op == "append":
        T, nh = case["tokens"], case["nh"]
        pos, slot, blocks = _runs(case, T, rng, (1, 1, 7, 200, 1000))
        cos, sin = _rotary_tables(8192, hd)
        s.update(qkv=_normal(gen, (T + case["pad"], (nh + 2 * nkv) * hd), _dtype(case["x"])),
                 positions=torch.from_numpy(pos).cuda(), slots=torch.from_numpy(slot).cuda(), cos=cos, sin=sin,
                 data=torch.zeros((blocks, nkv, S // 16 * _strip_bytes(hd, case["group"])), dtype=torch.uint8,
                                  device="cuda"),
                 every=torch.arange(blocks * S, device="cuda"))
        return s
    if op == "read":
        _, slot, blocks = _runs(case, case["rows"], rng, (300, 1500, 20000))
        s.update(slots=torch.from_numpy(slot).cuda(), data=_filled_cache(gen, case, blocks))
        return s
    lens = _paged_lengths(case)
    need = [_blocks(L, S) for L, _ in lens]
    pool = sum(need) + 16
    perm = rng.permutation(pool).astype(np.int32)
    table = np.full((len(lens), max(need) + 2), -1, dtype=np.int32)
    used = 0
    for r, n in enumerate(need):
        table[r, :n] = perm[used:used + n]
        used += n
    T = sum(n for _, n in lens)
    s.update(lens=lens, cu=_prefix([n for _, n in lens]), kv_lens=_i32([L for L, _ in lens]),
             block_table=torch.from_numpy(table).cuda(),
             q=_normal(gen, (T, case["nh"], hd), _dtype(case["dtype"]), 1.5), data=_filled_cache(gen, case, pool))
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        import group_quantized_moe_gb300 as lib

        s["lib"] = lib
        s["cache"] = lib.PagedKV4(s["data"], s["hd"], s["group"], s["block"])
        if s["op"] == "attend":  # a program keeps one workspace for all of its calls
            n = lib.qmm_attn_paged_workspace_bytes(s["q"], s["cache"], s["requests"])
            s["workspace"] = torch.empty((n,), dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    return (_run_own if own else _run_plain)[s["op"]](s)


def _own_append(s):
    q, k, v = s["lib"].rope_append(s["qkv"], s["nh"], s["positions"], s["slots"], s["cos"], s["sin"], s["cache"],
                                   keep_kv=s["keep"], y_dtype=_dtype(s["q"]))
    held = s["lib"].kv4_read(s["cache"], s["every"], y_dtype=_dtype(s["q"]))
    out = {"q": q, "held_k": held[0], "held_v": held[1]}
    if s["keep"]:
        out.update(k=k, v=v)
    return out


def _own_read(s):
    return s["lib"].kv4_read(s["cache"], s["slots"], y_dtype=_dtype(s["y"]))


def _own_attend(s):
    return s["lib"].attn_paged(s["q"], s["cache"], s["block_table"], s["cu"], s["kv_lens"], y_dtype=s["q"].dtype,
                               workspace=s["workspace"])


_run_own = {"append": _own_append, "read": _own_read, "attend": _own_attend}


def _row_places(s, heads, rows):
    """Byte offsets within a block of the codes and scales of `rows` (rows of
    their blocks) for all heads: [rows, heads, bytes]."""
    hd, S, nc, G = s["hd"], s["block"], _chunks(s["hd"]), _blocks(s["hd"], s["group"])
    dev, strip = rows.device, _strip_bytes(s["hd"], s["group"])
    ar = lambda n: torch.arange(n, device=dev)  # noqa: E731
    r = torch.arange(16, device=dev)[:, None]
    keys = r * 16 * nc + ar(16 * nc)
    word = (((r // 8 * 8 + ar(8)) * 4 + r % 8 // 2)[:, :, None] * nc + ar(nc)) * 4  # [16, 8, NC]
    values = 256 * nc + (word[..., None] + 2 * (r % 2)[:, :, None, None] + ar(2)).flatten(1)
    kp, vp = 512 * nc + r * 4 * G + ar(4 * G), 512 * nc + 64 * G + r * 4 * G + ar(4 * G)
    place = torch.cat([keys, values, kp, vp], 1)[rows % 16] + (rows // 16 * strip)[:, None]
    return place[:, None] + (ar(heads) * (S // 16 * strip))[:, None]


def _plain_append(s):
    nh, nkv, hd, S, group = s["nh"], s["nkv"], s["hd"], s["block"], s["group"]
    pos, slot = s["positions"].long(), s["slots"]
    x = s["qkv"].float().view(-1, nh + 2 * nkv, hd)
    # (a, b) -> (fma(a, c, -(b s)), fma(a, s, b c)): one product rounded to 32 bits, the other
    # not, then the sum; in 64 bits, because a code next to a border hangs on the last one
    c, n = s["cos"][pos.clamp(min=0)][:, None, :], s["sin"][pos.clamp(min=0)][:, None, :]
    a, b = x[:, :nh + nkv, 0::2], x[:, :nh + nkv, 1::2]
    u = (a.double() * c.double() - (b * n).double()).float()
    w = (a.double() * n.double() + (b * c).double()).float()
    rot = torch.stack([u, w], dim=-1).flatten(2)
    x = torch.cat([rot, x[:, nh + nkv:]], dim=1)
    if s["pad"]:
        x[pos < 0] = 0
    T = s["tokens"]  # the rows that are not padding
    k, v = x[:, nh:nh + nkv], x[:, nh + nkv:]
    bytes_ = []
    kc, kz, ks = _quantise(k[:T], group)
    vc, vz, vs = _quantise(v[:T], group)
    nc = _chunks(hd)
    kc = _padded(kc, hd).view(T, nkv, nc, 4, 8).transpose(2, 3)
    vc = _padded(vc, hd).view(T, nkv, nc, 8, 4).transpose(2, 3)
    for t in (kc, vc):
        bytes_.append((t[..., 0::2] | (t[..., 1::2] << 4)).flatten(2))
    bytes_ += [_params(kz, ks), _params(vz, vs)]
    s["data"].view(-1, s["data"][0].numel())[(slot[:T] // S)[:, None, None],
                                             _row_places(s, nkv, slot[:T] % S)] = torch.cat(bytes_, -1)
    dt = _dtype(s["q"])
    held = [t.transpose(1, 2).reshape(-1, nkv, hd).to(dt) for t in _unpack_strips(s["data"], hd, group)]
    res = {"q": x[:, :nh].to(dt), "held_k": held[0], "held_v": held[1]}
    if s["keep"]:
        res.update(k=k.to(dt), v=v.to(dt))
    return res


def _plain_read(s):
    S, group, slot = s["block"], s["group"], s["slots"]
    out = []
    for t in _unpack_strips(s["data"], s["hd"], group):
        rows = t[slot.clamp(min=0) // S, :, slot.clamp(min=0) % S]
        if s["pad"]:
            rows[slot < 0] = 0
        out.append(rows.to(_dtype(s["y"])))
    return out


def _plain_attention(q, k, v, scale):
    """q [n, nh, hd] over k, v [nkv, L, hd], query i sees keys 0 .. L - n + i;
    some key/value heads at a time, so that the scores fit."""
    n, nh, hd = q.shape
    nkv, L = k.shape[:2]
    g = nh // nkv
    hidden = (torch.arange(L, device=q.device)[None, :]
              > torch.arange(L - n, L, device=q.device)[:, None])
    out = torch.empty((n, nh, hd), dtype=torch.float32, device=q.device)
    step = max(1, (1 << 30) // max(1, n * g * L))
    for h in range(0, nkv, step):
        e = min(nkv, h + step)
        qh = q[:, h * g:e * g].float().reshape(n, e - h, g, hd).permute(1, 2, 0, 3)
        sc = torch.matmul(qh, k[h:e].transpose(1, 2)[:, None]) * scale
        if n > 1:
            sc = sc.masked_fill(hidden, -math.inf)
        p = torch.exp(sc - sc.amax(-1, keepdim=True))
        o = torch.matmul(p, v[h:e][:, None]) / p.sum(-1, keepdim=True)
        out[:, h * g:e * g] = o.permute(2, 0, 1, 3).reshape(n, (e - h) * g, hd)
    return out


def _plain_attend(s):
    outs, t = [], 0
    nkv, hd, S = s["nkv"], s["hd"], s["block"]
    for r, (L, n) in enumerate(s["lens"]):
        ids = s["block_table"][r, :_blocks(L, S)].long()
        k, v = (x.transpose(0, 1).reshape(nkv, -1, hd)[:, :L]
                for x in _unpack_strips(s["data"][ids], hd, s["group"]))
        outs.append(_plain_attention(s["q"][t:t + n], k, v, 1.0 / math.sqrt(hd)))
        t += n
    return torch.cat(outs).to(s["q"].dtype)


_run_plain = {"append": _plain_append, "read": _plain_read, "attend": _plain_attend}


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    """The outputs from the definitions, numbers in 64 bits."""
    s = _inputs(case, seed)
    return {"append": _exact_append, "read": _exact_read, "attend": _exact_attend}[s["op"]](s)


def _exact_rows(s, block, row):
    """Keys and values [len(row), heads, hd] of rows of blocks, code by code from the layout."""
    hd, nkv = s["hd"], s["nkv"]
    nc, G = _chunks(hd), _blocks(hd, s["group"])
    d = torch.arange(hd, device="cuda")
    c, w = d // 32, d % 32
    r = (row % 16)[:, None]
    base = row[:, None] // 16 * _strip_bytes(hd, s["group"])
    key = (r * 4 + w // 8) * 4 * nc + 4 * c + w % 8 // 2, d % 2
    val = 256 * nc + ((r // 8 * 8 + w // 4) * 4 + r % 8 // 2) * 4 * nc + 4 * c + 2 * (r % 2) + w % 4 // 2, d % 2
    out = []
    for (at, high), first in ((key, 512 * nc), (val, 512 * nc + 64 * G)):
        heads = []
        for h in range(nkv):
            mine = s["data"][:, h]
            byte = mine[block[:, None], base + at].int()
            code = torch.where(high == 1, byte >> 4, byte & 15)
            par = first + 4 * (r * G + d // s["group"])
            b = [mine[block[:, None], base + par + i].int() for i in range(4)]
            zp = (b[0] | b[1] << 8).short().view(torch.float16).double()
            scale = (b[2] << 16 | b[3] << 24).view(torch.float32).double()
            heads.append((code.double() - zp) * scale)
        out.append(torch.stack(heads, 1))
    return out


def _exact_read(s):
    slot = s["slots"]
    k, v = _exact_rows(s, slot.clamp(min=0) // s["block"], slot.clamp(min=0) % s["block"])
    k[slot < 0] = 0.0
    v[slot < 0] = 0.0
    return [k, v]


def _exact_append(s):
    nh, nkv, hd, T, group = s["nh"], s["nkv"], s["hd"], s["tokens"], s["group"]
    x = s["qkv"].double().reshape(-1, nh + 2 * nkv, hd // 2, 2)
    at = s["positions"].long().clamp(min=0)
    cos, sin = s["cos"][at].double()[:, None], s["sin"][at].double()[:, None]
    even, odd = x[:, :nh + nkv, :, 0], x[:, :nh + nkv, :, 1]
    turn = torch.view_as_real(torch.complex(even, odd) * torch.complex(cos, sin)).flatten(2)
    keep = (s["positions"] >= 0)[:, None, None]
    plain = torch.cat([turn, x[:, nh + nkv:].flatten(2)], 1) * keep
    # what is quantised is the rotated key as 32 bits hold it: the odd element's
    # product is rounded, then the sum
    r32 = lambda t: t.float().double()  # noqa: E731
    kept = torch.stack([r32(even * cos - r32(odd * sin)), r32(even * sin + r32(odd * cos))], -1).flatten(2)[:T, nh:]
    held = []
    for t in (kept, x[:T, nh + nkv:].flatten(2)):
        all_rows = torch.zeros((s["every"].numel(), nkv, hd), dtype=torch.float64, device="cuda")
        for first in range(0, hd, group):
            g = t[..., first:first + group]
            lo, hi = g.min(-1).values, g.max(-1).values
            step = torch.stack([r32(r32((hi - lo) / 16.0) * float(np.float32(16.0 / 15.0))),
                                torch.maximum(lo.abs(), hi.abs()) / 2048.0, torch.full_like(lo, 2.0 ** -100)]).amax(0)
            m, e = torch.frexp(step)
            step = torch.ldexp(torch.ceil(m * 256.0), e - 8)  # up to 8 bits
            inv = r32(1.0 / step)
            zero = torch.round(r32(lo * inv))
            code = torch.clamp(torch.round(r32(g * inv[..., None])) - zero[..., None], 0, 15)
            all_rows[s["slots"][:T], :, first:first + group] = (code + zero[..., None]) * step[..., None]
        held.append(all_rows)
    res = {"q": plain[:, :nh], "held_k": held[0], "held_v": held[1]}
    if s["keep"]:
        res.update(k=plain[:, nh:nh + nkv], v=plain[:, nh + nkv:])
    return res


def _exact_attend(s):
    S, hd, nkv = s["block"], s["hd"], s["nkv"]
    out, t = [], 0
    for r, (L, n) in enumerate(s["lens"]):
        # key j lies in row j mod S of page table[r, j div S]
        j = torch.arange(L, device="cuda")
        k, v = _exact_rows(s, s["block_table"][r][j // S].long(), j % S)
        q = s["q"][t:t + n].double()
        y = torch.zeros_like(q)
        for h in range(q.shape[1]):
            kh, vh = k[:, h * nkv // q.shape[1]], v[:, h * nkv // q.shape[1]]
            for i0 in range(0, n, 2048):
                i1 = min(n, i0 + 2048)
                logit = q[i0:i1, h] @ kh[:L - n + i1].T / hd ** 0.5
                late = (torch.arange(L - n + i1, device="cuda")
                        > torch.arange(L - n + i0, L - n + i1, device="cuda")[:, None])
                logit[late] = float("-inf")
                y[i0:i1, h] = torch.exp(logit - torch.logsumexp(logit, 1, keepdim=True)) @ vh[:L - n + i1]
        out.append(y)
        t += n
    return torch.cat(out)
