"""The paged-cache attention operators: the sizes they are timed at, their
inputs, their plain form, and their outputs computed in 64 bits.

Four operators that one serving step calls in order:

  plan    block tables and slot maps from the requests' lengths (kv_plan)
  append  rotary positions, and keys and values into their pages (rope_append)
  prompt  causal attention over packed prompts, grouped heads (attn_prompt)
  paged   attention of each request's new tokens (one or many) over its
          pages of the cache (attn_paged)

``run`` computes them in elementary torch operations, or, where ``own`` is
true, through the package's entry points.
"""
import math
import random

import numpy as np
import torch

own = False

BASE = 10000.0  # base of the rotary frequencies

# query heads, key/value heads, head size: from one query head per key/value
# head to eight, groups that are no power of two, head sizes likewise
SHAPES = ((32, 8, 128), (32, 8, 128), (32, 32, 128), (64, 8, 128), (32, 4, 64), (16, 2, 64),
          (10, 10, 64), (28, 4, 80), (12, 4, 96), (6, 1, 128), (8, 2, 32))
MAX_FLOPS = 1.1e12  # of a drawn attention case: just below the largest listed ones
MAX_BYTES = 1.4e9


def listed():
    return [
        # one decode step of a busy server: every request adds one token
        dict(name="plan_decode_256", op="plan", requests=256, ctx_max=32768, new_max=1, block=16,
             pad=0, shape=11),
        # admission of many prompts at once beside running requests, into a padded token buffer
        dict(name="plan_prompts_4096", op="plan", requests=4096, ctx_max=4096, new_max=300, block=32,
             pad=77, shape=12),
        # the tokens of a small decode batch, from fp32 projections into a bf16 cache
        dict(name="append_decode_7", op="append", tokens=7, nh=32, nkv=8, hd=128, x="f32",
             cache="bf16", block=16, keep=False, pad=0, shape=21),
        # a prompt step: bf16 projections, keys and values also kept packed for the prompt attention
        dict(name="append_prompt_16384", op="append", tokens=16384, nh=32, nkv=8, hd=128, x="bf16",
             cache="bf16", block=64, keep=True, pad=0, shape=22),
        # one short question
        dict(name="prompt_short_37", op="prompt", seqs=1, tokens=37, nh=16, nkv=2, hd=64,
             dtype="bf16", shape=31),
        # ordinary prompts of mixed lengths, a head size that is no power of two
        dict(name="prompt_mixed_hd80", op="prompt", seqs=9, tokens=5003, nh=28, nkv=4, hd=80,
             dtype="bf16", shape=32),
        # fp32 activations as the quantised projections give them by default
        dict(name="prompt_f32_1500", op="prompt", seqs=3, tokens=1500, nh=32, nkv=32, hd=128,
             dtype="f32", shape=33),
        # long documents
        dict(name="prompt_long_16384", op="prompt", seqs=2, tokens=16384, nh=32, nkv=8, hd=128,
             dtype="bf16", shape=35),
        # one user, one token at a time
        dict(name="decode_one_1500", op="paged", requests=1, ctx_max=1500, ctx_min=1500, chunk_max=1,
             chunks=0, nh=32, nkv=8, hd=128, dtype="bf16", block=16, shape=41),
        # a full decode batch of ragged contexts
        dict(name="decode_batch_64", op="paged", requests=64, ctx_max=16384, ctx_min=100,
             chunk_max=1, chunks=0, nh=32, nkv=8, hd=128, dtype="bf16", block=16, shape=42),
        # fp32 cache, as many key/value heads as query heads
        dict(name="decode_f32_12", op="paged", requests=12, ctx_max=4001, ctx_min=1, chunk_max=1,
             chunks=0, nh=32, nkv=32, hd=128, dtype="f32", block=32, shape=43),
        # chunked prefill beside decoding requests
        dict(name="chunk_mixed_20", op="paged", requests=20, ctx_max=32768, ctx_min=64,
             chunk_max=2048, chunks=4, nh=32, nkv=8, hd=128, dtype="bf16", block=64, shape=45),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(("plan", "append", "prompt", "prompt", "paged", "paged", "paged"))
    shape = rng.randrange(1 << 30)
    if op == "plan":
        R = _log(rng, 1, 4096)
        new_max = rng.choice((1, _log(rng, 2, 300)))
        return dict(op=op, requests=R, ctx_max=_log(rng, 1, 32768 if R <= 512 else 4096),
                    new_max=new_max, block=rng.choice((16, 32, 64, 128)),
                    pad=rng.choice((0, _log(rng, 1, 100))), shape=shape)
    nh, nkv, hd = rng.choice(SHAPES)
    block = rng.choice((16, 32, 64, 128))
    if op == "append":
        x = rng.choice(("f32", "bf16"))
        cap = max(1, int(8e7) // ((nh + 2 * nkv) * hd))
        return dict(op=op, tokens=_log(rng, 1, min(16384, cap)), nh=nh, nkv=nkv, hd=hd, x=x,
                    cache=rng.choice(("bf16", "bf16", "f32")), block=block,
                    keep=rng.choice((False, True)), pad=rng.choice((0, 0, 5)), shape=shape)
    f32 = rng.random() < 0.25
    dtype = "f32" if f32 else "bf16"
    cap = MAX_FLOPS / 10 if f32 else MAX_FLOPS
    while True:
        if op == "prompt":
            case = dict(op=op, seqs=_log(rng, 1, 16), tokens=0, nh=nh, nkv=nkv, hd=hd, dtype=dtype,
                        shape=shape)
            case["tokens"] = _log(rng, case["seqs"], 16384)
        else:
            R = _log(rng, 1, 128)
            chunks = rng.choice((0, 0, _log(rng, 1, 8)))
            case = dict(op=op, requests=R, ctx_max=_log(rng, 1, 32768), ctx_min=1,
                        chunk_max=_log(rng, 2, 2048) if chunks else 1, chunks=min(chunks, R), nh=nh,
                        nkv=nkv, hd=hd, dtype=dtype, block=block, shape=shape)
        w = work(case)
        if w["flops"] <= cap and w["bytes"] <= MAX_BYTES:
            return case


# ------------------------------------------------------------------ lengths

def _plan_lengths(case):
    """(context, new) lengths of the requests: a quarter of them new (context
    0); with more than one new token at most, some requests sit a step out."""
    r = random.Random(case["shape"])
    ctx, new = [], []
    for _ in range(case["requests"]):
        prompt = case["new_max"] > 1
        ctx.append(0 if prompt and r.random() < 0.25 else _log(r, 1, case["ctx_max"]))
        new.append(r.choice((0, 1, _log(r, 1, case["new_max"]))) if prompt else 1)
    return ctx, new


def _prompt_lengths(case):
    r = random.Random(case["shape"])
    n, total = case["seqs"], case["tokens"]
    w = [math.exp(r.uniform(0, 2.5)) for _ in range(n)]
    lens = [1 + int((total - n) * x / sum(w)) for x in w]
    lens[0] += total - sum(lens)
    return lens


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


def work(case):
    op = case["op"]
    if op == "plan":
        ctx, new = _plan_lengths(case)
        T, R, S = sum(new), len(ctx), case["block"]
        touched = sum(_blocks(c + n, S) - c // S for c, n in zip(ctx, new) if n)
        added = sum(_blocks(c + n, S) - _blocks(c, S) for c, n in zip(ctx, new))
        return {"bytes": 8 * R + 4 * touched + 4 * added + 12 * (T + case["pad"]) + 4 * (2 * R + 2),
                "flops": 2 * T + 4 * R}
    nh, nkv, hd = case["nh"], case["nkv"], case["hd"]
    if op == "append":
        T = case["tokens"]
        bi, bo = (4 if case["x"] == "f32" else 2), (4 if case["cache"] == "f32" else 2)
        row = (nh + 2 * nkv) * hd
        kept = 2 * nkv * hd * bo if case["keep"] else 0
        return {"bytes": T * (row * (bi + bo) + kept + hd * 4 + 12), "flops": T * (nh + nkv) * hd * 3}
    b = 4 if case["dtype"] == "f32" else 2
    if op == "prompt":
        lens = _prompt_lengths(case)
        pairs = sum(n * (n + 1) // 2 for n in lens)
        return {"bytes": sum(lens) * (2 * nh + 2 * nkv) * hd * b, "flops": 4 * hd * nh * pairs}
    lens = _paged_lengths(case)
    pairs = sum(n * (L - n) + n * (n + 1) // 2 for L, n in lens)
    return {"bytes": sum(2 * nkv * L * hd * b + 2 * n * nh * hd * b + 4 * _blocks(L, case["block"])
                         for L, n in lens), "flops": 4 * hd * nh * pairs}


# ------------------------------------------------------------------ inputs

def _dtype(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def _normal(gen, shape, dtype, scale=1.0):
    # written straight in the type it is kept in: no fp32 copy of a large cache
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


def _inputs(case, seed):
    """The tensors a program has before the call, from the seed."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rng = np.random.default_rng(seed)
    op = case["op"]
    s = dict(case)
    if op == "plan":
        ctx, new = _plan_lengths(case)
        S = case["block"]
        have = np.array([_blocks(c, S) for c in ctx])
        need = np.array([_blocks(c + n, S) for c, n in zip(ctx, new)])
        pool = int(need.sum()) + 16
        perm = rng.permutation(pool).astype(np.int32)
        table = np.full((len(ctx), int(need.max()) + 3), -1, dtype=np.int32)
        used = 0
        for r, h in enumerate(have):
            table[r, :h] = perm[used:used + h]
            used += h
        s.update(ctx_lens=_i32(ctx), new_lens=_i32(new), block_table=torch.from_numpy(table).cuda(),
                 free_blocks=torch.from_numpy(perm[used:].copy()).cuda(),
                 total=sum(new) + case["pad"])
        return s
    nh, nkv, hd = case["nh"], case["nkv"], case["hd"]
    if op == "append":
        T, S, pad = case["tokens"], case["block"], case["pad"]
        # runs of one to a thousand consecutive positions, as prompts and single
        # tokens give; padding rows at the end have neither position nor slot
        pos, slot, n = np.empty(T, np.int32), np.empty(T, np.int64), 0
        lens, runs = [], random.Random(case["shape"])
        while n < T:
            L = min(T - n, runs.choice((1, 1, 7, 200, 1000)))
            lens.append((n, L, runs.randrange(6000)))
            n += L
        blocks = sum(_blocks(L + p % S, S) for _, L, p in lens) + 8
        perm, b = rng.permutation(blocks), 0
        for n, L, p in lens:
            own_blocks = perm[b:b + _blocks(L + p % S, S)]
            b += len(own_blocks)
            j = p % S + np.arange(L)
            pos[n:n + L] = p + np.arange(L)
            slot[n:n + L] = own_blocks[j // S] * S + j % S
        pos = np.concatenate([pos, np.full(pad, -1, np.int32)])
        slot = np.concatenate([slot, np.full(pad, -1, np.int64)])
        cos, sin = _rotary_tables(8192, hd)
        shape = (blocks, nkv, S, hd)
        s.update(qkv=_normal(gen, (T + pad, (nh + 2 * nkv) * hd), _dtype(case["x"])),
                 positions=torch.from_numpy(pos).cuda(), slots=torch.from_numpy(slot).cuda(),
                 cos=cos, sin=sin, k_cache=torch.zeros(shape, dtype=_dtype(case["cache"]), device="cuda"),
                 v_cache=torch.zeros(shape, dtype=_dtype(case["cache"]), device="cuda"))
        return s
    dt = _dtype(case["dtype"])
    if op == "prompt":
        lens = _prompt_lengths(case)
        T = sum(lens)
        s.update(lens=lens, cu=_prefix(lens), q=_normal(gen, (T, nh, hd), dt, 2.0),
                 k=_normal(gen, (T, nkv, hd), dt), v=_normal(gen, (T, nkv, hd), dt))
        return s
    lens = _paged_lengths(case)
    S = case["block"]
    need = [_blocks(L, S) for L, _ in lens]
    pool = sum(need) + 16
    perm = rng.permutation(pool).astype(np.int32)
    table = np.full((len(lens), max(need) + 2), -1, dtype=np.int32)
    used = 0
    for r, n in enumerate(need):
        table[r, :n] = perm[used:used + n]
        used += n
    T = sum(n for _, n in lens)
    shape = (pool, nkv, S, hd)
    s.update(lens=lens, cu=_prefix([n for _, n in lens]), kv_lens=_i32([L for L, _ in lens]),
             block_table=torch.from_numpy(table).cuda(), q=_normal(gen, (T, nh, hd), dt, 2.0),
             k_cache=_normal(gen, shape, dt), v_cache=_normal(gen, shape, dt))
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        import group_quantized_moe_gb300 as lib

        s["lib"] = lib
        if "k_cache" in s:
            s["cache"] = lib.PagedKV(s["k_cache"], s["v_cache"])
        # a program keeps one workspace for all of its calls
        if s["op"] == "prompt":
            n = lib.qmm_attn_prompt_workspace_bytes(s["q"], s["k"], s["seqs"])
        elif s["op"] == "paged":
            n = lib.qmm_attn_paged_workspace_bytes(s["q"], s["cache"], s["requests"])
        else:
            n = 0
        s["workspace"] = torch.empty((n,), dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    return (_run_own if own else _run_plain)[s["op"]](s)


def _own_plan(s):
    p = s["lib"].kv_plan(s["ctx_lens"], s["new_lens"], s["block_table"], s["free_blocks"],
                         s["block"], s["total"])
    return {"table": s["block_table"], "cu": p.cu_new, "kv_lens": p.kv_lens,
            "positions": p.positions, "slots": p.slots, "used": p.blocks_used}


def _own_append(s):
    q, k, v = s["lib"].rope_append(s["qkv"], s["nh"], s["positions"], s["slots"], s["cos"], s["sin"],
                                   s["cache"], keep_kv=s["keep"])
    out = {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if s["keep"]:
        out.update(k=k, v=v)
    return out


def _own_prompt(s):
    return s["lib"].attn_prompt(s["q"], s["k"], s["v"], s["cu"], y_dtype=s["q"].dtype,
                                workspace=s["workspace"])


def _own_paged(s):
    return s["lib"].attn_paged(s["q"], s["cache"], s["block_table"], s["cu"], s["kv_lens"],
                               y_dtype=s["q"].dtype, workspace=s["workspace"])


_run_own = {"plan": _own_plan, "append": _own_append, "prompt": _own_prompt, "paged": _own_paged}


def _plain_plan(s):
    ctx, new, table, S = s["ctx_lens"], s["new_lens"], s["block_table"], s["block"]
    dev, total = table.device, s["total"]
    have = (ctx + S - 1) // S
    need = (ctx + new + S - 1) // S
    upto = torch.cumsum(need - have, 0)
    first = upto - (need - have)
    col = torch.arange(table.shape[1], device=dev)[None, :]
    at = (first[:, None] + col - have[:, None]).clamp(0, s["free_blocks"].numel() - 1)
    table = torch.where((col >= have[:, None]) & (col < need[:, None]), s["free_blocks"][at], table)
    cu = torch.cat([torch.zeros(1, dtype=torch.int64, device=dev), torch.cumsum(new, 0)])
    t = torch.arange(total, device=dev)
    r = torch.searchsorted(cu[1:], t, right=True)
    real = r < ctx.numel()
    r = r.clamp(max=ctx.numel() - 1)
    pos = ctx[r] + t - cu[r]
    slot = table[r, (pos // S).clamp(max=table.shape[1] - 1)].long() * S + pos % S
    return {"table": table, "cu": cu.int(), "kv_lens": ctx + new,
            "positions": torch.where(real, pos, -1).int(), "slots": torch.where(real, slot, -1),
            "used": upto[-1:].int()}


def _plain_append(s):
    nh, nkv, hd, S = s["nh"], s["nkv"], s["hd"], s["block"]
    x = s["qkv"].float().view(-1, nh + 2 * nkv, hd)
    pos, slot = s["positions"].long(), s["slots"]
    c, n = s["cos"][pos.clamp(min=0)][:, None, :], s["sin"][pos.clamp(min=0)][:, None, :]
    a, b = x[:, :nh + nkv, 0::2], x[:, :nh + nkv, 1::2]
    rot = torch.stack([a * c - b * n, a * n + b * c], dim=-1).flatten(2)
    out = torch.cat([rot, x[:, nh + nkv:]], dim=1).to(s["k_cache"].dtype)
    if s["pad"]:
        out[pos < 0] = 0
    q, k, v = out[:, :nh].contiguous(), out[:, nh:nh + nkv], out[:, nh + nkv:]
    T = s["tokens"]  # the rows that are not padding
    block, row = slot[:T] // S, slot[:T] % S
    s["k_cache"][block, :, row] = k[:T]
    s["v_cache"][block, :, row] = v[:T]
    res = {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if s["keep"]:
        res.update(k=k.contiguous(), v=v.contiguous())
    return res


def _plain_attention(q, k, v, scale):
    """q [n, nh, hd] over k, v [L, nkv, hd], query i sees keys 0 .. L - n + i;
    one key/value head at a time, so that the scores fit."""
    n, nh, hd = q.shape
    L, nkv = k.shape[0], k.shape[1]
    g = nh // nkv
    hidden = (torch.arange(L, device=q.device)[None, :]
              > torch.arange(L - n, L, device=q.device)[:, None])
    out = torch.empty((n, nh, hd), dtype=torch.float32, device=q.device)
    step = max(1, (1 << 30) // max(1, n * g * L))  # key/value heads at once
    for h in range(0, nkv, step):
        e = min(nkv, h + step)
        qh = q[:, h * g:e * g].float().reshape(n, e - h, g, hd).permute(1, 2, 0, 3)
        kh = k[:, h:e].float().permute(1, 2, 0)[:, None]
        vh = v[:, h:e].float().permute(1, 0, 2)[:, None]
        sc = torch.matmul(qh, kh) * scale
        if n > 1:
            sc = sc.masked_fill(hidden, -math.inf)
        p = torch.exp(sc - sc.amax(-1, keepdim=True))
        o = torch.matmul(p, vh) / p.sum(-1, keepdim=True)
        out[:, h * g:e * g] = o.permute(2, 0, 1, 3).reshape(n, (e - h) * g, hd)
    return out


def _plain_prompt(s):
    outs, t = [], 0
    for n in s["lens"]:
        outs.append(_plain_attention(s["q"][t:t + n], s["k"][t:t + n], s["v"][t:t + n],
                                     1.0 / math.sqrt(s["hd"])))
        t += n
    return torch.cat(outs).to(s["q"].dtype)


def _plain_paged(s):
    outs, t = [], 0
    nkv, hd, S = s["nkv"], s["hd"], s["block"]
    for r, (L, n) in enumerate(s["lens"]):
        ids = s["block_table"][r, :_blocks(L, S)].long()
        k = s["k_cache"][ids].transpose(1, 2).reshape(-1, nkv, hd)[:L]
        v = s["v_cache"][ids].transpose(1, 2).reshape(-1, nkv, hd)[:L]
        outs.append(_plain_attention(s["q"][t:t + n], k, v, 1.0 / math.sqrt(hd)))
        t += n
    return torch.cat(outs).to(s["q"].dtype)


_run_plain = {"plan": _plain_plan, "append": _plain_append, "prompt": _plain_prompt,
              "paged": _plain_paged}


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    """The outputs from the definitions, numbers in 64 bits."""
    s = _inputs(case, seed)
    op = case["op"]
    if op == "plan":
        return _exact_plan(s)
    if op == "append":
        return _exact_append(s)
    S = case.get("block")
    out, t = [], 0
    for r, item in enumerate(s["lens"]):
        L, n = item if op == "paged" else (item, item)
        if op == "paged":
            # key j lies in row j mod S of page table[r, j div S]
            j = torch.arange(L, device="cuda")
            page = s["block_table"][r][j // S].long()
            k, v = s["k_cache"][page, :, j % S].double(), s["v_cache"][page, :, j % S].double()
        else:
            k, v = s["k"][t:t + n].double(), s["v"][t:t + n].double()
        out.append(_exact_rows(s["q"][t:t + n].double(), k, v))
        t += n
    return torch.cat(out)


def _exact_rows(q, k, v):
    n, nh, hd = q.shape
    L, nkv = k.shape[:2]
    y = torch.zeros_like(q)
    for h in range(nh):
        kh, vh = k[:, h * nkv // nh], v[:, h * nkv // nh]
        for i0 in range(0, n, 2048):
            i1 = min(n, i0 + 2048)
            seen = L - n + i1  # no row of this block sees a later key
            logit = q[i0:i1, h] @ kh[:seen].T / hd ** 0.5
            last = torch.arange(L - n + i0, L - n + i1, device=q.device)
            late = torch.arange(seen, device=q.device) > last[:, None]
            logit[late] = float("-inf")
            y[i0:i1, h] = torch.exp(logit - torch.logsumexp(logit, 1, keepdim=True)) @ vh[:seen]
    return y


def _exact_plan(s):
    S, ctx, new = s["block"], s["ctx_lens"].tolist(), s["new_lens"].tolist()
    table, free = s["block_table"].cpu().numpy().copy(), s["free_blocks"].tolist()
    pos, slot, cu, used = [], [], [0], 0
    for r, (c, n) in enumerate(zip(ctx, new)):
        for b in range(_blocks(c, S), _blocks(c + n, S)):
            table[r, b] = free[used]
            used += 1
        p = np.arange(c, c + n)
        pos.append(p)
        slot.append(table[r, p // S].astype(np.int64) * S + p % S)
        cu.append(cu[-1] + n)
    fill = np.full(s["total"] - cu[-1], -1)
    return {"table": torch.from_numpy(table).cuda(), "cu": _i32(cu),
            "kv_lens": _i32([c + n for c, n in zip(ctx, new)]),
            "positions": _i32(np.concatenate(pos + [fill]).astype(np.int32)),
            "slots": torch.from_numpy(np.concatenate(slot + [fill]).astype(np.int64)).cuda(),
            "used": _i32([used])}


def _exact_append(s):
    nh, nkv, hd, S, T = s["nh"], s["nkv"], s["hd"], s["block"], s["tokens"]
    x = s["qkv"].double().reshape(-1, nh + 2 * nkv, hd // 2, 2)
    at = s["positions"].long().clamp(min=0)
    turn = torch.complex(s["cos"][at].double(), s["sin"][at].double())
    z = torch.view_as_complex(x) * turn[:, None]
    x = torch.cat([torch.view_as_real(z)[:, :nh + nkv], x[:, nh + nkv:]], 1).flatten(2)
    x[s["positions"] < 0] = 0.0
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    for cache, rows in ((kc, x[:T, nh:nh + nkv]), (vc, x[:T, nh + nkv:])):
        flat = cache.transpose(1, 2).reshape(-1, nkv, hd)
        flat[s["slots"][:T]] = rows
        cache.copy_(flat.reshape(-1, S, nkv, hd).transpose(1, 2))
    res = {"q": x[:, :nh], "k_cache": kc, "v_cache": vc}
    if s["keep"]:
        res.update(k=x[:, nh:nh + nkv], v=x[:, nh + nkv:])
    return res
