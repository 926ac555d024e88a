"""Timed cases of the paged 8-bit cache: page plan, append, attention.

Each case is one call of one operator, as a serving loop makes it:

  plan    block tables, slot map and positions of a step, from the requests'
          lengths and the stack of free blocks;
  append  rotary positions (one axis, or time / height / width), then keys and
          values into a paged cache held in 8 bits (e4m3) with a power-of-two
          scale for each block of tokens and KV head;
  attn    attention of packed query tokens over that cache: a token a sequence
          (decode), a few (a draft to verify) or a chunk; retrieval KV heads see
          the whole context, local ones the sinks and a sliding window.

`run` computes them in elementary torch operations, or (`own`) by this
package's entry points.  `exact` computes them again from their definitions in
64 bits.
"""

import math
import random

import numpy as np
import torch

own = False

FP8_MAX = 448.0        # largest e4m3 value
SCALE_MIN = 2.0 ** -64  # scale of a block that holds nothing larger
BASE = 10000.0

# The attention layer that the other workloads of this repository use, and the
# small fp32 one.
_LAYER = dict(hq=32, hkv=8, d=128, sink=64, window=2048, ret=0b100001, dtype="bf16")
_SMALL = dict(hq=4, hkv=2, d=64, sink=4, window=128, ret=0b01, dtype="fp32")


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one decode step of eight requests: the smallest plan, all latency
        dict(name="plan_step_b8", op="plan", b=8, bs=64, ctx_lo=8192, ctx_hi=32700, new_lo=1, new_hi=1,
             release=0, max_ctx=32768, pad=0, mix=1),
        # a step of continuous batching: 256 requests, some decode, some bring a
        # chunk of their prompt, some have ended; the token arrays are padded
        dict(name="plan_mixed_b256", op="plan", b=256, bs=16, ctx_lo=0, ctx_hi=30000, new_lo=1, new_hi=2048,
             release=24, max_ctx=32768, pad=1024, mix=2),
        # the append of one decode step: one token into each request's last block
        dict(name="append_step_b8", op="append", b=8, bs=64, ctx_lo=8192, ctx_hi=32700, new_lo=1, new_hi=1,
             axes=1, mix=3, **_LAYER),
        # the append of a multimodal prompt: three rotary axes, 8K tokens in all
        dict(name="append_prompt_8k_3axes", op="append", b=2, bs=64, ctx_lo=0, ctx_hi=100, new_lo=4096, new_hi=4096,
             axes=3, mix=4, **_LAYER),
        # a ragged append of a small fp32 layer, 16-token blocks
        dict(name="append_ragged_fp32", op="append", b=9, bs=16, ctx_lo=0, ctx_hi=333, new_lo=1, new_hi=517,
             axes=1, mix=5, **_SMALL),
        # the smallest decode step: a 2K context of the small fp32 layer
        dict(name="decode_2k_fp32", op="attn", b=1, bs=16, ctx_lo=2047, ctx_hi=2047, new_lo=1, new_hi=1,
             axes=1, mix=6, **_SMALL),
        # decode at 128K, one request
        dict(name="decode_128k", op="attn", b=1, bs=64, ctx_lo=131071, ctx_hi=131071, new_lo=1, new_hi=1,
             axes=1, mix=7, **_LAYER),
        # a decode batch of ragged contexts, three rotary axes
        dict(name="decode_ragged_b8_8k_32k", op="attn", b=8, bs=32, ctx_lo=8191, ctx_hi=32767, new_lo=1, new_hi=1,
             axes=3, mix=8, **_LAYER),
        # decode at 1M, one request: the longest stream
        dict(name="decode_1m", op="attn", b=1, bs=128, ctx_lo=1048575, ctx_hi=1048575, new_lo=1, new_hi=1,
             axes=1, mix=9, **{**_LAYER, "window": 4096}),
        # a draft of a few tokens to verify for each of eight requests
        dict(name="draft_b8_8k_32k", op="attn", b=8, bs=64, ctx_lo=8191, ctx_hi=32760, new_lo=2, new_hi=8,
             axes=1, mix=10, **_LAYER),
        # a mixed step: requests that decode beside requests that bring a chunk
        dict(name="chunk_mixed_b6", op="attn", b=6, bs=16, ctx_lo=0, ctx_hi=8192, new_lo=1, new_hi=1024,
             axes=1, mix=11, **_LAYER),
        # the last 2K chunk of a 32K prompt: the most arithmetic
        dict(name="chunk_2k_at_32k", op="attn", b=1, bs=64, ctx_lo=30720, ctx_hi=30720, new_lo=2048, new_hi=2048,
             axes=1, mix=12, **_LAYER),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _any_layer(rng):
    hkv, g = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 8])
    return dict(hq=hkv * g, hkv=hkv, d=rng.choice([64, 128]), sink=rng.choice([0, 4, 64, 100]),
                window=_log_int(rng, 1, 4096), ret=rng.randrange(1 << hkv), dtype=rng.choice(["bf16", "bf16", "bf16", "fp32"]))


def draw(rng):
    op = rng.choice(["plan", "append", "attn", "attn", "attn"])
    mix = rng.randrange(1 << 30)
    bs = rng.choice([16, 32, 64, 128])
    if op == "plan":
        max_ctx = _log_int(rng, 500, 40000)
        new = _log_int(rng, 1, min(2048, max_ctx // 2))
        b = _log_int(rng, 1, 300)
        return dict(op=op, b=b, bs=bs, ctx_lo=0, ctx_hi=max_ctx - new, new_lo=1, new_hi=new,
                    release=rng.randrange(0, b // 4 + 1), max_ctx=max_ctx, pad=rng.choice([0, 1, 77, 1024]), mix=mix)
    layer = _any_layer(rng)
    axes = rng.choice([1, 3])
    if op == "append":
        b = _log_int(rng, 1, 64)
        new = _log_int(rng, 1, max(1, 16384 // b))
        return dict(op=op, b=b, bs=bs, ctx_lo=0, ctx_hi=rng.choice([0, 100, 5000]), new_lo=min(new, rng.choice([1, new])),
                    new_hi=new, axes=axes, mix=mix, **layer)
    kind = rng.choice(["decode", "decode", "draft", "chunk"])
    b = _log_int(rng, 1, 16)
    if kind == "decode":
        ctx, new = _log_int(rng, 1, 400000 // b), 1
    elif kind == "draft":
        ctx, new = _log_int(rng, 16, 200000 // b), rng.randrange(2, 17)
    else:
        b = min(b, 6)
        new = _log_int(rng, 17, 2000 // b)
        ctx = _log_int(rng, 1, 30000 // b)
        layer["dtype"] = "bf16"  # chunks are a bf16 layer's
    return dict(op=op, b=b, bs=bs, ctx_lo=rng.choice([0, ctx // 2, ctx]), ctx_hi=ctx, new_lo=rng.choice([1, new]), new_hi=new,
                axes=axes, mix=mix, **layer)


def _lengths(case):
    """(cached tokens, new tokens) of each request; new = -1 releases it."""
    r = random.Random(case["mix"])
    ctx = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["b"])]
    # half of the requests of a mixed step decode one token
    new = [case["new_lo"] if r.random() < 0.5 else r.randint(case["new_lo"], case["new_hi"]) for _ in range(case["b"])]
    for k in range(case.get("release", 0)):
        new[(k * 7 + 3) % case["b"]] = -1
    return ctx, new


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _sections(case):
    """Rotary pairs of each axis, in order; their sum is d / 2."""
    h = case["d"] // 2
    return (h,) if case["axes"] == 1 else (h // 4, (h - h // 4) // 2, h - h // 4 - (h - h // 4) // 2)


def work(case):
    ctx, new = _lengths(case)
    add = [max(n, 0) for n in new]
    bs = case["bs"]
    if case["op"] == "plan":
        tokens = sum(add)
        blocks = sum(-(-(c + n) // bs) - -(-c // bs) for c, n in zip(ctx, add))
        gone = sum(-(-c // bs) for c, n in zip(ctx, new) if n < 0)
        # lengths in and out, blocks popped and pushed, slot (8) and position (4) of each token
        return {"bytes": 4 * (4 * case["b"] + 3) + 8 * (blocks + gone) + 12 * (tokens + case["pad"]), "flops": 0}
    hkv, d, g = case["hkv"], case["d"], case["hq"] // case["hkv"]
    es = 2 if case["dtype"] == "bf16" else 4
    tokens = sum(add)
    if case["op"] == "append":
        blocks = sum(-(-(c + n) // bs) - c // bs for c, n in zip(ctx, add))
        return {"bytes": tokens * (2 * hkv * d * (es + 1) + 8 + 4 * case["axes"]) + blocks * hkv * 8,
                "flops": tokens * hkv * d * 6}
    rows, pairs = 0, 0
    for c, n in zip(ctx, new):
        L = c + n
        for h in range(hkv):
            if case["ret"] >> h & 1:
                rows += L
                pairs += n * c + n * (n + 1) // 2
            else:
                lo = max(0, c + 1 - case["window"])  # the first row that the first query's window holds
                rows += L - lo + min(case["sink"], lo)
                seen = [min(case["window"], i + 1) + min(case["sink"], max(0, i + 1 - case["window"])) for i in (c, L - 1)]
                pairs += n * (seen[0] + seen[1]) // 2
    return {"bytes": rows * (2 * d + 8.0 / bs) + tokens * case["hq"] * d * 2 * es, "flops": 4 * d * g * pairs}


# ---------------------------------------------------------------------------
# what a program holds before the call
# ---------------------------------------------------------------------------
def _gen(seed, salt):
    return torch.Generator(device="cuda").manual_seed((seed * 1000003 + salt) & 0x7FFFFFFF)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _positions(case, ctx, new, gen):
    """[axes, tokens]: the token's index on the first axis; beside it, for a
    picture's tokens, a row and a column."""
    t = torch.cat([torch.arange(c, c + n) for c, n in zip(ctx, new)]).to("cuda", torch.int32)
    if case["axes"] == 1:
        return t[None].contiguous()
    side = torch.randint(0, 48, (2, t.numel()), generator=gen, device="cuda", dtype=torch.int32)
    picture = torch.rand(t.numel(), generator=gen, device="cuda") < 0.7
    return torch.stack([t, torch.where(picture, t - t % 48 + side[0], t), torch.where(picture, t - t % 48 + side[1], t)])


def _tables(case, lens, gen, spare=3):
    """A block table whose blocks lie anywhere in the pool, and the pool's size."""
    bs = case["bs"]
    n = [-(-x // bs) for x in lens]
    cols = max(1, max(n))
    pool = sum(n) + spare
    perm = torch.randperm(pool, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((case["b"], cols), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, k in enumerate(n):
        table[b, :k] = perm[at:at + k]
        at += k
    return table, pool, perm[at:].contiguous()


def _power_of_two_scale(amax):
    m, e = torch.frexp(amax / FP8_MAX)
    return torch.ldexp(torch.ones_like(amax), torch.where(m == 0.5, e - 1, e)).clamp_min(SCALE_MIN)


def _pool(case, n_blocks, gen):
    """A pool of blocks as appends leave them: normal values whose size varies
    from block to block, e4m3 with their power-of-two scales."""
    size = (n_blocks, case["hkv"], case["bs"], case["d"])
    out = []
    for _ in range(2):
        x = torch.randn(size, generator=gen, device="cuda", dtype=torch.float32)
        x *= torch.exp(0.5 * torch.randn(size[:2], generator=gen, device="cuda"))[..., None, None]
        s = _power_of_two_scale(x.abs().amax((2, 3)))
        out += [(x / s[..., None, None]).to(torch.float8_e4m3fn), s]
    return out[0], out[2], out[1].contiguous(), out[3].contiguous()


def prepare(case, seed):
    ctx, new = _lengths(case)
    add = [max(n, 0) for n in new]
    total = sum(add)
    gen = _gen(seed, 1)
    st = dict(case=case, tokens=total)
    if case["op"] == "plan":
        bs = case["bs"]
        need = sum(-(-(c + n) // bs) - -(-c // bs) for c, n in zip(ctx, add))
        held, pool, _ = _tables(case, ctx, gen, spare=need + 5)
        cols = -(-case["max_ctx"] // bs)
        table = torch.full((case["b"], cols), -1, dtype=torch.int32, device="cuda")
        table[:, :min(cols, held.shape[1])] = held[:, :cols]
        used = torch.zeros(pool, dtype=torch.bool, device="cuda")
        used[held[held >= 0].long()] = True
        free = torch.nonzero(~used).flatten().to(torch.int32)
        free = free[torch.randperm(free.numel(), generator=gen, device="cuda")]
        free_list = torch.zeros(pool, dtype=torch.int32, device="cuda")
        free_list[:free.numel()] = free
        m = total + case["pad"]
        st.update(ctx=_i32(ctx), new=_i32(new), table=table, free_list=free_list, n_free=_i32([free.numel()]),
                  seq_len=_i32([0] * case["b"]), cu=_i32([0] * (case["b"] + 1)), n_free_out=_i32([0]),
                  slots=torch.zeros(m, dtype=torch.int64, device="cuda"), pos=torch.zeros(m, dtype=torch.int32, device="cuda"),
                  status=_i32([0]))
        return st
    lens = [c + n for c, n in zip(ctx, new)]
    table, pool, _ = _tables(case, lens, gen)
    k8, v8, ks, vs = _pool(case, pool, gen)
    pos = _positions(case, ctx, new, gen)
    dt = _dtype(case)
    st.update(k8=k8, v8=v8, ks=ks, vs=vs, table=table, pos=pos, status=_i32([0]))
    if case["op"] == "append":
        t = torch.cat([torch.arange(c, c + n) for c, n in zip(ctx, new)]).cuda()
        b = torch.repeat_interleave(torch.arange(case["b"]), torch.tensor(new)).cuda()
        st["slots"] = table[b, t // case["bs"]].long() * case["bs"] + t % case["bs"]
        # keys and values as the fused projection leaves them: slices of one row a token
        qkv = torch.randn((total, (case["hq"] + 2 * case["hkv"]) * case["d"]), generator=gen, device="cuda").to(dt)
        q, kv = case["hq"] * case["d"], case["hkv"] * case["d"]
        st["k"] = qkv[:, q:q + kv].unflatten(1, (case["hkv"], case["d"]))
        st["v"] = qkv[:, q + kv:].unflatten(1, (case["hkv"], case["d"]))
        return st
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    st["q"] = (1.5 * torch.randn((total, case["hq"], case["d"]), generator=gen, device="cuda")).to(dt)
    st["out"] = torch.empty_like(st["q"])
    st.update(cu=_i32(cu), seq_len=_i32(lens), max_q=max(new), max_len=max(lens))
    return st


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
def _plain_plan(st):
    case = st["case"]
    bs = case["bs"]
    ctx, new, table = st["ctx"].long(), st["new"].long(), st["table"].long()
    gone, add = new < 0, new.clamp_min(0)
    have = (ctx + bs - 1) // bs
    col = torch.arange(table.shape[1], device="cuda")
    # blocks of ended requests go on top of the free stack, in order
    pushed = torch.where(gone, have, 0)
    base = st["n_free"].long() + pushed.cumsum(0) - pushed
    free = st["free_list"].long().clone()
    m = col < pushed[:, None]
    free[(base[:, None] + col)[m]] = table[m]
    top = st["n_free"].long() + pushed.sum()
    # requests take theirs from the top, in order, while they last
    need = torch.where(gone, 0, (ctx + add + bs - 1) // bs - have)
    before = need.cumsum(0) - need
    granted = ~gone & ((need == 0) | (before + need <= top))
    take = granted[:, None] & (col >= have[:, None]) & (col < (have + need)[:, None])
    table = torch.where(take, free[(top - 1 - before[:, None] - col + have[:, None]).clamp(0, free.numel() - 1)], table)
    seq_len = torch.where(gone, 0, ctx + add * granted)
    cu = torch.cat([add.new_zeros(1), add.cumsum(0)])
    t = torch.arange(st["slots"].numel(), device="cuda")
    b = torch.searchsorted(cu[1:], t, right=True).clamp_max(case["b"] - 1)
    live = t < cu[-1]
    at = torch.where(live, ctx[b] + t - cu[b], 0)
    slots = torch.where(live & granted[b], table[b, at // bs] * bs + at % bs, -1)
    i = torch.int32
    return dict(table=table.to(i), free_list=free.to(i), n_free=(top - (need * granted).sum()).to(i), seq_len=seq_len.to(i),
                cu=cu.to(i), slots=slots, pos=at.to(i))


def _angles(case, pos):
    """[tokens, d / 2] rotary angles in 64 bits."""
    h = case["d"] // 2
    axis = torch.repeat_interleave(torch.arange(case["axes"]), torch.tensor(_sections(case))).cuda()
    inv = BASE ** (-2.0 * torch.arange(h, device="cuda", dtype=torch.float64) / case["d"])
    return pos[axis].T.double() * inv


def _rotate(x, c, s):
    a, b = x.chunk(2, -1)
    return torch.cat([a * c - b * s, b * c + a * s], -1)


def _to_fp8(x):
    """The nearest e4m3 value (ties to even) of 64-bit x, |x| <= 448."""
    _, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), (e - 1).clamp_min(-6) - 3)
    return (torch.round(x / step) * step).float().to(torch.float8_e4m3fn)


def _plain_store(x, bad_value, ok, pool, scale, blk, off, bs):
    """The pool and its scales after rows x [tokens, heads, d] (64 bits; rows
    that are not `ok` hold bad_value and do not count) went to slots blk, off."""
    nb, hkv = scale.shape
    touched = torch.zeros(nb, dtype=torch.bool, device="cuda")
    touched[blk] = True
    first = torch.full((nb,), bs, dtype=torch.long, device="cuda").scatter_reduce(0, blk, off, "amin")
    amax = torch.zeros((nb, hkv), dtype=torch.float64, device="cuda")
    amax = amax.scatter_reduce(0, blk[:, None].expand(-1, hkv), torch.where(ok, x.abs().amax(-1), 0.0), "amax")
    old = torch.where((first > 0)[:, None], scale.double(), 0.0)
    new = torch.where(touched[:, None], torch.maximum(_power_of_two_scale(amax), old), scale.double())
    grown = touched[:, None] & (old > 0) & (new > old)
    row = torch.arange(bs, device="cuda") < first[:, None]
    again = (grown[:, :, None] & row[:, None, :])[..., None]
    vals = pool.double()
    out = torch.where(again, _to_fp8(vals * (scale.double() / new)[..., None, None]).float(), vals.float()).to(pool.dtype)
    out[blk, :, off] = torch.where(ok[..., None], _to_fp8(torch.where(ok[..., None], x, 0.0) / new[blk][..., None]).float(), bad_value).to(pool.dtype)
    return out, new.float()


def _plain_append(st):
    case = st["case"]
    th = _angles(case, st["pos"])[:, None]
    k = _rotate(st["k"].double(), th.cos(), th.sin())
    v = st["v"].double()
    ok = torch.isfinite(k).all(-1) & torch.isfinite(v).all(-1)
    live = st["slots"] >= 0
    s, k, v, ok = st["slots"][live], k[live], v[live], ok[live]
    blk, off = s // case["bs"], s % case["bs"]
    k8, ks = _plain_store(k, math.nan, ok, st["k8"], st["ks"], blk, off, case["bs"])
    v8, vs = _plain_store(v, 0.0, ok, st["v8"], st["vs"], blk, off, case["bs"])
    return dict(k8=k8, v8=v8, ks=ks, vs=vs)


def _plain_attn(st):
    case = st["case"]
    hq, hkv, d, bs, B = case["hq"], case["hkv"], case["d"], case["bs"], case["b"]
    g = hq // hkv
    # queries, padded to [B, hkv, g, T, d]
    cu, lens = st["cu"].long(), st["seq_len"].long()
    n = cu[1:] - cu[:-1]
    T, L = st["max_q"], st["table"].shape[1] * bs
    t = torch.arange(T, device="cuda")
    there = t < n[:, None]
    src = torch.where(there, cu[:-1, None] + t, 0)
    th = _angles(case, st["pos"])[:, None]
    q = _rotate(st["q"].float(), th.cos().float(), th.sin().float())
    q = q[src].unflatten(2, (hkv, g)).permute(0, 2, 3, 1, 4)
    # the context's rows, [B, hkv, L, d]
    tab = st["table"].long().clamp_min(0)

    def rows(pool, scale):
        x = pool[tab].float() * scale[tab][..., None, None]
        return x.transpose(1, 2).reshape(B, hkv, L, d)

    at = lens[:, None] - n[:, None] + t                    # [B, T] position of each query
    j = torch.arange(L, device="cuda")
    causal = (j <= at[..., None]) & there[..., None]        # [B, T, L]
    near = causal & ((j < case["sink"]) | (j > at[..., None] - case["window"]))
    ret = torch.tensor([bool(case["ret"] >> h & 1) for h in range(hkv)], device="cuda")
    s = (q.flatten(2, 3) @ rows(st["k8"], st["ks"]).transpose(-1, -2)).unflatten(2, (g, T))
    s *= d ** -0.5
    s.masked_fill_(~torch.where(ret[:, None, None], causal[:, None], near[:, None])[:, :, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    s -= torch.where(m == -math.inf, 0.0, m)
    p = s.exp_()
    z = p.sum(-1, keepdim=True)
    v = torch.where((j < lens[:, None])[:, None, :, None], rows(st["v8"], st["vs"]), 0.0)
    o = (p.flatten(2, 3) @ v).unflatten(2, (g, T)) / torch.where(z == 0, 1.0, z)
    o = o.permute(0, 3, 1, 2, 4).flatten(2, 3)              # [B, T, hq, d]
    return dict(out=o[there].to(st["q"].dtype))


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------
def _handle(st):
    """What a program makes once for its layer and keeps: the configuration, the
    cache's description, the rotary axes and the scratch memory."""
    import head_wise_sparse_local_b200 as rtp
    case = st["case"]
    if case["op"] == "plan":
        cfg = rtp.make_cfg(case["b"], 32, 8, 128, case["max_ctx"], 64, 2048, 1.0, (0, 5))
        return dict(rtp=rtp, cfg=cfg)
    cfg = rtp.make_cfg(case["b"], case["hq"], case["hkv"], case["d"], st["table"].shape[1] * case["bs"], case["sink"], case["window"],
                       1.0, [h for h in range(case["hkv"]) if case["ret"] >> h & 1], case["dtype"], BASE)
    h = dict(rtp=rtp, cfg=cfg, cache=rtp.make_q8_cache(st["k8"], st["v8"], st["ks"], st["vs"], st["status"]),
             rope=rtp.make_rope(case["d"], _sections(case)) if case["axes"] > 1 else None)
    if case["op"] == "attn":
        n = rtp.rtp_attn_q8_workspace_bytes(cfg, case["bs"], st["tokens"], st["max_q"], st["max_len"])
        h["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    return h


def _own(st):
    if "handle" not in st:
        st["handle"] = _handle(st)
    h, case = st["handle"], st["case"]
    rtp = h["rtp"]
    if case["op"] == "plan":
        rtp.rtp_page_plan(h["cfg"], case["bs"], st["ctx"], st["new"], st["table"], st["free_list"], st["n_free"], st["seq_len"],
                          st["cu"], st["slots"], st["pos"], st["n_free_out"], st["status"])
        return dict(table=st["table"], free_list=st["free_list"], n_free=st["n_free_out"], seq_len=st["seq_len"], cu=st["cu"],
                    slots=st["slots"], pos=st["pos"])
    if case["op"] == "append":
        rtp.rtp_append_q8(h["cfg"], h["cache"], st["k"], st["v"], st["slots"], st["pos"], h["rope"])
        return dict(k8=st["k8"], v8=st["v8"], ks=st["ks"], vs=st["vs"])
    rtp.rtp_attn_q8(h["cfg"], h["cache"], st["q"], st["cu"], st["seq_len"], st["table"], st["pos"], st["out"], st["max_q"],
                    st["max_len"], h["rope"], h["ws"], h["ws"].numel())
    return dict(out=st["out"])


_PLAIN = {"plan": _plain_plan, "append": _plain_append, "attn": _plain_attn}


def run(state):
    if own:
        return _own(state)
    return _PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_plan(st):
    bs = st["case"]["bs"]
    ctx, new = st["ctx"].tolist(), st["new"].tolist()
    table, free, top = st["table"].cpu().numpy().copy(), st["free_list"].cpu().numpy().copy(), int(st["n_free"])
    for b, n in enumerate(new):
        if n < 0:
            k = -(-ctx[b] // bs)
            free[top:top + k] = table[b, :k]
            top += k
    at, cu, seq, ok = top, [0], [], []
    for b, n in enumerate(new):
        n = max(n, 0)
        cu.append(cu[-1] + n)
        have, want = -(-ctx[b] // bs), -(-(ctx[b] + n) // bs)
        fits = new[b] >= 0 and (want == have or at - (want - have) >= 0)
        if new[b] >= 0:
            if fits:
                for c in range(have, want):
                    table[b, c] = free[at - 1 - (c - have)]
                top -= want - have
            at -= want - have
        ok.append(fits)
        seq.append(0 if new[b] < 0 else ctx[b] + (n if fits else 0))
    slots, pos = np.full(st["slots"].numel(), -1, np.int64), np.zeros(st["pos"].numel(), np.int32)
    for b, n in enumerate(new):
        for i in range(max(n, 0)):
            p = ctx[b] + i
            pos[cu[b] + i] = p
            if ok[b]:
                slots[cu[b] + i] = int(table[b, p // bs]) * bs + p % bs
    i = np.int32
    return dict(table=table, free_list=free, n_free=np.array([top], i), seq_len=np.array(seq, i), cu=np.array(cu, i), slots=slots, pos=pos)


def _exact_angles(case, pos):
    """numpy: the angle of each token and rotary pair."""
    p = pos.double().cpu().numpy()
    out, k = np.empty((p.shape[1], case["d"] // 2)), 0
    for a, width in enumerate(_sections(case)):
        for _ in range(width):
            out[:, k] = p[a] * math.pow(BASE, -2.0 * k / case["d"])
            k += 1
    return torch.from_numpy(out).cuda()


def _exact_turn(x, th):
    h = x.shape[-1] // 2
    z = torch.complex(x[..., :h], x[..., h:]) * torch.polar(torch.ones_like(th), th)[:, None]
    return torch.cat([z.real, z.imag], -1)


def _exact_append(st):
    case = st["case"]
    bs = case["bs"]
    new = {"k": _exact_turn(st["k"].double(), _exact_angles(case, st["pos"])), "v": st["v"].double()}
    slots = st["slots"].cpu()
    # the e4m3 values, to round against: neighbours and the midpoints between them
    grid = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().cuda()
    mid = (grid[1:] + grid[:-1]) / 2

    def nearest(x):
        a = x.abs()
        up, down = torch.searchsorted(mid, a, right=True), torch.searchsorted(mid, a, right=False)
        return grid[torch.where(up % 2 == 0, up, down)] * torch.sign(x)

    out = {}
    for name in ("k", "v"):
        pool, scale = st[name + "8"].double(), st[name + "s"].double()
        for blk in slots[slots >= 0].div(bs, rounding_mode="floor").unique().tolist():
            tok = torch.nonzero((slots >= blk * bs) & (slots < (blk + 1) * bs)).flatten()
            off = slots[tok] - blk * bs
            x = new[name][tok.cuda()]                       # [rows, hkv, d]
            a = x.abs().amax((0, 2))
            s = torch.full_like(a, SCALE_MIN)
            s = torch.maximum(s, torch.exp2(torch.ceil(torch.log2(a / FP8_MAX).clamp_min(-64.0))))
            first = int(off.min())
            if first > 0:
                s = torch.maximum(s, scale[blk])
                pool[blk, :, :first] = nearest(pool[blk, :, :first] * (scale[blk] / s)[:, None, None])
            pool[blk, :, off.cuda()] = nearest(x / s[:, None]).transpose(0, 1)
            scale[blk] = s
        out[name + "8"], out[name + "s"] = pool, scale
    return out


def _exact_attn(st):
    case = st["case"]
    hkv, d, bs = case["hkv"], case["d"], case["bs"]
    q = _exact_turn(st["q"].double(), _exact_angles(case, st["pos"]))
    out = torch.zeros_like(q)
    cu, lens, table = st["cu"].tolist(), st["seq_len"].tolist(), st["table"].long()
    g = case["hq"] // hkv
    for b, L in enumerate(lens):
        if cu[b] == cu[b + 1]:
            continue
        blocks = table[b, :-(-L // bs)]
        i = torch.arange(L - (cu[b + 1] - cu[b]), L, device="cuda")
        j = torch.arange(L, device="cuda")
        for h in range(hkv):
            k = (st["k8"][blocks, h].double() * st["ks"][blocks, h].double()[:, None, None]).flatten(0, 1)[:L]
            v = (st["v8"][blocks, h].double() * st["vs"][blocks, h].double()[:, None, None]).flatten(0, 1)[:L]
            hide = j > i[:, None]
            if not case["ret"] >> h & 1:
                hide |= (j >= case["sink"]) & (j <= i[:, None] - case["window"])
            for e in range(g):
                s = torch.einsum("td,ld->tl", q[cu[b]:cu[b + 1], h * g + e], k) / math.sqrt(d)
                p = torch.softmax(s.masked_fill(hide, -math.inf), -1)
                out[cu[b]:cu[b + 1], h * g + e] = p @ v
    return dict(out=out)


def exact(case, seed):
    st = prepare(case, seed)
    return {"plan": _exact_plan, "append": _exact_append, "attn": _exact_attn}[case["op"]](st)
