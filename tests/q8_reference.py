"""The paged 8-bit cache in plain 64-bit arithmetic, written from its
definitions in include/rtp.h; the tests hold the kernels to it."""

from __future__ import annotations

import math

import numpy as np
import torch

SCALE_MIN = 2.0 ** -64
GRID = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()  # the values >= 0


def to_e4m3(x: torch.Tensor) -> torch.Tensor:
    """Nearest e4m3 value (ties to the even code) of |x| <= 448, by its distance to the grid."""
    g = GRID.to(x.device)
    a = x.abs()
    hi = torch.searchsorted(g, a).clamp_max(126)
    lo = (hi - 1).clamp_min(0)
    up, down = g[hi] - a, a - g[lo]
    take_hi = (up < down) | ((up == down) & (hi % 2 == 0))
    return torch.where(take_hi, g[hi], g[lo]) * torch.sign(x)


def block_scale(amax: float) -> float:
    s = SCALE_MIN
    while amax > 448.0 * s:
        s *= 2.0
    return s


def angles(pos, axis, D, base=10000.0) -> torch.Tensor:
    """[N, D/2] from pos [axes, N] and the pairs' axes."""
    p = pos.double().cpu()
    inv = torch.tensor([base ** (-2.0 * k / D) for k in range(D // 2)], dtype=torch.float64)
    return p[torch.as_tensor(axis)].T * inv


def rotate(x, th) -> torch.Tensor:
    """x [N, heads, D], rotate-half, 64 bits."""
    x = x.double().cpu()
    h = x.shape[-1] // 2
    c, s = torch.cos(th)[:, None], torch.sin(th)[:, None]
    return torch.cat([x[..., :h] * c - x[..., h:] * s, x[..., h:] * c + x[..., :h] * s], -1)


class Pool:
    """k, v as the values held [n_blocks, Hkv, bs, D] (before their scales), and the scales."""

    def __init__(self, n_blocks, hkv, bs, D):
        self.k = torch.zeros(n_blocks, hkv, bs, D, dtype=torch.float64)
        self.v = torch.zeros_like(self.k)
        self.ks = torch.ones(n_blocks, hkv, dtype=torch.float64)
        self.vs = torch.ones(n_blocks, hkv, dtype=torch.float64)
        self.bs = bs

    def append(self, k_rot, v, slots):
        """One call's tokens: k_rot (64 bits), v [N, Hkv, D]; slots, negative ones skipped."""
        v = v.double().cpu()
        ok = torch.isfinite(k_rot).all(-1) & torch.isfinite(v).all(-1)  # [N, Hkv]
        slots = [int(s) for s in slots]
        by_block = {}
        for t, s in enumerate(slots):
            if s >= 0:
                by_block.setdefault(s // self.bs, []).append((s % self.bs, t))
        for blk, rows in by_block.items():
            first = rows[0][0]
            toks = [t for _, t in rows]
            offs = [o for o, _ in rows]
            for x, val, sc, poison in ((k_rot, self.k, self.ks, math.nan), (v, self.v, self.vs, 0.0)):
                for h in range(x.shape[1]):
                    good = [t for t in toks if ok[t, h]]
                    s = block_scale(max([float(x[t, h].abs().max()) for t in good], default=0.0))
                    if first > 0:
                        old = float(sc[blk, h])
                        s = max(s, old)
                        if s > old:
                            val[blk, h, :first] = torch.where(torch.isnan(val[blk, h, :first]), math.nan,
                                                              to_e4m3(torch.nan_to_num(val[blk, h, :first]) * (old / s)))
                    sc[blk, h] = s
                    for o, t in zip(offs, toks):
                        val[blk, h, o] = to_e4m3(x[t, h] / s) if ok[t, h] else torch.full_like(x[t, h], poison)

    def rows(self, table_row, L, h):
        """(k, v) [L, D] of a request's first L positions for KV head h."""
        n = -(-L // self.bs)
        ids = torch.as_tensor([int(i) for i in table_row[:n]])
        k = (self.k[ids, h] * self.ks[ids, h][:, None, None]).flatten(0, 1)[:L]
        v = (self.v[ids, h] * self.vs[ids, h][:, None, None]).flatten(0, 1)[:L]
        return k, v


def visible(i, L, retrieval, S, W):
    """Boolean [L]: the positions that a query at position i sees."""
    j = torch.arange(L)
    m = j <= i
    return m if retrieval else m & ((j < S) | (j > i - W))


def attend(q_rot, k, v, seen):
    """One row: (out, sum p |v|, largest sum |q k| / sqrt(D)) over the seen positions."""
    if not bool(seen.any()):
        z = torch.zeros(v.shape[1], dtype=torch.float64)
        return z, z, 0.0
    k, v = k[seen], v[seen]
    D = q_rot.shape[0]
    s = k @ q_rot / math.sqrt(D)
    p = torch.softmax(s, 0)
    return p @ v, p @ v.abs(), float((k.abs() @ q_rot.abs()).max()) / math.sqrt(D)


def plan(ctx, new, table, free_list, n_free, bs, max_ctx, max_tokens):
    """(table, free_list, n_free, seq_len, cu, slots, positions, flags) after the call, plain loops."""
    table, free = table.copy(), free_list.copy()
    SEQ, POS, BLOCKS = 1, 2, 8
    flags, B, cap = 0, len(ctx), len(free)
    ctx, new = [int(c) for c in ctx], [int(n) for n in new]
    for b in range(B):
        if ctx[b] < 0 or ctx[b] > max_ctx:
            flags |= SEQ
            ctx[b], new[b] = 0, min(new[b], 0)
    top = int(n_free)
    for b in range(B):
        if new[b] < 0:
            for i in range(-(-ctx[b] // bs)):
                if top < cap:
                    free[top] = table[b, i]
                else:
                    flags |= BLOCKS
                top = top + 1
    top = min(top, cap)
    before, taken, cu = 0, 0, [0]
    seq = []
    slots = np.full(max_tokens, -1, np.int64)
    pos = np.zeros(max_tokens, np.int32)
    total = 0
    for b in range(B):
        n = max(new[b], 0)
        start = total
        total += n
        cu.append(min(total, max_tokens))
        if new[b] < 0:
            seq.append(0)
            continue
        have = -(-ctx[b] // bs)
        fits = ctx[b] + n <= max_ctx
        need = -(-(ctx[b] + n) // bs) - have if fits else 0
        ok = fits
        if not fits:
            flags |= POS
        if ok and n > 0 and start + n > max_tokens:
            ok = False
            flags |= POS
        if ok and need > 0 and before + need > top:
            ok = False
            flags |= BLOCKS
        if ok:
            for i in range(need):
                table[b, have + i] = free[top - 1 - before - i]
            taken += need
        before += need
        seq.append(ctx[b] + (n if ok else 0))
        for i in range(n):
            t = start + i
            if t >= max_tokens:
                break
            p = ctx[b] + i
            pos[t] = p
            if ok:
                blk = int(table[b, p // bs])
                if blk >= 0:
                    slots[t] = blk * bs + p % bs
                else:
                    flags |= BLOCKS
    if total > max_tokens:
        flags |= POS
    return table, free, top - taken, np.array(seq), np.array(cu), slots, pos, flags
