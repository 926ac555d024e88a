"""GPU parity of the paged 8-bit cache (rtp_page_plan, rtp_append_q8,
rtp_attn_q8) against tests/q8_reference.py, in 64 bits.

The plan and the stored cache are exact: every integer, every e4m3 value and
every scale has to be equal.

Attention's bound, for one output with exact value o = sum p v, A = sum p |v| and
Z = max_j sum_d |q_d k_jd| / sqrt(D):
  - the score's error e = Z (r_q + 2^-20): r_q the queries' rounding (2^-11 as
    one fp16 part, 2^-21 as two), 2^-20 for the fp32 rotation and the fp32
    accumulation of D products;
  - the weights: softmax with scores off by e moves o by at most A (exp(2 e) - 1);
  - the weights' rounding for the second product, A 2^-11 (fp16; 2^-21 as two
    parts), and fp32 accumulation, A 2^-23 per product step (L / 16 + 64 of them);
  - weights below fp16's smallest step, against the largest weight w of a value
    scaled by its block: L 2^-31 448 max_j (p_j vs_j) <= L 2^-22 max_j p_j max|v|;
  - the output's rounding, |o| eps / 2 (bf16 2^-8, fp32 2^-24).
Chunks (more than 32 query rows a KV head) form a quarter of their weights by a
cubic whose relative error is 7.5e-5 < 2^-13: A 2^-13, and twice that in e.
"""

import math
import random

import numpy as np
import pytest
import torch

import head_wise_sparse_local_b200 as rtp
import q8_reference as ref

pytestmark = pytest.mark.gpu

DEV = "cuda"
AXIS3 = {64: (8, 12, 12), 128: (16, 24, 24)}


def _i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def _axis(D, sections):
    return [a for a, s in enumerate(sections) for _ in range(s)]


def _gen(seed):
    return torch.Generator().manual_seed(seed)


# ---------------------------------------------------------------------------
# page plan
# ---------------------------------------------------------------------------
def _run_plan(ctx, new, table, free_list, n_free, bs, max_ctx, max_tokens, in_place=False):
    B = len(ctx)
    cfg = rtp.make_cfg(B, 4, 2, 64, max_ctx, 4, 128, 1.0, (0,))
    c, n = _i32(ctx), _i32(new)
    tab, free, nf = _i32(table), _i32(free_list), _i32([n_free])
    seq = c if in_place else torch.full((B,), -7, dtype=torch.int32, device=DEV)
    nf_out = nf if in_place else torch.full((1,), -7, dtype=torch.int32, device=DEV)
    cu = torch.full((B + 1,), -7, dtype=torch.int32, device=DEV)
    slots = torch.full((max_tokens,), -7, dtype=torch.int64, device=DEV)
    pos = torch.full((max_tokens,), -7, dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    rtp.rtp_page_plan(cfg, bs, c, n, tab, free, nf, seq, cu, slots, pos, nf_out, status)
    torch.cuda.synchronize()
    return tab, free, int(nf_out), seq, cu, slots, pos, int(status)


def _check_plan(ctx, new, table, free_list, n_free, bs, max_ctx, max_tokens, in_place=False):
    got = _run_plan(ctx, new, table, free_list, n_free, bs, max_ctx, max_tokens, in_place)
    want = ref.plan(ctx, new, np.asarray(table), np.asarray(free_list), n_free, bs, max_ctx, max_tokens)
    for name, g, w in zip(("table", "free list", "n_free", "seq_len", "cu", "slots", "positions", "status"), got, want):
        g = g.cpu().numpy() if isinstance(g, torch.Tensor) else g
        assert np.array_equal(g, w), name
    return got


def _requests(seed, B, bs, max_ctx, new_hi, ended=0.2, spare=0):
    """Random requests whose blocks lie anywhere, and a stack of the others."""
    r = random.Random(seed)
    cols = -(-max_ctx // bs)
    ctx = [r.randrange(0, max_ctx + 1) if r.random() < 0.9 else 0 for _ in range(B)]
    new = [-1 if r.random() < ended else min(max_ctx - c, r.randrange(0, new_hi + 1)) for c in ctx]
    held = [-(-c // bs) for c in ctx]
    need = sum(-(-(c + max(n, 0)) // bs) - h for c, n, h in zip(ctx, new, held))
    pool = sum(held) + need + spare
    ids = list(range(pool))
    r.shuffle(ids)
    table = np.full((B, cols), -1, np.int64)
    for b in range(B):
        for i in range(held[b]):
            table[b, i] = ids.pop()
    free = np.zeros(max(pool, 1), np.int64)
    free[:len(ids)] = ids
    return ctx, new, table, free, len(ids)


@pytest.mark.parametrize("B,bs,max_ctx,new_hi", [(1, 64, 100, 1), (8, 64, 5000, 1), (33, 16, 3000, 40), (257, 32, 2000, 300),
                                                 (1100, 128, 700, 3), (4096, 16, 200, 20)])
@pytest.mark.parametrize("in_place", [False, True])
def test_plan_matches_its_definition(B, bs, max_ctx, new_hi, in_place):
    ctx, new, table, free, n_free = _requests(B + new_hi, B, bs, max_ctx, new_hi, spare=3)
    total = sum(max(n, 0) for n in new)
    out = _check_plan(ctx, new, table, free, n_free, bs, max_ctx, total + 13, in_place)
    assert out[-1] == 0


def test_plan_long_chunks_and_unaligned_ends():
    """Several CTAs; token arrays whose size is no multiple of four."""
    ctx, new = [0, 17, 16, 40000, 5], [50001, 1, 0, 3, 30000]
    table = np.full((5, -(-90000 // 16)), -1, np.int64)
    table[1, :2], table[2, 0], table[4, 0] = (7, 9), 11, 3
    table[3, :2500] = np.arange(10000, 12500)
    free = np.arange(20000, 28000)
    for pad in (0, 1, 2, 3):
        _check_plan(ctx, new, table, free, 8000, 16, 90000, sum(new) + pad)


def test_plan_runs_out_of_blocks():
    ctx, new = [64, 0, 10, 63, 128], [65, 64, 1, 2, 0]  # need 2, 1, 0, 1, 0
    table = np.array([[5, -1, -1, -1], [-1] * 4, [6, -1, -1, -1], [7, -1, -1, -1], [8, 9, -1, -1]])
    for n_free in range(5):
        out = _check_plan(ctx, new, table, np.arange(20, 28), n_free, 64, 256, 140)
        assert (out[-1] == rtp.RTP_DEV_BLOCKS) == (n_free < 4)


def test_plan_reuses_blocks_that_ended_requests_give_back():
    ctx, new = [130, 0], [-1, 190]
    table = np.array([[3, 4, 5], [-1, -1, -1]])
    out = _check_plan(ctx, new, table, np.array([9, 0, 0, 0]), 1, 64, 192, 190)
    assert out[0][1].tolist() == [5, 4, 3] and out[2] == 1 and out[-1] == 0


def test_plan_refuses_what_does_not_fit():
    table = np.full((4, 4), -1, np.int64)
    table[:, 0] = (1, 2, 3, 4)
    # past max_ctx; past max_tokens (only the last request's tokens); a context that cannot be
    assert _check_plan([60, 10, 20, 30], [200, 1, 2, 3], table, np.arange(10, 20), 10, 64, 256, 206)[-1] == rtp.RTP_DEV_POSITION
    assert _check_plan([60, 10, 20, 30], [2, 1, 2, 3], table, np.arange(10, 20), 10, 64, 256, 6)[-1] == rtp.RTP_DEV_POSITION
    assert _check_plan([60, -1, 257, 30], [2, 1, 2, 3], table, np.arange(10, 20), 10, 64, 256, 8)[-1] == rtp.RTP_DEV_SEQ_LEN
    # a stack with no room for what comes back, and a table entry that names no block
    assert _check_plan([256, 60], [-1, 3], np.array([[1, 2, 3, 4], [9, -1, -1, -1]]), np.array([7, 7]), 1, 64, 256, 3)[-1] & rtp.RTP_DEV_BLOCKS
    assert _check_plan([60], [3], np.array([[-1, -1, -1, -1]]), np.array([7]), 1, 64, 256, 3)[-1] == rtp.RTP_DEV_BLOCKS


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------
class _Held:
    """A device pool and the reference pool side by side."""

    def __init__(self, n_blocks, hkv, bs, D, dtype, G=2, sections=None, B=4, max_ctx=4096, **kw):
        self.sections = sections
        self.D, self.hkv, self.bs, self.dtype = D, hkv, bs, dtype
        self.dt = torch.bfloat16 if dtype == "bf16" else torch.float32
        self.cfg = rtp.make_cfg(B, hkv * G, hkv, D, max_ctx, kw.get("S", 4), kw.get("W", 128), 1.0, kw.get("ret", (0,)), dtype)
        self.rope = rtp.make_rope(D, sections) if sections else None
        self.axis = _axis(D, sections) if sections else [0] * (D // 2)
        size = (n_blocks, hkv, bs, D)
        self.k = torch.zeros(size, dtype=torch.float8_e4m3fn, device=DEV)
        self.v = torch.zeros(size, dtype=torch.float8_e4m3fn, device=DEV)
        self.ks, self.vs = torch.ones(size[:2], device=DEV), torch.ones(size[:2], device=DEV)
        self.status = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.cache = rtp.make_q8_cache(self.k, self.v, self.ks, self.vs, self.status)
        self.pool = ref.Pool(n_blocks, hkv, bs, D)

    def positions(self, n, gen, hi=5000):
        return torch.randint(0, hi, (len(self.sections) if self.sections else 1, n), generator=gen, dtype=torch.int32)

    def append(self, k, v, slots, pos):
        slots = torch.as_tensor(slots, dtype=torch.int64)
        self.pool.append(ref.rotate(k.double(), ref.angles(pos, self.axis, self.D)), v, slots)
        rtp.rtp_append_q8(self.cfg, self.cache, k.to(DEV), v.to(DEV), slots.to(DEV), pos.to(DEV), self.rope)
        torch.cuda.synchronize()

    def check(self):
        for name, g, w in (("k", self.k, self.pool.k), ("v", self.v, self.pool.v), ("k_scale", self.ks, self.pool.ks),
                           ("v_scale", self.vs, self.pool.vs)):
            g = g.cpu().double()
            same = (g == w) | (torch.isnan(g) & torch.isnan(w))
            assert bool(same.all()), (name, torch.nonzero(~same)[:5].tolist(), int((~same).sum()))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bs", [16, 32, 64, 128])
@pytest.mark.parametrize("axes", [1, 3])
def test_append_chunks(dtype, D, bs, axes):
    """Ragged chunks of three requests, some starting inside a block, then a
    second call that goes on in the blocks of the first."""
    gen = _gen(bs + D)
    h = _Held(40, 3, bs, D, dtype, sections=AXIS3[D] if axes == 3 else None)
    free = torch.randperm(40, generator=gen).tolist()
    tables, ctx = [[], [], []], [0, 0, 0]
    for lens in ((bs + 5, 1, 2 * bs), (3, 2 * bs - 1, 1), (1, 1, 1)):
        slots = []
        for b, n in enumerate(lens):
            for p in range(ctx[b], ctx[b] + n):
                if p // bs == len(tables[b]):
                    tables[b].append(free.pop())
                slots.append(tables[b][p // bs] * bs + p % bs)
            ctx[b] += n
        N = len(slots)
        k = torch.randn(N, 3, D, generator=gen).to(h.dt)
        v = (torch.randn(N, 3, D, generator=gen) * 3).to(h.dt)
        h.append(k, v, slots, h.positions(N, gen))
        h.check()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_append_token_by_token_grows_the_scale(dtype):
    """Values that double from token to token: the block's earlier rows are
    rounded again at each step, down to e4m3's subnormals and zero."""
    gen = _gen(3)
    h = _Held(2, 2, 16, 64, dtype, B=1)
    for t in range(16):
        k = (torch.randn(1, 2, 64, generator=gen) * 2.0 ** (t - 4)).to(h.dt)
        v = (torch.randn(1, 2, 64, generator=gen) * 4.0 ** (7 - t)).to(h.dt)  # shrinks: the scale stays
        h.append(k, v, [16 + t], torch.tensor([[t]], dtype=torch.int32))
        h.check()


def test_append_rounds_ties_to_even_and_hits_scale_borders():
    """At position 0 the rotation is exact: every tie of the grid, and largest
    values on either side of 448 times a power of two."""
    g = ref.GRID
    mids = ((g[1:] + g[:-1]) / 2).float()
    for top in (448.0, 450.0, 224.0, 446.0, 1.75 * 2.0 ** -30, 2.0 ** -70, 0.0):
        h = _Held(1, 1, 16, 128, "fp32", G=1, B=1)
        k = torch.zeros(1, 1, 128)
        k[0, 0, :126] = mids * (1.0 if top >= 224 else top / 448.0)
        k[0, 0, 126] = top
        k[0, 0, 127] = -top
        k[0, 0, 125] = 0.0
        h.append(k, -k, [0], torch.zeros(1, 1, dtype=torch.int32))
        h.check()


def test_append_far_and_negative_positions():
    gen = _gen(8)
    h = _Held(2, 2, 32, 128, "bf16", sections=AXIS3[128])
    pos = torch.tensor([[0, 1, 2 ** 23 - 1, -5, 2 ** 31 - 1], [1048575, -2 ** 31, 7, 0, 1], [3, 524288, -1, 99999, 2 ** 30]],
                       dtype=torch.int32)
    h.append(torch.randn(5, 2, 128, generator=gen).bfloat16(), torch.randn(5, 2, 128, generator=gen).bfloat16(), range(32, 37), pos)
    h.check()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_append_values_that_are_not_finite(dtype):
    """Such a row is stored as NaN keys and zero values and leaves the scale alone."""
    gen = _gen(4)
    h = _Held(3, 2, 16, 64, dtype)
    k, v = torch.randn(20, 2, 64, generator=gen), torch.randn(20, 2, 64, generator=gen)
    k[3, 0, 5], k[4, 1, 63], v[5, 0, 0], v[6, 1, 33], k[19, 0, 0] = math.nan, math.inf, -math.inf, math.nan, math.inf
    k[7, 0, :] = math.nan
    pos = h.positions(20, gen)
    h.append(k.to(h.dt), v.to(h.dt), list(range(20)), pos)
    h.check()
    # a block whose only new row is bad keeps its scale; a fresh one takes the least
    bad = torch.full((2, 2, 64), math.nan)
    h.append(bad.to(h.dt), bad.to(h.dt), [20, 32], h.positions(2, gen))
    h.check()
    assert float(h.ks[2, 0]) == ref.SCALE_MIN


def test_append_skips_rows_without_a_slot():
    gen = _gen(5)
    h = _Held(4, 2, 16, 64, "bf16")
    slots = [-1, 5, 6, -1, -1, 30, 31, 32, -1]
    n = len(slots)
    h.append(torch.randn(n, 2, 64, generator=gen).bfloat16(), torch.randn(n, 2, 64, generator=gen).bfloat16(), slots, h.positions(n, gen))
    h.check()
    before = h.k.clone().view(torch.uint8)
    k = torch.randn(3, 2, 64, generator=gen).bfloat16().to(DEV)
    rtp.rtp_append_q8(h.cfg, h.cache, k, k, torch.tensor([64, 1 << 40, -3], device=DEV), h.positions(3, gen).to(DEV))
    torch.cuda.synchronize()
    assert int(h.status) == rtp.RTP_DEV_BLOCKS and torch.equal(before, h.k.view(torch.uint8))


def test_append_slices_of_the_fused_projection():
    gen = _gen(6)
    h = _Held(6, 2, 32, 64, "bf16", G=2)
    qkv = torch.randn(70, (4 + 2 + 2) * 64, generator=gen).bfloat16().to(DEV)
    k, v = qkv[:, 256:384].unflatten(1, (2, 64)), qkv[:, 384:].unflatten(1, (2, 64))
    pos = h.positions(70, gen)
    slots = torch.arange(40, 110)
    h.pool.append(ref.rotate(k.cpu().double(), ref.angles(pos, h.axis, 64)), v.cpu(), slots)
    rtp.rtp_append_q8(h.cfg, h.cache, k, v, slots.to(DEV), pos.to(DEV))
    torch.cuda.synchronize()
    h.check()


@pytest.mark.parametrize("dtype,D,hkv,bs,B,runs", [
    ("bf16", 128, 1, 64, 4, [1, 1, 1, 1]),           # one head, a token each: a CTA of one warp
    ("fp32", 128, 1, 16, 3, [1, 2, 1]),
    ("bf16", 64, 2, 128, 200, [200]),                 # as many tokens as requests, but one brings them all
    ("bf16", 128, 2, 64, 300, [200]),
    ("fp32", 64, 3, 32, 60, [1] * 59 + [400]),
    ("bf16", 128, 8, 16, 16, [4] * 16),
    ("bf16", 64, 64, 16, 2, [1, 1]),
])
def test_append_steps_of_any_shape(dtype, D, hkv, bs, B, runs):
    gen = _gen(len(runs) + D)
    blocks = [-(-(3 + n) // bs) for n in runs]  # every run starts at a block's row 3
    h = _Held(sum(blocks), hkv, bs, D, dtype, G=1, B=B)
    first = np.concatenate([[0], np.cumsum(blocks)])
    slots = [int(first[i]) * bs + 3 + t for i, n in enumerate(runs) for t in range(n)]
    N = len(slots)
    assert N <= 8 * B
    for scale in (1.0, 30.0):  # the second call writes over the first and grows the scales
        h.append((torch.randn(N, hkv, D, generator=gen) * scale).to(h.dt), torch.randn(N, hkv, D, generator=gen).to(h.dt), slots,
                 h.positions(N, gen))
        h.check()


def test_append_big_step_of_many_requests():
    """More runs than SMs, one token each, and heads that fill no warp group evenly."""
    gen = _gen(7)
    h = _Held(700, 5, 16, 64, "bf16", G=1, B=600)
    perm = torch.randperm(700, generator=gen)[:600]
    slots = perm * 16 + torch.randint(0, 16, (600,), generator=gen)
    slots = slots // 16 * 16  # first rows
    h.append(torch.randn(600, 5, 64, generator=gen).bfloat16(), torch.randn(600, 5, 64, generator=gen).bfloat16(), slots, h.positions(600, gen))
    h.append(torch.randn(600, 5, 64, generator=gen).bfloat16() * 9, torch.randn(600, 5, 64, generator=gen).bfloat16(), slots + 1, h.positions(600, gen))
    h.check()


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
class _Attn:
    def __init__(self, lens, new, D=128, hkv=2, G=4, bs=64, dtype="bf16", S=4, W=100, ret=(0,), sections=None, seed=0, spare=2,
                 pad=0, q_scale=1.5):
        gen = _gen(seed)
        self.gen = gen
        self.lens, self.new, self.S, self.W, self.ret, self.G, self.hkv, self.bs, self.D = lens, new, S, W, ret, G, hkv, bs, D
        self.B = len(lens)
        self.max_ctx = max(max(lens), 1)
        self.dtype = dtype
        self.dt = torch.bfloat16 if dtype == "bf16" else torch.float32
        self.sections = sections
        self.axis = _axis(D, sections) if sections else [0] * (D // 2)
        self.rope = rtp.make_rope(D, sections) if sections else None
        self.cfg = rtp.make_cfg(self.B, hkv * G, hkv, D, self.max_ctx, S, W, 1.0, ret, dtype)
        n = [-(-max(x, 0) // bs) for x in lens]
        nb = sum(n) + spare
        perm = torch.randperm(nb, generator=gen).tolist()
        cols = -(-self.max_ctx // bs)
        self.table = np.full((self.B, cols), -1, np.int64)
        for b in range(self.B):
            for i in range(n[b]):
                self.table[b, i] = perm.pop()
        self.pool = ref.Pool(nb, hkv, bs, D)
        for x, s in ((self.pool.k, self.pool.ks), (self.pool.v, self.pool.vs)):
            e = torch.randint(-9, -3, (nb, hkv), generator=gen)
            s.copy_(2.0 ** e.double())
            x.copy_(ref.to_e4m3((torch.randn(x.shape, generator=gen, dtype=torch.float64) * 60).clamp(-448, 448)))
        self.N = sum(new) + pad
        self.q = (torch.randn(self.N, hkv * G, D, generator=gen) * q_scale).to(self.dt)
        self.pos = torch.randint(0, 4000, (len(sections) if sections else 1, self.N), generator=gen, dtype=torch.int32)
        self.cu = np.concatenate([[0], np.cumsum(new)])
        self.max_q = max(max(new), 1)

    def device(self):
        """Device copies; rows that no request holds are NaN in memory."""
        k = self.pool.k.float().to(torch.float8_e4m3fn).view(torch.uint8).clone()
        v = self.pool.v.float().to(torch.float8_e4m3fn).view(torch.uint8).clone()
        held = torch.zeros(k.shape[0], self.bs, dtype=torch.bool)
        for b in range(self.B):
            for p in range(max(self.lens[b], 0)):
                held[self.table[b, p // self.bs], p % self.bs] = True
        k[~held[:, None].expand(-1, self.hkv, -1)] = 0x7F
        v[~held[:, None].expand(-1, self.hkv, -1)] = 0xFF
        self.dk, self.dv = k.to(DEV), v.to(DEV)
        self.dks, self.dvs = self.pool.ks.float().to(DEV), self.pool.vs.float().to(DEV)
        self.status = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.cache = rtp.make_q8_cache(self.dk, self.dv, self.dks, self.dvs, self.status)
        self.dq, self.dpos, self.dcu, self.dlen, self.dtab = (self.q.to(DEV), self.pos.to(DEV), _i32(self.cu), _i32(self.lens), _i32(self.table))
        n = rtp.rtp_attn_q8_workspace_bytes(self.cfg, self.bs, self.N, self.max_q, 0)
        self.ws = torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV)
        self.out = torch.full((self.N, self.hkv * self.G, self.D), 77.0, dtype=self.dt, device=DEV)
        return self

    def call(self, **kw):
        a = dict(max_q=self.max_q, max_seq_len=0, rope=self.rope, workspace=self.ws, workspace_bytes=self.ws.numel())
        a.update(kw)
        rtp.rtp_attn_q8(self.cfg, self.cache, self.dq, self.dcu, self.dlen, self.dtab, self.dpos, self.out, **a)

    def run(self):
        self.device()
        self.call()
        torch.cuda.synchronize()
        return self.out.cpu().double()

    def r_q(self):
        return 2.0 ** -21 if self.dtype == "fp32" or self.max_q * self.G <= 8 else 2.0 ** -11

    def check(self, got, rows=None, there=None):
        """Every request's rows (all of them, or the chosen (request, query) pairs)."""
        qr = ref.rotate(self.q.double(), ref.angles(self.pos, self.axis, self.D))
        half = 2.0 ** -8 if self.dtype == "bf16" else 2.0 ** -24
        r_w = 2.0 ** -21 if self.dtype == "fp32" else 2.0 ** -11
        worst = 0.0
        for b in range(self.B):
            L, n = self.lens[b], self.new[b]
            if n == 0:
                continue
            for h in range(self.hkv):
                k, v = self.pool.rows(self.table[b], L, h)
                vmax = float(v.abs().max())
                for t in range(n):
                    if rows is not None and (b, t) not in rows:
                        continue
                    seen = ref.visible(L - n + t, L, h in self.ret, self.S, self.W)
                    if there is not None:
                        seen &= there[b][:L]
                    for g in range(self.G):
                        hq = h * self.G + g
                        o, A, Z = ref.attend(qr[self.cu[b] + t, hq], k, v, seen)
                        e = Z * (self.r_q() + 2.0 ** -20)
                        r_p = 2.0 ** -12 if self.dtype == "bf16" and self.max_q * self.G > 32 else 0.0
                        bound = o.abs() * half + A * (math.expm1(2 * e) + r_p + r_w + (L / 16 + 64) * 2.0 ** -23) + L * 2.0 ** -22 * vmax * min(1.0, 64.0 / max(1, int(seen.sum()))) + 1e-30
                        err = (got[self.cu[b] + t, hq] - o).abs()
                        ratio = float((err / bound).max())
                        worst = max(worst, ratio)
                        assert ratio <= 1.0, (b, t, hq, ratio)
        return worst


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("bs", [16, 64, 128])
def test_decode_heads_and_blocks(dtype, D, G, bs):
    """One token a request: contexts of one position up to several CTAs' worth."""
    a = _Attn([1, 2, 15, 16, 17, 33, 300, 5000], [1] * 8, D=D, hkv=3, G=G, bs=bs, dtype=dtype, ret=(0, 2), seed=D + G)
    a.check(a.run())
    assert int(a.status) == 0


@pytest.mark.parametrize("S,W,ret", [(0, 1, ()), (0, 1, (0, 1)), (1, 31, (1,)), (64, 32, ()), (33, 700, (0,)), (5000, 1, ()),
                                     (4, 5000, ())])
def test_decode_masks(S, W, ret):
    a = _Attn([1, 31, 32, 33, 64, 65, 97, 999, 2048], [1] * 9, bs=32, S=S, W=W, ret=ret, seed=S + W)
    a.check(a.run())


@pytest.mark.parametrize("dtype,G,new", [("bf16", 4, [2, 3, 1, 8]), ("bf16", 8, [5, 1, 16, 2]), ("bf16", 1, [8, 7, 9, 1]),
                                         ("bf16", 2, [33, 1, 0, 65]), ("fp32", 4, [2, 3, 1, 8]), ("fp32", 1, [17, 1, 40, 2])])
@pytest.mark.parametrize("bs", [16, 64])
def test_a_few_queries_a_request(dtype, G, new, bs):
    """Drafts: every query has its own causal border, window and position."""
    a = _Attn([400, 90, 66, 1300], new, G=G, bs=bs, dtype=dtype, S=10, W=50, sections=AXIS3[128], seed=G)
    a.check(a.run())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G,new", [(1, [33, 257, 128]), (2, [300, 17, 64]), (4, [9, 64, 65]), (8, [5, 33, 100])])
@pytest.mark.parametrize("bs", [16, 64, 128])
def test_chunks(D, G, new, bs):
    """Rows that end inside a slot, a group and a tile; contexts before the chunk."""
    a = _Attn([max(33, new[0]), 700, 390], new, D=D, G=G, bs=bs, S=10, W=150, sections=AXIS3[D], seed=D + G + bs)
    got = a.run()
    a.check(got, rows={(b, t) for b, n in enumerate(new) for t in range(n) if t % 7 == 0 or t >= n - 2})
    assert int(a.status) == 0


@pytest.mark.parametrize("S,W,ret", [(0, 1, ()), (0, 1, (0, 1)), (129, 300, (1,)), (64, 128, ()), (2000, 1, ())])
def test_chunk_masks(S, W, ret):
    a = _Attn([1500], [600], G=2, bs=32, S=S, W=W, ret=ret, seed=S + W)
    a.check(a.run(), rows={(0, t) for t in range(0, 600, 13)} | {(0, 599)})


def test_chunks_beside_decoding_requests():
    """Streamed and chunk requests, idle ones, and rows behind the last, in one call."""
    new = [1, 200, 0, 8, 9, 1, 513, 2]
    a = _Attn([900, 200, 50, 77, 300, 1, 1111, 640], new, G=4, bs=16, S=20, W=128, pad=7, seed=3)
    got = a.run()
    assert bool((got[sum(new):] == 77.0).all()) and int(a.status) == 0
    a.check(got, rows={(b, t) for b, n in enumerate(new) for t in range(n) if t % 17 == 0 or t == n - 1})


def test_chunk_long_context_is_split_and_joined():
    a = _Attn([20000], [70], hkv=2, G=4, bs=64, S=64, W=2048, ret=(1,), seed=31)
    a.check(a.run(), rows={(0, t) for t in range(0, 70, 9)} | {(0, 69)})
    a = _Attn([9000], [3], hkv=1, G=8, bs=64, ret=(0,), seed=32, pad=40)  # one small request where max_q allows a chunk
    a.device()
    a.max_q = 40
    n = rtp.rtp_attn_q8_workspace_bytes(a.cfg, a.bs, a.N, 40, 0)
    a.ws = torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV)
    a.call()
    torch.cuda.synchronize()
    a.check(a.out.cpu().double())


def test_chunk_that_is_its_whole_context():
    a = _Attn([1000, 129], [1000, 129], G=1, hkv=2, bs=64, S=2, W=70, ret=(1,), seed=33)
    a.check(a.run(), rows={(b, t) for b in range(2) for t in (0, 1, 2, 69, 70, 71, 127, 128)} | {(0, 999), (0, 500)})


def test_chunk_blocks_outside_the_pool_and_stored_nans():
    a = _Attn([400], [100], G=2, bs=64, W=64, S=0, ret=(0,), seed=34)
    a.pool.k[a.table[0, 350 // 64], :, 350 % 64] = math.nan  # position 350: row 50 of the chunk
    a.pool.v[a.table[0, 350 // 64], :, 350 % 64] = 0.0
    a.device()
    tab = a.dtab.clone()
    tab[0, 1] = a.dk.shape[0] + 5
    a.dtab.copy_(tab)
    a.call()
    torch.cuda.synchronize()
    got = a.out.cpu().double()
    assert int(a.status) == rtp.RTP_DEV_BLOCKS
    assert bool(torch.isnan(got[50:]).all()) and bool(torch.isfinite(got[:50]).all())
    a.pool.k.nan_to_num_(0.0)
    a.check(got, rows={(0, t) for t in range(0, 50, 7)}, there=[torch.arange(400) // 64 != 1])


def test_chunk_value_scales_far_apart_and_large_scores():
    a = _Attn([512], [60], bs=64, hkv=1, G=4, ret=(0,), seed=35, q_scale=20.0)
    e = torch.tensor([-30, -20, 0, 10, -7, -5, -60, -1], dtype=torch.float64)
    for i in range(8):
        a.pool.vs[a.table[0, i]] = 2.0 ** e[i]
    a.pool.v[a.table[0, 3]] = 0.0
    a.pool.vs[a.table[0, 3]] = ref.SCALE_MIN
    a.check(a.run())


def test_chunk_call_repeated_captured_and_on_two_streams():
    a, b = _Attn([800, 60], [300, 1], seed=36).device(), _Attn([1300], [256], seed=37).device()
    a.call()
    torch.cuda.synchronize()
    first = a.out.clone()
    s, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            a.call()
    a.ws.random_(0, 255)
    a.out.zero_()
    torch.cuda.synchronize()
    for _ in range(5):
        with torch.cuda.stream(s):
            g.replay()
        b.call(stream=s2)
    torch.cuda.synchronize()
    assert torch.equal(first, a.out)
    a.check(a.out.cpu().double(), rows={(0, 0), (0, 150), (0, 299), (1, 0)})
    b.check(b.out.cpu().double(), rows={(0, 0), (0, 77), (0, 255)})


def test_first_tokens_of_a_request():
    """The queries are the whole context: the first row sees one position."""
    a = _Attn([5, 16, 1, 37], [5, 16, 1, 37], bs=16, S=2, W=3, ret=(1,), seed=2)
    a.check(a.run())


def test_idle_requests_and_rows_behind_the_last_stay_as_they_were():
    a = _Attn([0, 300, 70, 0, 128], [0, 1, 0, 0, 2], bs=64, pad=5, seed=1)
    got = a.run()
    a.check(got)
    assert int(a.status) == 0 and bool((got[3:] == 77.0).all())


def test_requests_that_cannot_be_are_skipped():
    a = _Attn([300, 50, 200], [1, 2, 1], seed=1).device()
    a.dlen.copy_(_i32([300, 1, 301]))  # fewer positions than queries; more than max_ctx
    a.call()
    torch.cuda.synchronize()
    got = a.out.cpu().double()
    assert int(a.status) == rtp.RTP_DEV_SEQ_LEN and bool((got[1:] == 77.0).all())
    a.check(got, rows={(0, 0)})
    for cu, flag in (([0, 1, 0, 1], rtp.RTP_DEV_POSITION), ([0, 1, 9, 4], rtp.RTP_DEV_POSITION), ([0, 1, 4, 4], rtp.RTP_DEV_POSITION)):
        a.device()
        a.dcu.copy_(_i32(cu))
        a.call()
        torch.cuda.synchronize()
        assert int(a.status) & flag
        if cu != [0, 1, 0, 1]:  # there the third request names row 0 too, validly: either may be the last to write it
            a.check(a.out.cpu().double(), rows={(0, 0)})


@pytest.mark.parametrize("bs", [16, 64])
def test_blocks_outside_the_pool_count_as_not_there(bs):
    a = _Attn([300, bs, 1], [1, 1, 1], bs=bs, W=200, S=20, seed=6)
    a.device()
    tab = a.dtab.clone()
    tab[0, 1], tab[0, 300 // bs], tab[1, 0] = -5, a.dk.shape[0], 1 << 30
    a.dtab.copy_(tab)
    a.call()
    torch.cuda.synchronize()
    assert int(a.status) == rtp.RTP_DEV_BLOCKS
    p = torch.arange(300) // bs
    there = [(p != 1) & (p != 300 // bs), torch.zeros(bs, dtype=torch.bool), torch.ones(1, dtype=torch.bool)]
    got = a.out.cpu().double()
    a.check(got, there=there)
    assert bool((got[1] == 0).all())  # a query that sees nothing


def test_a_row_stored_as_nan_reaches_only_the_queries_that_see_it():
    a = _Attn([200, 200], [4, 1], bs=32, S=0, W=10, ret=(0,), seed=9)
    a.pool.k[a.table[0, 197 // 32], :, 197 % 32] = math.nan  # position 197 of request 0: queries at 197, 198, 199 see it
    a.pool.v[a.table[0, 197 // 32], :, 197 % 32] = 0.0
    a.pool.k[a.table[1, 3], :, 0] = math.nan  # position 96 of request 1: only the retrieval head's queries see it
    a.pool.v[a.table[1, 3], :, 0] = 0.0
    got = a.run()
    assert bool(torch.isnan(got[1:4]).all()) and bool(torch.isnan(got[4, :4]).all())
    assert bool(torch.isfinite(got[0]).all()) and bool(torch.isfinite(got[4, 4:]).all())
    a.pool.k.nan_to_num_(0.0)
    a.check(got, rows={(0, 0)})


def test_value_scales_far_apart():
    """Blocks of values 2^40 apart, an all-zero block of the least scale among them."""
    a = _Attn([512], [1], bs=64, hkv=1, G=8, ret=(0,), dtype="fp32", seed=11, q_scale=0.2)
    e = torch.tensor([-30, -20, 0, 10, -7, -5, -60, -1], dtype=torch.float64)
    for i in range(8):
        a.pool.vs[a.table[0, i]] = 2.0 ** e[i]
    a.pool.v[a.table[0, 3]] = 0.0
    a.pool.vs[a.table[0, 3]] = ref.SCALE_MIN
    a.check(a.run())


def test_large_scores_and_flat_ones():
    for scale in (0.0, 1e-3, 30.0):
        a = _Attn([700, 3], [1, 1], seed=5, q_scale=scale)
        got = a.run()
        a.check(got)


def test_long_context_split_over_all_ctas():
    a = _Attn([70001], [1], hkv=1, G=2, bs=64, seed=12)
    a.check(a.run())


def test_many_short_requests():
    r = random.Random(3)
    lens = [r.randrange(1, 120) for _ in range(300)]
    a = _Attn(lens, [1] * 300, hkv=2, G=2, D=64, bs=16, seed=13)
    a.check(a.run(), rows={(b, 0) for b in range(0, 300, 7)})


def test_same_call_twice_gives_the_same_bits():
    a = _Attn([5000, 777], [1, 3], seed=14)
    first = a.run()
    a.ws.random_(0, 255)
    a.out.fill_(5.0)
    a.call()
    torch.cuda.synchronize()
    assert torch.equal(first, a.out.cpu().double())


def test_captured_and_replayed_with_new_lengths():
    a = _Attn([900, 2000], [1, 1], seed=15).device()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        a.call()
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            a.call()
    for lens in ([900, 2000], [33, 1], [1, 1999]):
        a.dlen.copy_(_i32(lens))
        g.replay()
        torch.cuda.synchronize()
        a.lens = lens
        a.check(a.out.cpu().double())


def test_two_streams_with_a_workspace_each():
    a, b = _Attn([3000], [1], seed=16).device(), _Attn([2500, 100], [2, 1], seed=17).device()
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(20):
        a.call(stream=sa)
        b.call(stream=sb)
    torch.cuda.synchronize()
    a.check(a.out.cpu().double())
    b.check(b.out.cpu().double())


@pytest.mark.parametrize("new", [[1, 3], [90, 1]])
def test_requests_that_share_blocks(new):
    a = _Attn([700, 650], new, bs=32, seed=22)
    a.table[1, :12] = a.table[0, :12]  # a common prefix of 384 positions
    a.check(a.run())


def test_a_graph_outlives_its_layers_scratch():
    from synth.workloads import LayerShape
    sh = LayerShape(batch=2, n_q_heads=8, n_kv_heads=2, head_dim=64, n_sink=4, window=100, top_p=1.0, retrieval=(0,), dtype="bf16")
    a = _Attn([1900, 400], [1, 1], D=64, seed=23).device()
    layer = rtp.PagedLayer(sh, a.max_ctx, a.dk.shape[0], a.bs)
    layer.cache = a.cache
    layer.reserve(2, 1)
    small, s, g = layer.ws, torch.cuda.Stream(), torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        with torch.cuda.graph(g, stream=s):
            layer.attend(a.dq, a.dcu, a.dlen, a.dtab, a.dpos, a.out, 1)
    layer.reserve(500, 400)
    assert layer.ws.numel() >= 2 * small.numel() and any(t is small for t in layer._outgrown)
    filler = torch.full_like(small, 0xFF)  # would lie where the scratch was, had it been freed
    a.out.fill_(77.0)
    g.replay()
    torch.cuda.synchronize()
    a.check(a.out.cpu().double())
    assert bool((filler == 0xFF).all())


def test_pool_past_two_gigabytes():
    """Blocks at the far end of a 4.5 GB pool: offsets beyond 32 bits, for the append and the attention."""
    nb, hkv, bs, D = 34400, 8, 128, 128
    size = (nb, hkv, bs, D)
    k, v = torch.zeros(size, dtype=torch.uint8, device=DEV), torch.zeros(size, dtype=torch.uint8, device=DEV)
    ks, vs = torch.ones(size[:2], device=DEV), torch.ones(size[:2], device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    cfg = rtp.make_cfg(1, 8, 8, 128, 256, 4, 128, 1.0, range(8), "bf16")
    cache = rtp.make_q8_cache(k, v, ks, vs, status)
    gen = _gen(1)
    x, y = torch.randn(200, 8, 128, generator=gen).bfloat16(), torch.randn(200, 8, 128, generator=gen).bfloat16()
    pos = torch.arange(200, dtype=torch.int32)[None]
    slots = torch.cat([torch.arange(128) + (nb - 1) * bs, torch.arange(72) + (nb - 7) * bs])
    rtp.rtp_append_q8(cfg, cache, x.to(DEV), y.to(DEV), slots.to(DEV), pos.to(DEV))
    pool = ref.Pool(2, 8, bs, D)
    pool.append(ref.rotate(x.double(), ref.angles(pos, [0] * 64, D)), y, torch.cat([torch.arange(128) + bs, torch.arange(72)]))
    for dst, src in ((k, pool.k), (v, pool.v)):
        assert torch.equal(dst[nb - 1].view(torch.float8_e4m3fn).cpu().double(), src[1])
        assert torch.equal(dst[nb - 7].view(torch.float8_e4m3fn).cpu().double(), src[0])
    assert int(k[0].sum()) == 0 and int(k[nb - 2].sum()) == 0
    q = torch.randn(1, 8, 128, generator=gen).bfloat16()
    out = torch.empty_like(q, device=DEV)
    ws = torch.empty(rtp.rtp_attn_q8_workspace_bytes(cfg, bs, 1, 1), dtype=torch.uint8, device=DEV)
    rtp.rtp_attn_q8(cfg, cache, q.to(DEV), _i32([0, 1]), _i32([200]), _i32([[nb - 1, nb - 7]]), _i32([[199]]), out, 1, 0, None, ws, ws.numel())
    qr = ref.rotate(q.double(), ref.angles(torch.tensor([[199]]), [0] * 64, D))
    for h in range(8):
        kk, vv = pool.rows([1, 0], 200, h)
        o, A, Z = ref.attend(qr[0, h], kk, vv, torch.ones(200, dtype=torch.bool))
        e = Z * (2.0 ** -21 + 2.0 ** -20)
        assert bool(((out[0, h].cpu().double() - o).abs() <= o.abs() * 2.0 ** -8 + A * (math.expm1(2 * e) + 2.0 ** -10)).all())
    assert int(status) == 0


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype,bs", [("bf16", 16), ("bf16", 64), ("fp32", 32)])
def test_a_serving_loop(dtype, bs):
    """Steps of plan, append and attention: prompts in chunks, decoding, a
    request that ends and another that takes its blocks."""
    from synth.workloads import LayerShape
    D, hkv, G, B, max_ctx = 64, 2, 4, 3, 512
    sh = LayerShape(batch=B, n_q_heads=hkv * G, n_kv_heads=hkv, head_dim=D, n_sink=4, window=60, top_p=1.0, retrieval=(1,), dtype=dtype)
    n_blocks = -(-700 // bs) + B
    layer = rtp.PagedLayer(sh, max_ctx, n_blocks, bs)
    a = _Attn([1] * B, [1] * B, D=D, hkv=hkv, G=G, bs=bs, dtype=dtype, S=4, W=60, ret=(1,))
    a.pool = ref.Pool(n_blocks, hkv, bs, D)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    gen = _gen(21)
    cols = -(-max_ctx // bs)
    tab = torch.full((B, cols), -1, dtype=torch.int32, device=DEV)
    free = torch.arange(n_blocks, dtype=torch.int32, device=DEV)
    n_free = _i32([n_blocks])
    length = _i32([0] * B)
    cu = _i32([0] * (B + 1))
    cap = 256
    slots, pos = torch.zeros(cap, dtype=torch.int64, device=DEV), torch.zeros(cap, dtype=torch.int32, device=DEV)
    for new in ([100, 0, 33], [100, 57, 1], [1, 1, 1], [1, -1, 1], [1, 0, 1], [3, 140, 100], [1, 1, 1], [1, 1, 4]):
        rtp.rtp_page_plan(layer.cfg, bs, length, _i32(new), tab, free, n_free, length, cu, slots, pos, n_free, layer.status)
        n = sum(max(x, 0) for x in new)
        k, v = (torch.randn(cap, hkv, D, generator=gen).to(dt) for _ in range(2))
        q = torch.randn(cap, hkv * G, D, generator=gen).to(dt)
        out = torch.full((cap, hkv * G, D), 77.0, dtype=dt, device=DEV)
        layer.append(k.to(DEV), v.to(DEV), slots, pos)  # padded to cap: rows past the last have no slot
        layer.attend(q.to(DEV), cu, length, tab, pos, out, max(max(new), 1))
        torch.cuda.synchronize()
        assert layer.device_status() == 0
        p = pos.cpu()[None]
        a.pool.append(ref.rotate(k.double(), ref.angles(p, a.axis, D)), v, slots.cpu())
        a.lens, a.new = [int(x) for x in length], [max(x, 0) for x in new]
        a.cu, a.table, a.q, a.pos, a.max_q = cu.cpu().numpy(), tab.cpu().numpy(), q, p, max(max(new), 1)
        rows = {(b, t) for b in range(B) for t in range(a.new[b]) if t % 9 == 0 or t == a.new[b] - 1}
        a.check(out.cpu().double(), rows=rows)
        assert bool((out[n:] == 77.0).all())
