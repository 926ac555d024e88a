"""The paged 8-bit cache at the ends of what its calls allow: configuration
values, value and query sizes, batches, rotary axes, streams, lengths that
fall.  The references and the bounds are those of tests/test_gpu_q8.py unless
a test gives its own."""

import math

import pytest
import torch

import head_wise_sparse_local_b200 as rtp
import q8_reference as ref
from test_gpu_q8 import AXIS3, _Attn, _Held

pytestmark = pytest.mark.gpu

DEV = "cuda"
INT_MAX = 2 ** 31 - 1


# ---------------------------------------------------------------------------
# sinks and windows past every position
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("S,W", [(INT_MAX, 1), (INT_MAX - 30, 5), (INT_MAX - 126, 7), (0, INT_MAX), (3, INT_MAX - 1), (INT_MAX, INT_MAX)])
def test_every_position_a_sink_or_in_the_window(S, W):
    a = _Attn([1, 32, 97, 999, 2048], [1, 2, 1, 3, 1], bs=32, S=S, W=W, ret=(1,), seed=41)
    a.check(a.run())
    a = _Attn([1500, 40], [300, 1], G=2, bs=32, S=S, W=W, ret=(1,), seed=42)
    a.check(a.run(), rows={(0, t) for t in range(0, 300, 13)} | {(0, 299), (1, 0)})
    assert int(a.status) == 0


def test_prefill_and_decode_where_every_position_is_a_sink():
    """The layer's own cache: the same bits as for sinks that just cover the context."""
    from parity import run_gpu_decode, run_gpu_prefill
    from synth import LayerShape, make_decode_inputs, make_prefill_inputs
    outs = []
    for S in (700, INT_MAX, INT_MAX - 126):
        sh = LayerShape(batch=1, n_q_heads=8, n_kv_heads=2, head_dim=128, n_sink=S, window=40, top_p=0.85, retrieval=(1,), dtype="bf16")
        w = dict(seed=31, ctx=260, needles=6, shape=sh)
        p = run_gpu_prefill(make_prefill_inputs(dict(w, kind="prefill"), T=260, start_pos=0, max_ctx=600))
        d = run_gpu_decode(make_decode_inputs(dict(w, kind="decode"), max_ctx=600))
        outs.append((torch.as_tensor(p["out"]), torch.as_tensor(d["out"])))
    for p, d in outs[1:]:
        assert torch.equal(p, outs[0][0]) and torch.equal(d, outs[0][1])


# ---------------------------------------------------------------------------
# a pool that is not the configuration's
# ---------------------------------------------------------------------------
def test_a_pool_of_other_heads_is_refused_before_the_call():
    a = _Attn([100], [1], D=64, hkv=2, G=2, bs=32, seed=3).device()
    a.call()
    torch.cuda.synchronize()
    for kw in (dict(n_kv_heads=4, n_q_heads=8), dict(head_dim=128)):
        base = dict(batch=1, n_q_heads=4, n_kv_heads=2, head_dim=64, max_ctx=100, n_sink=4, window=100, top_p=1.0, retrieval=(0,))
        base.update(kw)
        cfg = rtp.make_cfg(**base)
        shape = (1, cfg.n_kv_heads, cfg.head_dim)
        k = torch.zeros(shape, dtype=torch.bfloat16, device=DEV)
        q = torch.zeros(1, cfg.n_q_heads, cfg.head_dim, dtype=torch.bfloat16, device=DEV)
        with pytest.raises(ValueError, match="pool"):
            rtp.rtp_append_q8(cfg, a.cache, k, k, torch.zeros(1, dtype=torch.int64, device=DEV), a.dpos)
        with pytest.raises(ValueError, match="pool"):
            rtp.rtp_attn_q8(cfg, a.cache, q, a.dcu, a.dlen, a.dtab, a.dpos, torch.empty_like(q), 1, 0, None, a.ws, a.ws.numel())


# ---------------------------------------------------------------------------
# a layer's own memory on streams that are not the current one
# ---------------------------------------------------------------------------
def _layer(n_blocks=60, bs=32, B=2):
    from synth import LayerShape
    sh = LayerShape(batch=B, n_q_heads=8, n_kv_heads=2, head_dim=64, n_sink=4, window=100, top_p=1.0, retrieval=(0,), dtype="bf16")
    return rtp.PagedLayer(sh, 1900, n_blocks, bs)


def _busy(stream=None):
    """About a tenth of a second of work."""
    with torch.cuda.stream(stream or torch.cuda.current_stream()):
        torch.cuda._sleep(200_000_000)


def test_a_new_layer_can_be_appended_to_on_any_stream():
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    x = torch.randn(4, 2, 64, device=DEV).bfloat16()
    slots, pos = torch.arange(4, device=DEV), torch.zeros(1, 4, dtype=torch.int32, device=DEV)
    for busy in (False, True):  # (the first loads the kernels and leaves its blocks to the allocator)
        torch.cuda.synchronize()
        if busy:
            _busy()  # the pool's zeros would wait behind this
        layer = None
        layer = _layer()
        layer.append(x, x, slots, pos, stream=s)
    torch.cuda.synchronize()
    assert bool((layer.v[0, :, :4].float() * layer.v_scale[0][:, None, None] != 0).any(-1).all()) and layer.device_status() == 0


@pytest.mark.parametrize("how", ["stream argument", "current stream", "raw handle"])
def test_scratch_is_not_memory_that_another_stream_still_uses(how):
    a = _Attn([1900, 400], [70, 1], D=64, bs=32, seed=23).device()
    layer = _layer(a.dk.shape[0])
    layer.cache = a.cache
    n = rtp.rtp_attn_q8_workspace_bytes(layer.cfg, 32, a.N, 70)
    s = torch.cuda.Stream()
    a.call()  # (loads the kernels)
    a.out.zero_()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    old = torch.zeros(n, dtype=torch.uint8, device=DEV)
    at = old.data_ptr()
    torch.cuda.synchronize()
    _busy()
    old.fill_(0xFF)
    pending = torch.cuda.Event()
    pending.record()
    del old  # its block is the allocator's to give, and its last user has not run
    args = (a.dq, a.dcu, a.dlen, a.dtab, a.dpos, a.out, 70)
    if how == "current stream":
        with torch.cuda.stream(s):
            layer.attend(*args)
    else:
        layer.attend(*args, stream=s if how == "stream argument" else s.cuda_stream)
    assert layer.ws.numel() >= n
    assert pending.query() or not at <= layer.ws.data_ptr() < at + n
    torch.cuda.synchronize()
    a.check(a.out.cpu().double(), rows={(0, 0), (0, 33), (0, 69), (1, 0)})


def test_memory_of_a_layer_that_goes_waits_for_its_streams():
    a = _Attn([1900, 400], [70, 1], D=64, bs=32, seed=24).device()
    a.call()  # (loads the kernels)
    a.out.zero_()
    s = torch.cuda.Stream()
    layer = _layer(a.dk.shape[0])
    layer.cache = a.cache
    n = rtp.rtp_attn_q8_workspace_bytes(layer.cfg, 32, a.N, 70)
    layer.reserve(a.N, 70)
    held = [(t.data_ptr(), t.numel()) for t in (layer.ws, layer.k, layer.v)]
    torch.cuda.synchronize()
    _busy(s)
    layer.attend(a.dq, a.dcu, a.dlen, a.dtab, a.dpos, a.out, 70, stream=s)
    done = torch.cuda.Event()
    done.record(s)
    del layer
    new = [torch.empty(k, dtype=torch.uint8, device=DEV) for _, k in held]
    taken = [t.data_ptr() for t in new]
    assert not done.query()  # (else the test shows nothing)
    assert not any(at <= p < at + k for p in taken for at, k in held)
    torch.cuda.synchronize()
    a.check(a.out.cpu().double(), rows={(0, 0), (0, 33), (0, 69), (1, 0)})


def test_prefill_scratch_on_another_stream_and_in_a_graph_that_outlives_it():
    """The layer's own cache: a chunk on a stream that is not the current one, then a
    longer one; the first one's graph still has its scratch."""
    from synth import LayerShape
    sh = LayerShape(batch=1, n_q_heads=8, n_kv_heads=2, head_dim=64, n_sink=4, window=40, top_p=0.9, retrieval=(1,), dtype="bf16")
    gen = torch.Generator(device=DEV).manual_seed(5)
    x = [torch.randn(1, 900, h, 64, device=DEV, generator=gen).bfloat16() for h in (8, 2, 2)]
    w_q, w_k = torch.randn(1, 16, 64, device=DEV, generator=gen), torch.randn(1, 16, 64, device=DEV, generator=gen)
    start, s = torch.zeros(1, dtype=torch.int32, device=DEV), torch.cuda.Stream()

    def chunk(layer, T, out, stream=None):
        layer.append(x[1][:, :T].contiguous(), x[2][:, :T].contiguous(), start, w_k, stream=stream)
        layer.prefill(x[0][:, :T].contiguous(), start, w_q, out, stream=stream)

    out = {T: torch.empty(1, T, 8, 64, dtype=torch.bfloat16, device=DEV) for T in (300, 900)}
    layer = rtp.Layer(sh, 1024)
    for T in out:
        chunk(layer, T, out[T])
    want = {T: o.clone() for T, o in out.items()}
    layer = rtp.Layer(sh, 1024)
    n = rtp.rtp_prefill_workspace_bytes(layer.cfg, 300)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    old = torch.zeros(n, dtype=torch.uint8, device=DEV)
    at = old.data_ptr()
    q, k, v = (y[:, :300].contiguous() for y in x)
    torch.cuda.synchronize()
    _busy()
    old.fill_(0xFF)
    pending = torch.cuda.Event()
    pending.record()
    del old
    layer.append(k, v, start, w_k, stream=s)
    layer.prefill(q, start, w_q, out[300].zero_(), stream=s)
    assert pending.query() or not at <= layer.ws_prefill.data_ptr() < at + n
    torch.cuda.synchronize()
    layer.prefill(q, start, w_q, out[300], stream=s)
    torch.cuda.synchronize()
    assert torch.equal(out[300], want[300])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(g, stream=s):
            layer.prefill(q, start, w_q, out[300])
    small = layer.ws_prefill
    chunk(layer, 900, out[900])
    assert torch.equal(out[900], want[900]) and layer.ws_prefill is not small and any(t is small for t in layer._outgrown)
    out[300].zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[300], want[300]) and layer.device_status() == 0


# ---------------------------------------------------------------------------
# value scales of any size beside one another
# ---------------------------------------------------------------------------
def _with_value_scales(a, exps, b=0):
    """Request b's blocks get these value scales, the least one together with zero values."""
    for i, e in enumerate(exps):
        blk = a.table[b, i]
        a.pool.vs[blk] = 2.0 ** e
        if e == -64:
            a.pool.v[blk] = 0.0
    return a


FAR_APART = [(-64, 100, -64, -40, 110, -64, 3, -64), (110, -64, -64, -64, -64, -64, -64, 105), (-64,) * 7 + (112,), (112,) + (-64,) * 7,
             (60, -64, 56, -63, -64, 0, 61, -64)]


@pytest.mark.parametrize("exps", FAR_APART)
@pytest.mark.parametrize("dtype,G,new", [("fp32", 4, 1), ("bf16", 8, 1), ("bf16", 4, 4), ("bf16", 4, 60)])
@pytest.mark.parametrize("ret", [(0,), ()])
def test_value_scales_over_their_whole_range(exps, dtype, G, new, ret):
    """Every position has about the same weight, so a block whose weights vanish
    beside another's scale would take its share of the sum with it."""
    a = _Attn([512], [new], bs=64, hkv=1, G=G, ret=ret, S=20, W=200, dtype=dtype, seed=11, q_scale=0.2)
    a.check(_with_value_scales(a, exps).run())


def test_value_scales_over_their_whole_range_in_cut_items():
    """Partials of CTAs, and of warps, whose maxima lie as far apart."""
    exps = [(-64, 110, -64, -64, 40, -64, -64, 105, 0)[i % 9] for i in range(313)]
    a = _Attn([20000], [1], bs=64, hkv=2, G=4, ret=(0, 1), S=0, W=1, seed=12, q_scale=0.2)
    a.check(_with_value_scales(a, exps).run())
    a = _Attn([20000], [70], bs=64, hkv=2, G=4, ret=(0, 1), S=0, W=1, seed=13, q_scale=0.2)
    a.check(_with_value_scales(a, sorted(exps)).run(), rows={(0, t) for t in range(0, 70, 23)})
    a = _Attn([20000], [70], bs=64, hkv=2, G=4, ret=(0, 1), S=0, W=1, seed=13, q_scale=0.2)
    a.check(_with_value_scales(a, sorted(exps, reverse=True)).run(), rows={(0, t) for t in range(0, 70, 23)})


@pytest.mark.parametrize("new", [1, 100])
def test_a_query_that_sees_nothing_gets_zero_whatever_lies_behind_it(new):
    """A chunk's first queries see only blocks that are not there; the positions
    after theirs have values of any scale."""
    for e in (-64, -20, 0, 10, 40, 100):
        a = _Attn([128], [new], bs=16, hkv=1, G=4, ret=(0,), seed=17)
        _with_value_scales(a, (e,) * 8)
        a.device()
        tab = a.dtab.clone()
        tab[0, :3] = -1
        if new == 1:
            tab[0, :] = -1
        a.dtab.copy_(tab)
        a.call()
        torch.cuda.synchronize()
        got = a.out.cpu().double()
        assert bool((got[:20] == 0).all()), e  # positions 28 to 47 (or 127 alone)
        if new > 1:
            a.check(got, rows={(0, t) for t in range(20, 100, 9)}, there=[torch.arange(128) >= 48])


# ---------------------------------------------------------------------------
# queries of any size
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype,G,new", [("fp32", 4, 1), ("bf16", 8, 1), ("bf16", 4, 4), ("bf16", 4, 60)])
@pytest.mark.parametrize("size", [-100, -70, -45, 50])
def test_small_and_large_queries_against_keys_of_the_inverse_size(dtype, G, new, size):
    if new == 60:
        size = max(size, -64)  # chunks
    a = _Attn([300], [new], bs=32, hkv=1, G=G, ret=(0,), dtype=dtype, seed=19, q_scale=1.5 * 2.0 ** size)
    a.pool.ks *= 2.0 ** -size
    a.check(a.run())


@pytest.mark.parametrize("dtype,new", [("fp32", 1), ("fp32", 60), ("bf16", 1), ("bf16", 4)])  # (chunks want scores below 2^23)
def test_the_largest_finite_queries(dtype, new):
    """Scores of 2^60 and more: the position of the largest takes all, where it leads
    the next by more than the scores' error."""
    a = _Attn([200], [new], bs=32, hkv=1, G=4, ret=(0,), dtype=dtype, seed=20, q_scale=1.0)
    a.q = (a.q / a.q.float().abs().amax() * 2.0 ** 127).to(a.dt)
    a.pos.zero_()  # not turned: a rotation could pass the largest number
    a.pool.ks[:] = ref.SCALE_MIN
    got, led = a.run(), 0
    assert bool(torch.isfinite(got).all())
    k, v = a.pool.rows(a.table[0], 200, 0)
    for t in range(new):
        for g in range(4):
            q = a.q[t, g].double()
            s = (k @ q)[:200 - new + t + 1]
            err = float((k.abs() @ q.abs()).max()) * (a.r_q() + 2.0 ** -20)
            top = torch.topk(s, 2)
            if float(top.values[0] - top.values[1]) > 4 * err:
                led += 1
                want = v[top.indices[0]]
                assert bool(((got[t, g] - want).abs() <= want.abs() * 2.0 ** -8).all())
    assert led >= 2 * new


@pytest.mark.parametrize("ascending", [False, True])
def test_chunk_scores_up_to_2_23(ascending):
    """Scores that grow (or fall) by powers of two over the context, to just below
    2^23: one position takes all."""
    a = _Attn([400], [60], bs=32, hkv=1, G=4, ret=(0,), seed=21, q_scale=1.0)
    a.pos.zero_()
    for i in range(13):  # 13 blocks of 32
        a.pool.ks[a.table[0, i]] = 2.0 ** ((i if ascending else 12 - i) + 1)
    qm = float((a.q.double().abs().sum(-1)).amax()) * 448 * 2.0 ** 13 / 128 ** 0.5
    a.q = (a.q.double() * (2.0 ** 22 * 1.9 / qm)).to(a.dt)
    got = a.run()
    assert bool(torch.isfinite(got).all()) and int(a.status) == 0
    k, v = a.pool.rows(a.table[0], 400, 0)
    led = 0
    for t in range(0, 60, 7):
        for g in range(4):
            q = a.q[t, g].double()
            s = (k @ q)[:400 - 60 + t + 1] / 128 ** 0.5
            err = float((k.abs() @ q.abs()).max()) / 128 ** 0.5 * (a.r_q() + 2.0 ** -20)
            top = torch.topk(s, 2)
            if float(top.values[0] - top.values[1]) > 4 * err + 40:
                led += 1
                want = v[top.indices[0]]
                assert bool(((got[t, g] - want).abs() <= want.abs() * (2.0 ** -8 + 2.0 ** -10)).all())
    assert led >= 12


# ---------------------------------------------------------------------------
# bf16 layers held to what their own roundings allow
# ---------------------------------------------------------------------------
class _Strict(_Attn):
    """With one fp16 part a row's queries (over 8 query rows a KV head), the bound of
    test_gpu_q8.py takes the rounding of every query dim at its worst, and leaves large
    scores nearly free.  Here the reference rounds the queries as the kernels do, so
    what is left of the score's error is
      - dims that the fp32 rotation (off by 1.125 2^-22 (|x1| + |x2|)) may bring to
        either side of a rounding border: a step of fp16 times |k|;
      - one truncation, 2^-23 of sum |q k|, for each 16 products, D / 16 <= 8 of them;
      - the factor from products to base 2 (three roundings and a reciprocal root) and
        the scaled score's own rounding: 2^-20 of the score, and 2^-18.
    A weight p_j is then off by b_j = expm1 of that, and in chunks by the cubic's 7.5e-5;
    the numerator's weights also by their fp16 rounding 2^-11, or 2^-25 where they are
    subnormal, against a largest weight of 2^5 or more.  So
      |out - o| <= sum p_j b_j |v_j - o| + 2^-11 sum p_j |v_j| + L 2^-30 448 max_j p_j vs_j
                   + (L / 16 + 64) 2^-23 sum p_j |v_j| + |o| 2^-8
    (times 1 + 2 max b for the second order)."""

    def strict(self, got, rows):
        told = []  # rows of which the bound rejects an answer of zeros
        sc = 1.0 / math.sqrt(self.D)
        th = ref.angles(self.pos, self.axis, self.D)
        qr, x = ref.rotate(self.q.double(), th), self.q.double().abs()
        h = self.D // 2
        pair = x[..., :h] + x[..., h:]
        off = torch.cat([pair, pair], -1) * 1.25 * 2.0 ** -22
        chunk = self.max_q * self.G > 32
        for b in range(self.B):
            L, n = self.lens[b], self.new[b]
            if n == 0:
                continue
            own = chunk and (n * self.G > 32 or self.B == 1)  # its kernel
            for hk in range(self.hkv):
                k, v = self.pool.rows(self.table[b], L, hk)
                vs = self.pool.vs[torch.as_tensor(self.table[b][:-(-L // self.bs)]), hk].repeat_interleave(self.bs)[:L]
                for t in range(n):
                    if (b, t) not in rows:
                        continue
                    seen = ref.visible(L - n + t, L, hk in self.ret, self.S, self.W)
                    ks, vv, vss = k[seen], v[seen], vs[seen]
                    for g in range(self.G):
                        tok, hq = self.cu[b] + t, hk * self.G + g
                        y, d = qr[tok, hq], off[tok, hq]
                        unit = 2.0 ** (math.floor(math.log2(float(y.abs().max()))) - 8)
                        q = (y / unit).half().double() * unit
                        step = (((y + d) / unit).half().double() - ((y - d) / unit).half().double()).abs() * unit
                        s = ks @ q * sc
                        e = (ks.abs() @ step + ks.abs() @ q.abs() * 2.0 ** -20) * sc + s.abs() * 2.0 ** -20 + 2.0 ** -18
                        p = torch.softmax(s, 0)
                        o = p @ vv
                        bj = torch.expm1(e) + (7.5e-5 if own else 0.0)
                        A = p @ vv.abs()
                        bound = (((p * bj) @ (vv - o).abs()) * (1 + 2 * float((bj * p).sum())) + A * (2.0 ** -11 + (L / 16 + 64) * 2.0 ** -23)
                                 + L * 2.0 ** -30 * 448 * float((p * vss).max()) + o.abs() * 2.0 ** -8)
                        err = (got[tok, hq] - o).abs()
                        assert bool((err <= bound).all()), (b, t, hq, float((err / bound).max()))
                        told.append(bool((o.abs() > 2 * bound).any()))
        assert sum(told) >= 0.95 * len(told), (sum(told), len(told))


@pytest.mark.parametrize("q_scale", [0.3, 1.5, 6.0, 20.0])
@pytest.mark.parametrize("new,G", [(60, 4), (4, 4), (300, 1)])
def test_large_scores_and_value_scales_far_apart(q_scale, new, G):
    a = _Strict([512], [new], bs=64, hkv=1, G=G, ret=(0,), seed=35, q_scale=q_scale)
    for i, e in enumerate((-30, -20, 0, 10, -7, -5, -60, -1)):
        a.pool.vs[a.table[0, i]] = 2.0 ** e
    a.pool.v[a.table[0, 3]] = 0.0
    a.pool.vs[a.table[0, 3]] = ref.SCALE_MIN
    a.strict(a.run(), {(0, t) for t in range(0, new, max(1, new // 15))})


@pytest.mark.parametrize("q_scale", [1.5, 12.0])
@pytest.mark.parametrize("new", [[600, 64, 3], [17, 200, 9]])
def test_chunks_drafts_and_windows_strictly(q_scale, new):
    a = _Strict([1500, 700, 333], new, D=128, hkv=2, G=2, bs=32, S=33, W=150, ret=(1,), sections=AXIS3[128], seed=36, q_scale=q_scale)
    a.strict(a.run(), {(b, t) for b, n in enumerate(new) for t in range(0, n, max(1, n // 9))})


@pytest.mark.parametrize("q_scale", [1.5, 12.0])
def test_cut_items_strictly(q_scale):
    for lens, new, D in (([20000], [70], 128), ([15000, 9000], [100, 5], 64)):
        a = _Strict(lens, new, D=D, hkv=2, G=4, bs=64, S=64, W=2048, ret=(1,), seed=37, q_scale=q_scale)
        a.strict(a.run(), {(b, t) for b, n in enumerate(new) for t in (0, n // 2, n - 1)})


def test_scores_that_rise_along_the_context():
    """The maximum moves again and again, in either half of a tile: what was weighed
    before it is brought down by factors that are exact."""
    a = _Strict([1024], [100], bs=16, hkv=1, G=4, ret=(0,), seed=38, q_scale=6.0)
    for i in range(64):
        a.pool.ks[a.table[0, i]] = 2.0 ** -9 if i % 3 else 2.0 ** (-9 + i // 11)
    a.strict(a.run(), {(0, t) for t in range(0, 100, 9)})


# ---------------------------------------------------------------------------
# steps of a serving loop
# ---------------------------------------------------------------------------
class _Serving:
    """A layer with the arrays of a loop, and what it ought to hold."""

    def __init__(self, B, n_blocks, bs=16, max_ctx=256, cap=256, D=64, hkv=2, G=4, seed=51):
        from synth import LayerShape
        sh = LayerShape(batch=B, n_q_heads=hkv * G, n_kv_heads=hkv, head_dim=D, n_sink=4, window=60, top_p=1.0, retrieval=(1,), dtype="bf16")
        self.layer, self.B, self.bs, self.cap, self.D = rtp.PagedLayer(sh, max_ctx, n_blocks, bs), B, bs, cap, D
        self.a = _Attn([1] * B, [1] * B, D=D, hkv=hkv, G=G, bs=bs, S=4, W=60, ret=(1,))
        self.a.pool, self.gen = ref.Pool(n_blocks, hkv, bs, D), torch.Generator().manual_seed(seed)
        i32 = dict(dtype=torch.int32, device=DEV)
        self.table, self.free = torch.full((B, -(-max_ctx // bs)), -1, **i32), torch.arange(n_blocks, **i32)
        self.n_free, self.length, self.cu = torch.tensor([n_blocks], **i32), torch.zeros(B, **i32), torch.zeros(B + 1, **i32)
        self.slots, self.pos = torch.zeros(cap, dtype=torch.int64, device=DEV), torch.zeros(cap, **i32)

    def plan(self, new):
        rtp.rtp_page_plan(self.layer.cfg, self.bs, self.length, torch.tensor(new, dtype=torch.int32, device=DEV), self.table, self.free,
                          self.n_free, self.length, self.cu, self.slots, self.pos, self.n_free, self.layer.status)

    def step(self, new, refused=()):
        """Plan, append, attend; the outputs of the requests that are served are checked."""
        a, cap = self.a, self.cap
        self.plan(new)
        k, v = (torch.randn(cap, a.hkv, self.D, generator=self.gen).bfloat16() for _ in range(2))
        q = torch.randn(cap, a.hkv * a.G, self.D, generator=self.gen).bfloat16()
        out = torch.full((cap, a.hkv * a.G, self.D), 77.0, dtype=torch.bfloat16, device=DEV)
        self.layer.append(k.to(DEV), v.to(DEV), self.slots, self.pos)
        mq = max(max(new), 1)
        self.layer.attend(q.to(DEV), self.cu, self.length, self.table, self.pos, out, mq)
        torch.cuda.synchronize()
        p = self.pos.cpu()[None]
        a.pool.append(ref.rotate(k.double(), ref.angles(p, a.axis, self.D)), v, self.slots.cpu())
        a.lens, a.new = [int(x) for x in self.length], [max(x, 0) for x in new]
        a.cu, a.table, a.q, a.pos, a.max_q = self.cu.cpu().numpy(), self.table.cpu().numpy(), q, p, mq
        a.check(out.cpu().double(), rows={(b, t) for b in range(self.B) if b not in refused for t in range(a.new[b])})
        assert bool((out[sum(a.new):] == 77.0).all())
        return out


def test_a_refused_request_beside_others():
    """Out of blocks: the request's rows are those without a slot, nothing of it is
    stored, the others' outputs are right, and it is served once there is room."""
    s = _Serving(3, 8)
    s.step([40, 30, 16])  # 3, 2 and 1 blocks of 8
    held = (s.layer.k.clone().view(torch.uint8), s.table.clone())
    s.step([8, 40, 0], refused=(1,))  # the second wants 3 more
    # (attention says too that 30 cached positions cannot hold 40 queries)
    assert s.layer.device_status() == rtp.RTP_DEV_BLOCKS | rtp.RTP_DEV_SEQ_LEN
    slots, cu = s.slots.cpu(), s.cu.tolist()
    assert s.length.tolist() == [48, 30, 16] and int(s.n_free) == 2 and cu == [0, 8, 48, 48]
    assert bool((slots[8:48] == -1).all()) and bool((slots[:8] >= 0).all())
    own = s.table[1, :2].long()
    assert torch.equal(s.layer.k.view(torch.uint8)[own], held[0][own]) and torch.equal(s.table[1], held[1][1])
    s.layer.status.zero_()
    s.step([1, 20, -1])  # a block from the third
    assert s.layer.device_status() == 0 and s.length.tolist() == [49, 50, 0] and int(s.n_free) == 0
    s.step([1, 17, 0], refused=(1,))  # here its newest 17 cached tokens answer in place of the new ones
    assert s.layer.device_status() == rtp.RTP_DEV_BLOCKS and s.length.tolist() == [50, 50, 0]
    assert s.slots[:19].lt(0).tolist() == [False] + [True] * 18


def test_lengths_that_fall_and_blocks_that_go_back():
    """Drafts of which some tokens are rejected: within a block, over one edge and over
    several; every block stays either a request's or free."""
    s = _Serving(3, 30, seed=52)
    bs, cols = s.bs, s.table.shape[1]

    def accounted():
        held = [int(x) for b in range(3) for x in s.table[b, :-(-int(s.length[b]) // bs)]]
        return sorted(held + s.free[:int(s.n_free)].tolist()) == list(range(30))

    def fall(to):
        """The lengths after verification; blocks behind them go back."""
        had, s.length = s.length, torch.tensor(to, dtype=torch.int32, device=DEV)
        keep, had = (s.length + bs - 1) // bs, (had + bs - 1) // bs
        at = (keep[:, None] + torch.arange(cols, device=DEV)).clamp_max(cols - 1)
        none = torch.empty(0, dtype=torch.int32, device=DEV)
        scratch = torch.empty(3, dtype=torch.int32, device=DEV)
        rtp.rtp_page_plan(s.layer.cfg, bs, ((had - keep) * bs).clamp_max(s.layer.cfg.max_ctx).int(), torch.full_like(scratch, -1), s.table.gather(1, at.long()).contiguous(),
                          s.free, s.n_free, scratch, torch.empty(4, dtype=torch.int32, device=DEV), none.long(), none, s.n_free, s.layer.status)

    s.step([30, 16, 47])
    for new, to in (([8, 8, 8], [33, 17, 48]), ([20, 40, 1], [33, 18, 49]), ([70, 15, 20], [35, 33, 49]), ([1, 1, 1], [36, 34, 50]),
                    ([16, 16, 16], [36, 34, 50]), ([13, 15, 15], [49, 49, 65])):
        s.step(new)
        assert accounted()
        fall(to)
        assert accounted()
    s.step([1, -1, 1])
    assert accounted() and s.layer.device_status() == 0


# ---------------------------------------------------------------------------
# rotary axes
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("D,sections,interleaved", [(64, (20, 12), False), (128, (10, 20, 30, 4), False), (64, (8, 12, 12), True),
                                                    (128, (16, 16, 16, 16), True), (128, (0, 64), False), (128, (1, 62, 1), True)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_two_to_four_axes_in_turn_or_dealt_out(D, sections, interleaved, dtype):
    rope = rtp.make_rope(D, sections, interleaved)
    axis = list(rope.axis[:D // 2])
    assert [axis.count(k) for k in range(len(sections))] == list(sections)
    gen = torch.Generator().manual_seed(D + len(sections))
    h = _Held(12, 2, 16, D, dtype, sections=sections)
    h.rope, h.axis = rope, axis
    for n, first in ((70, 3), (4, 73)):  # a chunk, a step
        h.append(torch.randn(n, 2, D, generator=gen).to(h.dt), torch.randn(n, 2, D, generator=gen).to(h.dt),
                 torch.arange(first, first + n), h.positions(n, gen))
        h.check()
    for new in ([1, 1], [3, 2], [60, 1]):
        a = _Attn([300, 90], new, D=D, hkv=2, G=4, bs=32, dtype=dtype, sections=sections, seed=61)
        a.rope, a.axis = rope, axis
        a.check(a.run(), rows={(0, 0), (0, new[0] - 1), (0, new[0] // 2), (1, 0)})


# ---------------------------------------------------------------------------
# batches
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("B,every", [(300, 7), (700, 31)])
def test_chunks_in_batches_of_more_than_256(B, every):
    """Idle, decoding and drafting requests, and chunks among them on both sides of 256."""
    new = [(0, 1, 1, 3, 1)[b % 5] if b % every else 9 + b % 40 for b in range(B)]
    lens = [n + (b * 37) % 150 + (n == 0) for b, n in enumerate(new)]
    a = _Attn(lens, new, D=64, hkv=2, G=4, bs=16, S=3, W=40, ret=(1,), seed=62, pad=11)
    got = a.run()
    some = {(b, t) for b, n in enumerate(new) if b % every == 0 or b % 17 == 0 or b > B - 4 for t in {0, n // 2, n - 1} if n}
    a.check(got, rows=some)
    assert bool((got[sum(new):] == 77.0).all()) and int(a.status) == 0


def test_a_batch_of_4096():
    """The largest that a plan takes: a token each, and the same with one chunk."""
    B = 4096
    for chunk in (0, 80):
        new = [1] * B
        new[3000] = max(1, chunk)
        lens = [n + b % 33 for b, n in enumerate(new)]
        a = _Attn(lens, new, D=64, hkv=1, G=2, bs=16, S=2, W=9, ret=(0,), seed=63)
        a.check(a.run(), rows={(b, 0) for b in range(0, B, 61)} | {(3000, t) for t in range(0, new[3000], 9)} | {(B - 1, 0)})
        assert int(a.status) == 0


@pytest.mark.parametrize("G,max_q", [(1, 40), (4, 200), (8, 7)])
def test_one_token_where_many_are_allowed(G, max_q):
    """Alone, and in rows of its own behind nothing: n_tokens below a chunk's tile of rows."""
    for lens, new in (([500], [1]), ([500, 33], [1, 0]), ([500], [2])):
        a = _Attn(lens, new, G=G, hkv=2, bs=32, seed=64)
        a.max_q = max_q
        a.check(a.run())
        assert int(a.status) == 0


def test_two_calls_at_once_and_in_graphs():
    """Two layers' calls of every kind, on two streams and replayed side by side: the
    bits of each alone."""
    made = []
    for seed, new in ((65, [1, 2, 1]), (66, [90, 1, 5])):
        a = _Attn([3000, 700, 90], new, bs=32, seed=seed).device()
        a.call()
        torch.cuda.synchronize()
        made.append((a, a.out.clone(), torch.cuda.Stream(), torch.cuda.CUDAGraph()))
        with torch.cuda.stream(made[-1][2]):
            with torch.cuda.graph(made[-1][3], stream=made[-1][2]):
                a.call()
    for how in ("calls", "graphs"):
        for a, _, _, _ in made:
            a.out.zero_()
            a.ws.fill_(0xA5)
        torch.cuda.synchronize()
        for _ in range(10):
            for a, _, s, g in made:
                with torch.cuda.stream(s):
                    g.replay() if how == "graphs" else a.call()
        torch.cuda.synchronize()
        for a, want, _, _ in made:
            assert torch.equal(a.out, want), how


@pytest.mark.parametrize("B,G", [(1, 4), (3, 8)])
def test_calls_in_which_no_request_has_a_query(B, G):
    """Rows behind the last stay as they were, with chunks allowed and without."""
    a = _Attn([50] * B, [0] * B, G=G, hkv=2, bs=16, seed=67, pad=5)
    for max_q in (1, 3, 40):
        a.max_q = max_q
        assert bool((a.run() == 77.0).all()) and int(a.status) == 0


def test_a_bare_description_of_no_block_size_is_refused():
    a = _Attn([50], [1], seed=68).device()
    cache = rtp.rtp_q8_cache(a.dk.data_ptr(), a.dv.data_ptr(), a.dks.data_ptr(), a.dvs.data_ptr(), a.status.data_ptr(), a.dk.shape[0], 0)
    with pytest.raises((ValueError, rtp.RtpError)):
        rtp.rtp_attn_q8(a.cfg, cache, a.dq, a.dcu, a.dlen, a.dtab, a.dpos, a.out, 1, 0, None, a.ws, a.ws.numel())
    with pytest.raises(rtp.RtpError):
        rtp.rtp_append_q8(a.cfg, cache, a.dq[:, :2].contiguous(), a.dq[:, :2].contiguous(), torch.zeros(1, dtype=torch.int64, device=DEV), a.dpos)
