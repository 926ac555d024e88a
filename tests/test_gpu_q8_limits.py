"""The paged 8-bit cache at the ends of what its calls allow: configuration
values, value and query sizes, batches, rotary axes, streams, lengths that
fall.  The references and the bounds are those of tests/test_gpu_q8.py unless
a test gives its own."""

import pytest
import torch

import head_wise_sparse_local_b200 as rtp
import q8_reference as ref
from test_gpu_q8 import _Attn

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
