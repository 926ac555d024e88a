"""CPU checks of the paged 8-bit cache's entry points: sizes, and every argument
that the host refuses (no call here reaches a kernel launch)."""

import pytest
import torch

import head_wise_sparse_local_b200 as rtp

FAKE = 1 << 20  # an address that validation never follows


def _cfg(**kw):
    base = dict(batch=2, n_q_heads=32, n_kv_heads=8, head_dim=128, max_ctx=4096, n_sink=64, window=2048, top_p=1.0,
                retrieval=(0, 5), dtype="bf16")
    base.update(kw)
    return rtp.make_cfg(**base)


def _cache(**kw):
    base = dict(k=FAKE, v=FAKE, k_scale=FAKE, v_scale=FAKE, status=FAKE, n_blocks=100, block_size=64)
    base.update(kw)
    return rtp.rtp_q8_cache(*base.values())


def _append(cfg=None, cache=None, k=FAKE, ks=0, v=FAKE, vs=0, slot=FAKE, pos=FAKE, rope=None, n=4):
    from head_wise_sparse_local_b200 import _abi
    import ctypes
    _abi.check(_abi.load().rtp_append_q8(ctypes.byref(cfg or _cfg()), ctypes.byref(cache or _cache()), k, ks, v, vs, slot, pos,
                                         None if rope is None else ctypes.byref(rope), n, None))


def _attn(cfg=None, cache=None, q=FAKE, qs=0, cu=FAKE, seq=FAKE, tab=FAKE, pos=FAKE, rope=None, n=4, max_q=2, max_seq=0, out=FAKE,
          ws=FAKE, ws_bytes=1 << 40):
    from head_wise_sparse_local_b200 import _abi
    import ctypes
    _abi.check(_abi.load().rtp_attn_q8(ctypes.byref(cfg or _cfg()), ctypes.byref(cache or _cache()), q, qs, cu, seq, tab, pos,
                                       None if rope is None else ctypes.byref(rope), n, max_q, max_seq, out, ws, ws_bytes, None))


def _plan(cfg=None, bs=64, max_tokens=16, free_cap=10, slots=FAKE, **kw):
    from head_wise_sparse_local_b200 import _abi
    import ctypes
    p = dict(ctx=FAKE, new=FAKE, table=FAKE, free=FAKE, n_free=FAKE, seq=FAKE, cu=FAKE, pos=FAKE, n_out=FAKE, status=FAKE)
    p.update(kw)
    _abi.check(_abi.load().rtp_page_plan(ctypes.byref(cfg or _cfg()), bs, p["ctx"], p["new"], p["table"], p["free"], free_cap,
                                         p["n_free"], p["seq"], p["cu"], slots, p["pos"], max_tokens, p["n_out"], p["status"], None))


def _refused(code, f, *a, **kw):
    with pytest.raises(rtp.RtpError) as e:
        f(*a, **kw)
    assert e.value.code == code and rtp.rtp_last_error() != ""


def test_pool_sizes():
    kv, sc = rtp.rtp_q8_cache_bytes(_cfg(), 100, 64)
    assert kv == 100 * 8 * 64 * 128 and sc == 100 * 8 * 4
    kv32, _ = rtp.rtp_q8_cache_bytes(_cfg(dtype="fp32"), 100, 64)
    assert kv32 == kv  # the pool is 8 bits whatever the layer's type


@pytest.mark.parametrize("kw", [dict(top_p=0.9), dict(top_k=5), dict(local_cap=3000), dict(head_dim=96)])
def test_configurations_that_the_paged_cache_does_not_take(kw):
    for f in (lambda c: rtp.rtp_q8_cache_bytes(c, 10, 64), lambda c: rtp.rtp_attn_q8_workspace_bytes(c, 64, 1, 1),
              lambda c: _append(cfg=c), lambda c: _attn(cfg=c), lambda c: _plan(cfg=c)):
        _refused(2, f, _cfg(**kw))


@pytest.mark.parametrize("bs", [0, 8, 48, 256, -64])
def test_block_sizes(bs):
    _refused(2, rtp.rtp_q8_cache_bytes, _cfg(), 10, bs)
    _refused(2, _plan, bs=bs)
    _refused(2, _append, cache=_cache(block_size=bs))
    _refused(2, _attn, cache=_cache(block_size=bs))


def test_pool_refusals():
    for f in (_append, _attn):
        _refused(2, f, cache=_cache(n_blocks=0))
        _refused(2, f, cache=_cache(n_blocks=(1 << 31) // (8 * 64)))
        for name in ("k", "v", "k_scale", "v_scale", "status"):
            _refused(1, f, cache=_cache(**{name: None}))
        for name in ("k", "v", "k_scale", "v_scale"):
            _refused(1, f, cache=_cache(**{name: FAKE + 8}))
    _refused(2, rtp.rtp_q8_cache_bytes, _cfg(), 0, 64)
    _refused(2, rtp.rtp_q8_cache_bytes, _cfg(), (1 << 31) // (8 * 64), 64)


def test_append_refusals():
    for name in ("k", "v", "slot", "pos"):
        _refused(1, _append, **{name: None})
    for name in ("k", "v"):
        _refused(1, _append, **{name: FAKE + 2})
    for name in ("ks", "vs"):
        _refused(2, _append, **{name: 8 * 128 - 8})  # rows would overlap
        _refused(2, _append, **{name: 8 * 128 + 4})  # not 16 bytes apart
        _refused(2, _append, **{name: -2048})
    _refused(2, _append, n=-1)
    bad = rtp.make_rope(128, (16, 24, 24))
    bad.n_axes = 2  # names axis 2
    _refused(2, _append, rope=bad)
    bad.n_axes = 5
    _refused(2, _append, rope=bad)
    _append(n=0, k=None, v=None, slot=None, pos=None)  # nothing to do


def test_attn_refusals():
    for name in ("q", "cu", "seq", "tab", "pos", "out"):
        _refused(1, _attn, **{name: None})
    _refused(1, _attn, q=FAKE + 2)
    _refused(1, _attn, out=FAKE + 2)
    _refused(2, _attn, qs=32 * 128 - 8)
    _refused(2, _attn, n=-1)
    _refused(2, _attn, max_q=0)
    _refused(2, _attn, max_q=4097)
    _refused(2, _attn, max_seq=4097)
    _refused(2, _attn, max_seq=-1)
    _refused(4, _attn, ws=None)
    _refused(4, _attn, ws=FAKE + 16)
    need = rtp.rtp_attn_q8_workspace_bytes(_cfg(), 64, 4, 2)
    _refused(4, _attn, ws_bytes=need - 1)
    _attn(n=0, q=None, cu=None, seq=None, tab=None, pos=None, out=None, ws=None)


def test_plan_refusals():
    for name in ("ctx", "new", "table", "free", "n_free", "seq", "cu", "pos", "n_out", "status"):
        _refused(1, _plan, **{name: None})
    _refused(1, _plan, slots=None)
    _refused(1, _plan, slots=FAKE + 8)
    _refused(1, _plan, pos=FAKE + 4)
    _refused(2, _plan, max_tokens=-1)
    _refused(2, _plan, free_cap=-1)
    _refused(2, _plan, cfg=_cfg(batch=4097))


def test_workspace_grows_with_the_call():
    cfg = _cfg(batch=64)
    sizes = [rtp.rtp_attn_q8_workspace_bytes(cfg, 64, n, 1) for n in (1, 8, 64)]
    assert sizes == sorted(sizes) and sizes[0] > 0 and all(s % 256 == 0 for s in sizes)
    _refused(2, rtp.rtp_attn_q8_workspace_bytes, cfg, 64, -1, 1)


def test_rope_axes():
    r = rtp.make_rope(128, (16, 24, 24))
    assert r.n_axes == 3 and list(r.axis[:64]) == [0] * 16 + [1] * 24 + [2] * 24
    r = rtp.make_rope(64, (8, 12, 12), interleaved=True)
    ax = list(r.axis[:32])
    assert ax[:6] == [0, 1, 2, 0, 1, 2] and [ax.count(a) for a in range(3)] == [8, 12, 12]
    for bad in ((16, 24), (64, 1), (), (-1, 65)):
        with pytest.raises(ValueError):
            rtp.make_rope(128, bad)


def test_binding_checks_tensors_before_the_call():
    cfg, cache = _cfg(), _cache()
    x = torch.zeros(4, 8, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):  # a CPU tensor
        rtp.rtp_append_q8(cfg, cache, x, x, torch.zeros(4, dtype=torch.int64), torch.zeros(1, 4, dtype=torch.int32))
    with pytest.raises(ValueError):  # a pool of two bytes an element
        k = torch.zeros(3, 8, 64, 128, dtype=torch.bfloat16)
        rtp.make_q8_cache(k, k, torch.ones(3, 8), torch.ones(3, 8), torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError):  # scales of another shape
        k = torch.zeros(3, 8, 64, 128, dtype=torch.uint8)
        rtp.make_q8_cache(k, k, torch.ones(3, 4), torch.ones(3, 8), torch.zeros(1, dtype=torch.int32))


def test_attention_line_stays_below_2_31():
    # 4096 requests x 8 KV heads x 2^15 tiles of 32 positions: 2^30 a 16-row chunk of queries
    big = _cfg(batch=4096, max_ctx=1 << 20)
    rtp.rtp_attn_q8_workspace_bytes(big, 64, 4096, 1)
    rtp.rtp_attn_q8_workspace_bytes(big, 64, 4096, 4)  # 16 rows
    _refused(2, rtp.rtp_attn_q8_workspace_bytes, big, 64, 8192, 8)  # 32 rows: two chunks
    rtp.rtp_attn_q8_workspace_bytes(big, 64, 8192, 8, 1 << 19)
    _refused(2, _attn, cfg=big, n=8192, max_q=8)
    fp32 = _cfg(batch=4096, max_ctx=1 << 20, dtype="fp32")
    rtp.rtp_attn_q8_workspace_bytes(fp32, 64, 4096, 2)  # 8 rows
    _refused(2, rtp.rtp_attn_q8_workspace_bytes, fp32, 64, 8192, 3)
