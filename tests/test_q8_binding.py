"""CPU checks of what the binding of the paged 8-bit cache refuses before it
calls the library (nothing here launches a kernel).  CPU tensors count as
device -1, so the checks of a call's arguments are reached one by one."""

import pytest
import torch

import head_wise_sparse_local_b200 as rtp


def _cfg(**kw):
    base = dict(batch=2, n_q_heads=8, n_kv_heads=2, head_dim=64, max_ctx=256, n_sink=4, window=64, top_p=1.0, retrieval=(0,))
    base.update(kw)
    return rtp.make_cfg(**base)


def test_packed_rows_that_overlap_are_refused():
    """Above all a row that a broadcast repeats: its stride of 0 would mean
    dense rows to the library, which would read past the one row there is."""
    dt = torch.bfloat16
    for name, heads in (("k_pre", 2), ("v_in", 2), ("q_pre", 8)):
        one = torch.zeros(1, heads, 64, dtype=torch.bfloat16)
        with pytest.raises(ValueError, match=name):
            rtp._packed(one.expand(5, heads, 64), 64, dt, heads, name, -1)
        flat = torch.zeros(heads * 64 * 5, dtype=torch.bfloat16)
        with pytest.raises(ValueError, match=name):
            rtp._packed(flat.as_strided((3, heads, 64), (64, 64, 1)), 64, dt, heads, name, -1)
        # one row, dense rows, and slices of wider ones
        assert rtp._packed(one, 64, dt, heads, name, -1) == (one.data_ptr(), 0)
        assert rtp._packed(one.expand(1, heads, 64), 64, dt, heads, name, -1)[1] == 0
        assert rtp._packed(torch.zeros(3, heads, 64, dtype=torch.bfloat16), 64, dt, heads, name, -1)[1] == heads * 64
        wide = torch.zeros(3, 12 * 64, dtype=torch.bfloat16)[:, 128:128 + heads * 64].unflatten(1, (heads, 64))
        assert rtp._packed(wide, 64, dt, heads, name, -1)[1] == 12 * 64


class _FakeCuda:
    """What make_q8_cache asks of a tensor, on a device of the test's choice."""
    is_cuda = True

    def __init__(self, shape, dtype, index=0):
        self._x, self.device, self.shape, self.dtype = torch.empty(shape, dtype=dtype), torch.device("cuda", index), torch.Size(shape), dtype

    def __getattr__(self, name):
        return getattr(self._x, name)

    def get_device(self):
        return self.device.index


def _pool(monkeypatch, heads=2, D=64, status=((1,), torch.int32), devices=(0,) * 5):
    monkeypatch.setattr(rtp, "_ptr", lambda x: x.data_ptr())
    dt = torch.uint8
    return rtp.make_q8_cache(*(_FakeCuda(shape, t, i) for (shape, t), i in zip(
        (((3, heads, 32, D), dt), ((3, heads, 32, D), dt), ((3, heads), torch.float32), ((3, heads), torch.float32), status), devices)))


def test_a_pool_is_held_against_the_call(monkeypatch):
    cache = _pool(monkeypatch, devices=(1,) * 5)
    rtp._check_pool(cache, 2, 64, 1)
    for heads, D, dev in ((4, 64, 1), (1, 64, 1), (2, 128, 1), (2, 64, 0)):
        with pytest.raises(ValueError, match="pool"):
            rtp._check_pool(cache, heads, D, dev)
    rtp._check_pool(rtp.rtp_q8_cache(0, 0, 0, 0, 0, 3, 32), 2, 64, 0)  # bare addresses: the caller's word


def test_a_pool_of_several_devices_or_of_another_status_is_refused(monkeypatch):
    _pool(monkeypatch)
    for k in range(1, 5):
        with pytest.raises(ValueError, match="device"):
            _pool(monkeypatch, devices=tuple(int(i == k) for i in range(5)))
    for status in (((1,), torch.int64), ((2,), torch.int32), ((0,), torch.int32)):
        with pytest.raises(ValueError, match="status"):
            _pool(monkeypatch, status=status)


def test_table_rows_of_block_sizes_that_are_refused():
    assert [rtp._table_cols(_cfg(max_ctx=100), bs) for bs in (16, 128, 0, -64)] == [7, 1, 0, 0]
