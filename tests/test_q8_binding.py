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
    cfg = _cfg()
    for name, heads in (("k_pre", 2), ("v_in", 2), ("q_pre", 8)):
        one = torch.zeros(1, heads, 64, dtype=torch.bfloat16)
        with pytest.raises(ValueError, match=name):
            rtp._packed(one.expand(5, heads, 64), cfg, heads, name, -1)
        flat = torch.zeros(heads * 64 * 5, dtype=torch.bfloat16)
        with pytest.raises(ValueError, match=name):
            rtp._packed(flat.as_strided((3, heads, 64), (64, 64, 1)), cfg, heads, name, -1)
        # one row, dense rows, and slices of wider ones
        assert rtp._packed(one, cfg, heads, name, -1) == (one.data_ptr(), 0)
        assert rtp._packed(one.expand(1, heads, 64), cfg, heads, name, -1)[1] == 0
        assert rtp._packed(torch.zeros(3, heads, 64, dtype=torch.bfloat16), cfg, heads, name, -1)[1] == heads * 64
        wide = torch.zeros(3, 12 * 64, dtype=torch.bfloat16)[:, 128:128 + heads * 64].unflatten(1, (heads, 64))
        assert rtp._packed(wide, cfg, heads, name, -1)[1] == 12 * 64
