"""Rows whose strides the paged calls do not take are refused by name, with the reason (no GPU)."""
import pytest
import torch

from tests.test_paged_host import _tensors, host, ra  # noqa: F401


def _bf(*s):
    return torch.zeros(s, dtype=torch.bfloat16)


BAD = [lambda h: _bf(5, 1, 64).expand(5, h, 64),                 # the same row for every head
       lambda h: _bf(1, h, 64).expand(5, h, 64),                 # and for every token
       lambda h: _bf(5, h, 65)[..., :64],                        # rows 65 elements apart
       lambda h: _bf(5 * h * 64 + 4)[4:].view(5, h, 64),         # on an 8-byte boundary
       lambda h: _bf(5 * h * 64).as_strided((5, h, 64), (h * 64, 32, 1))]  # rows that overlap


@pytest.mark.parametrize("bad", BAD)
def test_rows_are_refused_by_name(host, bad):  # noqa: F811
    x = _tensors()
    pool, batch = (x["k_cache"], x["v_cache"]), (x["block_table"], x["cu"], x["kv_len"])
    for name, k, v in (("k_new", bad(2), _bf(5, 2, 64)), ("v_new", _bf(5, 2, 64), bad(2))):
        with pytest.raises(ValueError, match=name + ".*multiples of 8"):
            host.cache_append(k, v, *pool, *batch)
    lse, ws = torch.zeros(5, 4), torch.zeros((1 << 24) + 256, dtype=torch.uint8)
    ws = ws[-ws.data_ptr() % 256:][:1 << 24]
    for name, q, out in (("q", bad(4), _bf(5, 4, 64)), ("out", _bf(5, 4, 64), bad(4))):
        with pytest.raises(ValueError, match=name + ".*multiples of 8"):
            host.fwd_paged(q, *pool, out, lse, *batch, ws, max_q=1)
