"""The numbers and the pool's description as the binding hands them to the library (no GPU)."""
import ctypes

import pytest
import torch

from tests.test_paged_host import _tensors, host, ra  # noqa: F401


def _call(host, **kw):
    x = _tensors()
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    return host.fwd_paged(bf(5, 4, 64), x["k_cache"], x["v_cache"], bf(5, 4, 64), torch.zeros(5, 4), x["block_table"], x["cu"],
                          x["kv_len"], torch.zeros(1 << 20, dtype=torch.uint8), **dict(dict(max_q=1), **kw))


@pytest.mark.parametrize("kw", [dict(window=2 ** 32 + 5), dict(window=2 ** 31), dict(sinks=2 ** 40), dict(max_q=2 ** 32 + 1),
                                dict(max_q=2 ** 31), dict(window=-2 ** 32 + 7), dict(causal=2 ** 32 + 1)])
def test_numbers_that_no_int_holds(host, kw):  # noqa: F811
    """They would reach the library without their upper bits, as other numbers."""
    with pytest.raises(ValueError, match="32-bit"):
        _call(host, **kw)


@pytest.mark.parametrize("args", [(2 ** 32 + 1, 1, 8, 2, 128, 1), (1, 1, 8, 2, 128, 2 ** 32 + 1), (1, 2 ** 33 + 3, 8, 2, 128, 1)])
def test_workspace_of_numbers_that_no_int_holds(ra, args):  # noqa: F811
    with pytest.raises(ValueError, match="32-bit"):
        ra.paged_workspace_bytes(*args)


@pytest.mark.parametrize("e4m3", [False, True])
def test_the_binding_packs_the_struct_of_the_header(host, e4m3):  # noqa: F811
    """Every value of the packed description, by the header's field of that name; no two alike."""
    n, h, page, d, batch, max_pages, total = 9, 2, 16, 64, 3, 4, 5
    dt = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    pool = lambda stride: torch.zeros(n * stride, dtype=torch.uint8 if e4m3 else torch.bfloat16).view(dt).as_strided(  # noqa: E731
        (n, h, page, d), (stride, page * d, d, 1))
    k, v = pool(h * page * d + 32), pool(h * page * d + 64)
    scale = lambda stride: torch.zeros(n * stride).as_strided((n, h, page), (stride, page, 1)) if e4m3 else None  # noqa: E731
    ks, vs = scale(h * page + 4), scale(h * page + 8)
    table = torch.zeros((batch, max_pages + 3), dtype=torch.int32)[:, :max_pages]
    cu, ln = torch.zeros(batch + 1, dtype=torch.int32), torch.zeros(batch, dtype=torch.int32)
    got_h, got_d, packed = host._paged(k, v, ks, vs, table, cu, ln, total, 0)
    assert (got_h, got_d) == (h, d)
    a = host._PagedKV.from_buffer_copy(packed)
    want = dict(k=k.data_ptr(), v=v.data_ptr(), k_scale=ks.data_ptr() if e4m3 else None, v_scale=vs.data_ptr() if e4m3 else None,
                block_table=table.data_ptr(), cu=cu.data_ptr(), kv_len=ln.data_ptr(), k_page_stride=h * page * d + 32,
                v_page_stride=h * page * d + 64, k_scale_page_stride=h * page + 4 if e4m3 else 0,
                v_scale_page_stride=h * page + 8 if e4m3 else 0, table_stride=max_pages + 3, n_pages=n, page_size=page, Hkv=h, d=d,
                dtype=int(e4m3), batch=batch, max_pages=max_pages, total=total)
    assert {f: getattr(a, f) for f, _ in host._PagedKV._fields_} == want
    assert len(packed) == ctypes.sizeof(host._PagedKV)
