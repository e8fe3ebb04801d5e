"""The paged cache on the host (no GPU): the oracle's pins and the refusals of the C ABI and the
binding."""
import ctypes
import os

import numpy as np
import pytest
import torch

from oracle import attention as oatt
from oracle import paged as opaged

F = 0x10000  # a 256-byte aligned address that is never dereferenced: every call must be refused first


@pytest.fixture(scope="module")
def ra():
    from online_softmax_attention_zigzag_gb300 import ringattn
    if not os.path.exists(ringattn.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return ringattn


# ------------------------------------------------------------------ the oracle
def test_oracle_attention_is_the_last_rows_of_full_attention():
    r = np.random.default_rng(0)
    q, k, v = r.normal(size=(37, 4, 8)), r.normal(size=(37, 2, 8)), r.normal(size=(37, 2, 8))
    fo, fl = oatt.full_attention(*(x.transpose(1, 0, 2) for x in (q, k, v)), True)
    out, lse, _, _ = opaged.attention(q[-5:], k, v)
    assert np.allclose(out, fo.transpose(1, 0, 2)[-5:], atol=1e-13)
    assert np.allclose(lse, fl.T[-5:], atol=1e-13)


def test_oracle_window_by_brute_force():
    for n, L, W, s in ((3, 11, 4, 2), (5, 3, 2, 1), (4, 9, 100, 3), (2, 8, 1, 0)):
        see = opaged.visible(n, L, True, W, s)
        for t in range(n):
            i = L - n + t
            assert [j for j in range(L) if see[t, j]] == [j for j in range(L) if j <= i and (j > i - W or j < s)]


def test_oracle_rows_without_keys():
    out, lse, _, _ = opaged.attention(np.ones((4, 2, 8)), np.ones((2, 1, 8)), np.ones((2, 1, 8)))
    assert np.isneginf(lse[:2]).all() and not out[:2].any() and np.allclose(out[2:], 1.0)


def test_oracle_quantise_against_the_table_of_e4m3_numbers():
    """Every code by nearest search among the 127 non-negative e4m3 numbers, ties to even codes."""
    table = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    x = torch.randn((200, 64), generator=torch.Generator().manual_seed(3))
    x = (x * torch.exp2(torch.arange(200).float()[:, None] - 100)).to(torch.bfloat16).double().numpy()
    codes, scale = opaged.quantise(x)
    assert (np.log2(scale) == np.round(np.log2(scale))).all()
    y = np.abs(x / scale[:, None])
    assert (y.max(1) <= 448).all() and (y.max(1)[scale > 2.0 ** -120] > 224).all()
    for a, c in zip(y.ravel()[::7], np.abs(codes).ravel()[::7]):
        d = np.abs(table - a)
        near = np.nonzero(d == d.min())[0]
        assert c == table[near[near % 2 == 0][0] if len(near) > 1 else near[0]]
    t = torch.from_numpy(x / scale[:, None]).float().to(torch.float8_e4m3fn)
    assert np.array_equal(t.double().numpy(), codes)


# ------------------------------------------------------------------ refusals of the C ABI
def _kv(ra, **kw):
    a = ra._PagedKV()
    base = dict(k=F, v=2 * F, k_scale=0, v_scale=0, block_table=3 * F, cu=4 * F, kv_len=5 * F, n_pages=10, page_size=32,
                Hkv=2, d=128, dtype=0, batch=3, max_pages=7, total=5)
    base.update(kw)
    rows = base["Hkv"] * base["page_size"]
    base.setdefault("k_page_stride", rows * base["d"])
    base.setdefault("v_page_stride", rows * base["d"])
    base.setdefault("k_scale_page_stride", rows)
    base.setdefault("v_scale_page_stride", rows)
    base.setdefault("table_stride", base["max_pages"])
    for n, v in base.items():
        setattr(a, n, v)
    return a


BAD_KV = [
    (dict(k=0), -1), (dict(v=0), -1), (dict(v=F), -1), (dict(k=F + 8), -1), (dict(v=F + 8), -1), (dict(block_table=0), -1),
    (dict(cu=0), -1), (dict(kv_len=0), -1), (dict(cu=F + 2), -1), (dict(block_table=F + 1), -1), (dict(kv_len=F + 2), -1),
    (dict(k_scale=F), -1), (dict(v_scale=F), -1), (dict(dtype=1), -1), (dict(dtype=1, k_scale=F), -1), (dict(dtype=2), -1),
    (dict(dtype=1, k_scale=F, v_scale=F + 2), -1), (dict(n_pages=0), -1), (dict(page_size=0), -1), (dict(Hkv=0), -1),
    (dict(d=0), -1), (dict(batch=0), -1), (dict(max_pages=0), -1), (dict(total=-1), -1), (dict(d=96), -2),
    (dict(page_size=24), -2), (dict(page_size=65552), -2), (dict(batch=4097), -2), (dict(max_pages=2 ** 30), -2),
    (dict(k_page_stride=2 * 32 * 128 - 8), -1), (dict(v_page_stride=2 * 32 * 128 + 4), -1), (dict(table_stride=6), -1),
    (dict(dtype=1, k_scale=F, v_scale=F, k_page_stride=2 * 32 * 128 + 8), -1),
    (dict(dtype=1, k_scale=F, v_scale=F, k_scale_page_stride=63), -1), (dict(k_page_stride=2 ** 36 + 8), -2),
]


@pytest.mark.parametrize("kw,want", BAD_KV)
def test_pool_and_batch_are_refused(ra, kw, want):
    L, a = ra.lib(), _kv(ra, **kw)
    r = ctypes.byref(a)
    assert L.ringattn_cache_append(F, F, 256, 128, 256, 128, r, 0) == want
    assert L.ringattn_cache_read(r, F, F, 0) == want
    assert L.ringattn_fwd_paged(F, 512, 128, r, F, 512, 128, 0, F, 4, 1, 4, 1, 1, 0, 0, F, 1 << 40, 0) == want


def test_no_pool_at_all(ra):
    L = ra.lib()
    assert L.ringattn_cache_append(F, F, 256, 128, 256, 128, None, 0) == -1
    assert L.ringattn_cache_read(None, F, F, 0) == -1
    assert L.ringattn_fwd_paged(F, 512, 128, None, F, 512, 128, 0, F, 4, 1, 4, 1, 1, 0, 0, F, 1 << 40, 0) == -1


def test_nothing_to_do_needs_no_device(ra):
    L, a = ra.lib(), _kv(ra, total=0)
    r = ctypes.byref(a)
    assert L.ringattn_cache_append(None, None, 0, 0, 0, 0, r, 0) == 0
    assert L.ringattn_cache_read(r, None, None, 0) == 0
    assert L.ringattn_fwd_paged(None, 0, 0, r, None, 0, 0, 0, None, 0, 0, 4, 1, 1, 0, 0, None, 0, 0) == 0


@pytest.mark.parametrize("args", [
    (0, F, 256, 128, 256, 128), (F, 0, 256, 128, 256, 128), (F + 8, F, 256, 128, 256, 128), (F, F + 2, 256, 128, 256, 128),
    (F, F, 252, 128, 256, 128), (F, F, 256, 132, 256, 128), (F, F, 256, 128, -256, 128), (F, F, 256, 128, 256, 2 ** 33),
    (F, F, 0, 128, 256, 128), (F, F, 256, 64, 256, 128),
])
def test_append_refuses_rows(ra, args):
    assert ra.lib().ringattn_cache_append(*args, ctypes.byref(_kv(ra)), 0) == -1


def test_too_many_rows(ra):
    L = ra.lib()
    a = _kv(ra, total=2 ** 30, Hkv=2)
    assert L.ringattn_cache_append(F, F, 256, 128, 256, 128, ctypes.byref(a), 0) == -2
    assert L.ringattn_cache_read(ctypes.byref(a), F, F, 0) == -2
    assert L.ringattn_fwd_paged(F, 512, 128, ctypes.byref(a), F, 512, 128, 0, F, 4, 1, 4, 1, 1, 0, 0, F, 1 << 40, 0) == -2


def test_more_rows_than_positions(ra):
    L, a = ra.lib(), _kv(ra, total=2 ** 30 + 1, Hkv=1)  # (one head: no other limit says no)
    r = ctypes.byref(a)
    assert L.ringattn_cache_append(F, F, 256, 128, 256, 128, r, 0) == -2
    assert L.ringattn_cache_read(r, F, F, 0) == -2
    assert L.ringattn_fwd_paged(F, 512, 128, r, F, 512, 128, 0, F, 1, 1, 1, 1, 1, 0, 0, F, 1 << 40, 0) == -2


def test_read_refuses_outputs(ra):
    L, a = ra.lib(), _kv(ra)
    for k, v in ((0, F), (F, 0), (F + 4, F), (F, F + 8)):
        assert L.ringattn_cache_read(ctypes.byref(a), k, v, 0) == -1


ATT = dict(q=F, qt=512, qh=128, out=F, ot=512, oh=128, f32=0, lse=F, lt=4, lh=1, Hq=4, max_q=1, causal=1, window=0,
           sinks=0, ws=F, bytes=1 << 40)


@pytest.mark.parametrize("kw,want", [
    (dict(q=0), -1), (dict(out=0), -1), (dict(lse=0), -1), (dict(ws=0), -1), (dict(q=F + 8), -1), (dict(out=F + 8), -1),
    (dict(lse=F + 2), -1), (dict(ws=F + 16), -1), (dict(bytes=0), -1), (dict(bytes=-1), -1), (dict(Hq=5), -1), (dict(Hq=0), -1),
    (dict(max_q=0), -1), (dict(causal=2), -1), (dict(causal=0, window=5), -1), (dict(window=-1), -1), (dict(sinks=-1), -1),
    (dict(f32=2), -1), (dict(qt=516), -1), (dict(oh=64), -1), (dict(lt=0), -1), (dict(lh=0), -1), (dict(Hq=258), -2),
])
def test_attention_refuses(ra, kw, want):
    c = dict(ATT, **kw)
    got = ra.lib().ringattn_fwd_paged(c["q"], c["qt"], c["qh"], ctypes.byref(_kv(ra)), c["out"], c["ot"], c["oh"], c["f32"],
                                      c["lse"], c["lt"], c["lh"], c["Hq"], c["max_q"], c["causal"], c["window"], c["sinks"],
                                      c["ws"], c["bytes"], 0)
    assert got == want


def test_workspace_bytes(ra):
    L, n = ra.lib(), ctypes.c_longlong(0)
    assert ra.paged_workspace_bytes(1, 1, 8, 2, 128, 1) > 0
    assert L.ringattn_paged_workspace_bytes(1, 1, 8, 2, 128, 1, None) == -1
    for bad in ((-1, 1, 8, 2, 128, 1), (1, 0, 8, 2, 128, 1), (1, 1, 8, 3, 128, 1), (1, 1, 0, 2, 128, 1), (1, 1, 8, 2, 0, 1),
                (1, 1, 8, 2, 128, 0)):
        assert L.ringattn_paged_workspace_bytes(*bad, ctypes.byref(n)) == -1


def test_header_and_binding_agree(ra):
    import re
    hdr = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "ringattn.h")).read()
    assert int(re.search(r"#define RINGATTN_PAGED_MAX_BATCH (\d+)", hdr).group(1)) == ra.PAGED_MAX_BATCH
    fields = re.search(r"typedef struct \{(.*?)\} ra_paged_kv;", hdr, re.S).group(1)
    names = [n for decl in re.sub(r"/\*.*?\*/", "", fields, flags=re.S).split(";") for n in re.findall(r"(\w+)\s*(?:,|$)", decl.strip())]
    assert names == [n for n, _ in ra._PagedKV._fields_]
    import struct
    assert struct.calcsize("7P5q8i") == ctypes.sizeof(ra._PagedKV)  # the order that the binding packs


# ------------------------------------------------------------------ refusals of the binding
@pytest.fixture
def host(ra, monkeypatch):
    """CPU tensors stand for the device's: the checks run, the library refuses or is not reached."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 0)
    monkeypatch.setattr(ra, "_raw_stream", lambda s, dev: 0)
    return ra


def _tensors(e4m3=False):
    t = torch
    dt = t.float8_e4m3fn if e4m3 else t.bfloat16
    x = dict(k_cache=t.zeros((9, 2, 16, 64)).to(dt), v_cache=t.zeros((9, 2, 16, 64)).to(dt),
             block_table=t.zeros((3, 4), dtype=t.int32), cu=t.zeros(4, dtype=t.int32), kv_len=t.zeros(3, dtype=t.int32))
    if e4m3:
        x.update(k_scale=t.zeros((9, 2, 16)), v_scale=t.zeros((9, 2, 16)))
    return x


@pytest.mark.parametrize("change,match", [
    (dict(k_cache=torch.zeros((9, 2, 16, 64))), "bfloat16"),
    (dict(v_cache=torch.zeros((9, 2, 16, 64)).to(torch.float8_e4m3fn)), "bfloat16"),
    (dict(v_cache=torch.zeros((9, 2, 32, 64)).to(torch.bfloat16)), "same shape"),
    (dict(k_cache=torch.zeros((9, 2, 64, 16)).to(torch.bfloat16).transpose(2, 3)), "contiguous"),
    (dict(k_cache=torch.zeros((9, 16, 2, 64)).to(torch.bfloat16).transpose(1, 2)), "contiguous"),
    (dict(k_scale=torch.zeros((9, 2, 16))), "has none"),
    (dict(block_table=torch.zeros((3, 4), dtype=torch.int64)), "int32"),
    (dict(block_table=torch.zeros((12,), dtype=torch.int32)), "2 axes"),
    (dict(cu=torch.zeros(3, dtype=torch.int32)), "batch"),
    (dict(kv_len=torch.zeros(4, dtype=torch.int32)), "batch"),
])
def test_binding_refuses_pool_and_batch(host, change, match):
    x = dict(_tensors(), **change)
    x = dict(dict(k_scale=None, v_scale=None), **x)
    rows = torch.zeros((5, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match=match):
        host.cache_append(rows, rows, x["k_cache"], x["v_cache"], x["block_table"], x["cu"], x["kv_len"],
                          k_scale=x["k_scale"], v_scale=x["v_scale"])


def test_binding_refuses_rows_and_outputs(host):
    x = _tensors()
    pool = (x["k_cache"], x["v_cache"])
    batch = (x["block_table"], x["cu"], x["kv_len"])
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    for k, v in ((bf(5, 3, 64), bf(5, 3, 64)), (bf(5, 2, 64), bf(6, 2, 64)), (bf(5, 2, 128), bf(5, 2, 128)),
                 (torch.zeros(5, 2, 64), bf(5, 2, 64)), (bf(10, 64), bf(10, 64)), (bf(5, 2, 128)[..., ::2], bf(5, 2, 64))):
        with pytest.raises(ValueError):
            host.cache_append(k, v, *pool, *batch)
    for k, v in ((bf(3, 5, 64), bf(3, 5, 64)), (bf(2, 5, 64), bf(2, 6, 64)), (bf(5, 2, 64).transpose(0, 1), bf(2, 5, 64))):
        with pytest.raises(ValueError):
            host.cache_read(*pool, k, v, *batch)
    q, out, lse, ws = bf(5, 4, 64), bf(5, 4, 64), torch.zeros(5, 4), torch.zeros(1 << 20, dtype=torch.uint8)
    for bad in (dict(q=bf(5, 4, 128)), dict(out=bf(5, 3, 64)), dict(out=torch.zeros(5, 4, 64, dtype=torch.float16)),
                dict(lse=torch.zeros(4, 5)), dict(lse=torch.zeros(5, 4, dtype=torch.float64)), dict(ws=torch.zeros(4096))):
        a = dict(dict(q=q, out=out, lse=lse, ws=ws), **bad)
        with pytest.raises(ValueError):
            host.fwd_paged(a["q"], *pool, a["out"], a["lse"], *batch, a["ws"], max_q=1)
    with pytest.raises(host.RingAttnError):  # the library's refusal comes through as its error
        host.fwd_paged(q, *pool, out, lse, *batch, ws, max_q=1, window=-1)


def test_binding_refuses_another_device(host, monkeypatch):
    x = _tensors()
    rows = torch.zeros((5, 2, 64), dtype=torch.bfloat16)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError, match="current device"):
        host.cache_append(rows, rows, x["k_cache"], x["v_cache"], x["block_table"], x["cu"], x["kv_len"])


def test_binding_refuses_host_tensors(ra, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    x = _tensors()
    rows = torch.zeros((5, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        ra.cache_append(rows, rows, x["k_cache"], x["v_cache"], x["block_table"], x["cu"], x["kv_len"])
