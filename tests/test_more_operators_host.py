"""Norm and rotation of q and k, attention weights a cached position, eviction, on the host (no GPU): the oracle's pins and
the refusals of the C ABI and the binding."""
import ctypes
import math
import os

import numpy as np
import pytest
import torch

from oracle import attention as oatt
from oracle import evict as oevict
from oracle import qk_norm as onorm
from tests.test_paged_host import BAD_KV, F, _kv


@pytest.fixture(scope="module")
def ra():
    from online_softmax_attention_zigzag_gb300 import ringattn
    if not os.path.exists(ringattn.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return ringattn


# ------------------------------------------------------------------ the oracle
@pytest.mark.parametrize("interleaved", [False, True])
def test_oracle_norm_by_brute_force(interleaved):
    r = np.random.default_rng(0)
    d, rot, pos = 12, 8, 5
    x, w = r.normal(size=d), r.normal(size=d)
    angle = [pos * 100.0 ** (-2 * j / rot) for j in range(rot // 2)]
    table = np.array([[math.cos(a) for a in angle] + [math.sin(a) for a in angle]])
    z, _ = onorm.forward(x[None, None], w, table, interleaved, 0.1, 0.5)
    rms = math.sqrt(sum(v * v for v in x) / d + 0.1)
    y = [a * b / rms for a, b in zip(x, w)]
    want = list(y)
    for j in range(rot // 2):
        a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + rot // 2)
        t = complex(y[a], y[b]) * complex(math.cos(angle[j]), math.sin(angle[j]))
        want[a], want[b] = t.real, t.imag
    assert np.allclose(z[0, 0], np.array(want) * 0.5, atol=1e-13)


def test_oracle_rotation_makes_scores_depend_on_the_distance_alone():
    r = np.random.default_rng(1)
    q, k = r.normal(size=(1, 1, 16)), r.normal(size=(1, 1, 16))
    angle = np.arange(40)[:, None] * 10.0 ** (-np.arange(4) / 2)[None]
    table = np.concatenate([np.cos(angle), np.sin(angle)], 1)

    def score(i, j):
        return float((onorm.forward(q, None, table[i:i + 1])[0] * onorm.forward(k, None, table[j:j + 1])[0]).sum())

    assert abs(score(30, 25) - score(7, 2)) < 1e-12 and abs(score(30, 25) - score(30, 24)) > 1e-3


@pytest.mark.parametrize("interleaved", [False, True])
def test_oracle_norm_gradients_against_differences_and_autograd(interleaved):
    r = np.random.default_rng(2)
    T, H, d, rot = 3, 2, 8, 4
    x, w, dz, table = r.normal(size=(T, H, d)), r.normal(size=d), r.normal(size=(T, H, d)), r.normal(size=(T, rot))
    dx, dw, dx_abs, dw_abs = onorm.backward(x, w, table, dz, interleaved, 0.01, 0.7)

    def f(x, w):
        return (onorm.forward(x, w, table, interleaved, 0.01, 0.7)[0] * dz).sum()

    for at in np.ndindex(T, H, d):
        e = np.zeros_like(x)
        e[at] = 1e-5
        assert abs((f(x + e, w) - f(x - e, w)) / 2e-5 - dx[at]) < 1e-8
    for i in range(d):
        e = np.zeros(d)
        e[i] = 1e-5
        assert abs((f(x, w + e) - f(x, w - e)) / 2e-5 - dw[i]) < 1e-8
    assert (dx_abs >= np.abs(dx) - 1e-12).all() and (dw_abs >= np.abs(dw) - 1e-12).all()
    xt, wt = torch.from_numpy(x).requires_grad_(), torch.from_numpy(w).requires_grad_()
    y = wt * xt * (xt.square().mean(-1, keepdim=True) + 0.01).rsqrt() * 0.7
    z = torch.einsum("tij,thj->thi", torch.from_numpy(onorm.turn_matrix(table, d, interleaved)), y)
    gx, gw = torch.autograd.grad(z, (xt, wt), torch.from_numpy(dz))
    assert np.allclose(gx.numpy(), dx, atol=1e-13) and np.allclose(gw.numpy(), dw, atol=1e-13)


def test_oracle_weights_are_the_columns_of_the_attention_matrix():
    """Every row's weights add up to 1, and v = the identity shows the matrix itself."""
    r = np.random.default_rng(3)
    n, L, hq, hkv, d = 5, 11, 4, 2, 11
    q, k = r.normal(size=(L, hq, d)), r.normal(size=(L, hkv, d))
    eye = np.broadcast_to(np.eye(L)[:, None, :], (L, hkv, L))
    out, lse = oatt.full_attention(q.transpose(1, 0, 2), k.transpose(1, 0, 2), eye.transpose(1, 0, 2), True)
    old = r.random((L, hkv))
    new, _ = oevict.add_weights(old, q[-n:], lse.T[-n:], k, 0.5)
    want = np.where(np.arange(L)[:, None] < L - n, 0.5 * old, 0.0)
    for h in range(hq):
        want[:, h // 2] += out[h, -n:].sum(0)
    assert np.allclose(new, want, atol=1e-13)
    new, _ = oevict.add_weights(old, q[-n:], lse.T[-n:], k, 0.0)
    assert np.allclose(new.sum(0), n * hq / hkv)
    assert np.array_equal(oevict.add_weights(old, q[:0], lse.T[:0], k, 0.0)[0], old)


def test_oracle_weights_under_a_window_by_brute_force():
    r = np.random.default_rng(4)
    q, k, lse = r.normal(size=(3, 1, 8)), r.normal(size=(9, 1, 8)), r.normal(size=(3, 1))
    lse[1] = -np.inf
    new, _ = oevict.add_weights(np.zeros((9, 1)), q, lse, k, 1.0, True, 4, 2)
    for j in range(9):
        want = sum(math.exp(float(q[t, 0] @ k[j, 0]) - lse[t, 0]) for t in (0, 2) if j <= 6 + t and (j > 6 + t - 4 or j < 2))
        assert abs(new[j, 0] - want) < 1e-12


def test_oracle_eviction():
    nan, inf = float("nan"), float("inf")
    assert oevict.stay([1, 5, 3, 5, 2], 3) == [1, 2, 3]
    assert oevict.stay([1, 5, 3, 5, 5], 2) == [1, 3]
    assert oevict.stay([1, 5, 3, 5, 5], 3, sinks=1, recent=1) == [0, 1, 4]
    assert oevict.stay([0, -0.0, 0, 0], 2) == [0, 1]
    assert oevict.stay([1, nan, inf, 2, -inf], 3) == [1, 2, 3]
    assert oevict.stay([1, 2, 3, 4], 2, sinks=3, recent=1) == [0, 1]
    assert oevict.stay([1, 2], 9) == [0, 1] and oevict.stay([1, 2], 0) == []


# ------------------------------------------------------------------ refusals of the C ABI
def _rows(ra, **kw):
    base = dict(q=F, k=2 * F, q_token_stride=512, q_head_stride=128, k_token_stride=256, k_head_stride=128, dtype=0)
    base.update(kw)
    return ra._pack_qk_rows(*(base[n] for n in ("q", "k", "q_token_stride", "q_head_stride", "k_token_stride", "k_head_stride", "dtype")))


def _norm(ra, **kw):
    base = dict(q_weight=F, k_weight=F, cos_sin=F, position=F, total=5, Hq=4, Hkv=2, d=128, rot=64, n_pos=10, weight_f32=0,
                interleaved=0, eps=1e-6, q_scale=1.0)
    base.update(kw)
    return ra._pack_qk_norm(*base.values())


BAD_NORM = [
    (dict(total=-1), -1), (dict(Hq=0), -1), (dict(Hkv=0), -1), (dict(d=0), -1), (dict(rot=-16), -1), (dict(rot=144), -1),
    (dict(n_pos=0), -1), (dict(weight_f32=2), -1), (dict(interleaved=-1), -1), (dict(eps=-1e-9), -1), (dict(eps=math.nan), -1),
    (dict(eps=math.inf), -1), (dict(q_scale=math.nan), -1), (dict(q_scale=-math.inf), -1), (dict(q_weight=F + 8), -1),
    (dict(k_weight=F + 2), -1), (dict(cos_sin=F + 4), -1), (dict(cos_sin=0), -1), (dict(position=0), -1), (dict(position=F + 1), -1),
    (dict(d=96), -2), (dict(rot=24), -2), (dict(total=2 ** 30 + 1), -2), (dict(Hq=65535), -2),
]


@pytest.mark.parametrize("kw,want", BAD_NORM)
def test_norm_is_refused(ra, kw, want):
    L, rows, norm = ra.lib(), _rows(ra), _norm(ra, **kw)
    assert L.ringattn_qk_norm_rope(rows, rows, norm, 0) == want
    assert L.ringattn_qk_norm_rope_bwd(rows, rows, rows, F, 2 * F, norm, F, 1 << 30, 0) == want


BAD_ROWS = [dict(q=0), dict(k=0), dict(q=F + 8), dict(k=F + 2), dict(q_token_stride=508), dict(q_head_stride=64),
            dict(k_token_stride=-256), dict(k_head_stride=2 ** 32), dict(dtype=2), dict(dtype=-1)]


@pytest.mark.parametrize("kw", BAD_ROWS)
def test_norm_rows_are_refused(ra, kw):
    L, good, bad, norm = ra.lib(), _rows(ra), _rows(ra, **kw), _norm(ra)
    assert L.ringattn_qk_norm_rope(bad, good, norm, 0) == -1
    assert L.ringattn_qk_norm_rope(good, bad, norm, 0) == -1
    for at in range(3):
        args = [good, good, good]
        args[at] = bad
        assert L.ringattn_qk_norm_rope_bwd(*args, F, 2 * F, norm, F, 1 << 30, 0) == -1


def test_norm_types_that_a_call_does_not_take(ra):
    L, good, f32, norm = ra.lib(), _rows(ra), _rows(ra, dtype=1), _norm(ra)
    assert L.ringattn_qk_norm_rope(f32, good, norm, 0) == -1
    assert L.ringattn_qk_norm_rope(good, f32, norm, 0) == -1
    assert L.ringattn_qk_norm_rope_bwd(f32, good, good, F, 2 * F, norm, F, 1 << 30, 0) == -1


def test_norm_arguments_that_are_missing(ra):
    L, rows, norm = ra.lib(), _rows(ra), _norm(ra)
    assert L.ringattn_qk_norm_rope(None, rows, norm, 0) == -1
    assert L.ringattn_qk_norm_rope(rows, None, norm, 0) == -1
    assert L.ringattn_qk_norm_rope(rows, rows, None, 0) == -1
    n = ra.qk_norm_rope_workspace_bytes(5, 4, 2, 128)
    for dw, ws, size in (((F, 2 * F), 0, n), ((F, 2 * F), F + 128, n), ((F, 2 * F), F, n - 1), ((F, 0), F, n - 256), ((F, F), F, n),
                         ((F + 2, 0), F, n)):
        assert L.ringattn_qk_norm_rope_bwd(rows, rows, rows, *dw, norm, ws, size, 0) == -1


def test_nothing_to_do_needs_no_device(ra):
    L, norm = ra.lib(), _norm(ra, total=0, position=0, cos_sin=0)
    assert L.ringattn_qk_norm_rope(None, None, norm, 0) == 0
    assert L.ringattn_qk_norm_rope_bwd(None, None, None, 0, 0, norm, 0, 0, 0) == 0
    kv = ctypes.byref(_kv(ra, total=0))
    assert L.ringattn_cache_weights(0, 0, 0, 0, 0, 0, kv, 0, 0, 1.0, 4, 1, 1, 0, 0, 0, 0, 0) == 0


def test_norm_workspace(ra):
    b = ctypes.c_longlong()
    f = ra.lib().ringattn_qk_norm_rope_workspace_bytes
    for args, want in (((5, 4, 2, 96), -1), ((-1, 4, 2, 128), -1), ((5, 0, 2, 128), -1), ((5, 4, 0, 64), -1), ((5, 65536, 1, 64), -2)):
        assert f(*args, ctypes.byref(b)) == want
    assert f(5, 4, 2, 128, None) == -1
    for d in (64, 128):
        for hq, hkv in ((64, 8), (6, 2), (1, 1), (300, 300)):
            last = 0
            for total in (0, 1, 15, 16, 17, 1000, 10 ** 6, 2 ** 30):
                n = ra.qk_norm_rope_workspace_bytes(total, hq, hkv, d)
                groups = -(-hq // 4) + -(-hkv // 4)
                assert n % 256 == 0 and last <= n <= max(2048, groups) * d * 4 + 256
                last = n


def _weights_args(kv, **kw):
    a = dict(q=F, q_ts=512, q_hs=128, lse=F, l_ts=4, l_hs=1, kv=kv, w=F, w_ps=64, decay=1.0, Hq=4, max_q=1, causal=1, window=0, sinks=0,
             ws=F, size=1 << 40, stream=0)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw,want", BAD_KV)
def test_pool_and_batch_are_refused(ra, kw, want):
    r = ctypes.byref(_kv(ra, **kw))
    assert ra.lib().ringattn_cache_weights(*_weights_args(r)) == want
    if not {"cu", "total"} & set(kw):  # eviction has no rows
        assert ra.lib().ringattn_cache_evict(r, F, 64, F, 9, 0, 0, F, F, 0) == want


@pytest.mark.parametrize("kw", [
    dict(q=0), dict(q=F + 8), dict(q_ts=508), dict(q_hs=64), dict(lse=0), dict(lse=F + 2), dict(l_ts=0), dict(l_hs=-1), dict(kv=None),
    dict(w=0), dict(w=F + 4), dict(w_ps=60), dict(w_ps=66), dict(decay=-0.1), dict(decay=1.1), dict(decay=math.nan), dict(Hq=0),
    dict(Hq=5), dict(max_q=0), dict(causal=2), dict(window=-1), dict(sinks=-1), dict(causal=0, window=5), dict(ws=0), dict(ws=F + 16),
    dict(size=1000),
])
def test_weights_refuse(ra, kw):
    assert ra.lib().ringattn_cache_weights(*_weights_args(**{"kv": ctypes.byref(_kv(ra)), **kw})) == -1


def test_sizes_that_are_not_supported(ra):
    L, kv = ra.lib(), ctypes.byref(_kv(ra))
    assert L.ringattn_cache_weights(*_weights_args(kv, Hq=258)) == -2
    assert L.ringattn_cache_weights(*_weights_args(ctypes.byref(_kv(ra, total=2 ** 30, Hkv=2)))) == -2
    assert L.ringattn_cache_weights(*_weights_args(kv, w_ps=2 ** 36 + 4)) == -2
    assert L.ringattn_cache_evict(kv, F, 64, F, 2 ** 30 + 1, 0, 0, F, F, 0) == -2
    assert L.ringattn_cache_evict(kv, F, 2 ** 36 + 4, F, 9, 0, 0, F, F, 0) == -2


@pytest.mark.parametrize("args", [
    (0, 64, F, 9, 0, 0, F, F), (F + 8, 64, F, 9, 0, 0, F, F), (F, 63, F, 9, 0, 0, F, F), (F, 66, F, 9, 0, 0, F, F), (F, 64, 0, 9, 0, 0, F, F),
    (F, 64, F + 2, 9, 0, 0, F, F), (F, 64, F, 0, 0, 0, F, F), (F, 64, F, 9, -1, 0, F, F), (F, 64, F, 9, 0, -1, F, F), (F, 64, F, 9, 0, 0, 0, F),
    (F, 64, F, 9, 0, 0, F, 0), (F, 64, F, 9, 0, 0, F + 1, F), (F, 64, F, 9, 0, 0, F, F + 3),
])
def test_evict_refuses(ra, args):
    assert ra.lib().ringattn_cache_evict(ctypes.byref(_kv(ra)), *args, 0) == -1


# ------------------------------------------------------------------ refusals of the binding
def test_binding_refuses_host_tensors_and_wrong_shapes(ra, monkeypatch):
    """Host tensors report device -1; with the current device taken as that, the checks of types and shapes are reached."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)
    q, k = torch.zeros((5, 4, 64), dtype=torch.bfloat16), torch.zeros((5, 2, 64), dtype=torch.bfloat16)
    pos, table = torch.zeros(5, dtype=torch.int32), torch.zeros((9, 32))

    def norm(**kw):
        a = dict(q=q, k=k, q_out=q, k_out=k, position=pos, cos_sin=table)
        a.update(kw)
        ra.qk_norm_rope(**a, stream=0)

    def bwd(**kw):
        a = dict(q=q, k=k, dq_out=q, dk_out=k, dq=q, dk=k, position=pos, cos_sin=table)
        a.update(kw)
        ra.qk_norm_rope_bwd(**a, stream=0)

    for call in (norm, bwd):
        for kw in (dict(q=q.float()), dict(k=k[:4]), dict(k=k[..., :32]), dict(q=q[0]), dict(position=pos.long()), dict(position=pos[:4]),
                   dict(cos_sin=table.double()), dict(cos_sin=table[0]), dict(cos_sin=table.t()), dict(q_weight=torch.ones(63)),
                   dict(q_weight=torch.ones(64), k_weight=torch.ones(64, dtype=torch.bfloat16)), dict(k_weight=torch.ones(64, dtype=torch.float16))):
            with pytest.raises(ValueError):
                call(**kw)
    for kw in (dict(q_out=q[:, :3]), dict(k_out=k.float()), dict(q_out=torch.zeros((5, 64, 4), dtype=torch.bfloat16).transpose(1, 2))):
        with pytest.raises(ValueError):
            norm(**kw)
    for kw in (dict(dq=q.float()), dict(dk_out=k.float()), dict(dq_out=q.half(), dk_out=k.half()), dict(dq_weight=torch.zeros(64)),
               dict(dq_weight=torch.zeros(64, dtype=torch.bfloat16)), dict(dk_weight=torch.zeros(32))):
        with pytest.raises(ValueError):
            bwd(**kw)
    cache = [torch.zeros((6, 2, 16, 64), dtype=torch.bfloat16) for _ in range(2)]
    w, bt, cu = torch.zeros((6, 2, 16)), torch.zeros((3, 2), dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    i3, kept = torch.zeros(3, dtype=torch.int32), torch.zeros((3, 2, 7), dtype=torch.int32)
    ws, lse = torch.zeros(8, dtype=torch.uint8), torch.zeros((5, 4))

    def weights(**kw):
        a = dict(q=q, lse=lse, k_cache=cache[0], v_cache=cache[1], weights=w, block_table=bt, cu=cu, kv_len=i3, workspace=ws, max_q=2)
        a.update(kw)
        ra.cache_weights(**a, stream=0)

    def evict(**kw):
        a = dict(k_cache=cache[0], v_cache=cache[1], weights=w, block_table=bt, kv_len=i3, keep=i3, kv_len_out=i3, kept=kept)
        a.update(kw)
        ra.cache_evict(**a, stream=0)

    for call in (weights, evict):
        for kw in (dict(weights=w.double()), dict(weights=w[:5]), dict(weights=w[..., :8]), dict(weights=w.transpose(0, 1)), dict(kv_len=i3[:2]),
                   dict(block_table=bt.long()), dict(k_scale=w), dict(k_cache=cache[0][:5]), dict(sinks=2 ** 31)):
            with pytest.raises(ValueError):
                call(**kw)
    for kw in (dict(lse=lse.double()), dict(lse=lse[:, :3]), dict(cu=cu[:3]), dict(workspace=ws.int()), dict(max_q=2 ** 31), dict(window=-2 ** 31 - 1),
               dict(q=torch.zeros((5, 4, 128), dtype=torch.bfloat16))):
        with pytest.raises(ValueError):
            weights(**kw)
    for kw in (dict(keep=i3.long()), dict(keep=i3[:2]), dict(kv_len_out=torch.zeros(6, dtype=torch.int32)[::2]), dict(kept=kept[:, :1]),
               dict(kept=kept[:2]), dict(kept=kept[..., ::2]), dict(kept=kept.float()), dict(recent=2 ** 31)):
        with pytest.raises(ValueError):
            evict(**kw)


def test_binding_refuses_host_tensors(ra, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    q, pos, table = torch.zeros((5, 4, 64), dtype=torch.bfloat16), torch.zeros(5, dtype=torch.int32), torch.zeros((9, 32))
    with pytest.raises(ValueError, match="current device"):
        ra.qk_norm_rope(q, q, q, q, pos, table)
    cache, i3 = torch.zeros((6, 2, 16, 64), dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        ra.cache_evict(cache, cache, torch.zeros((6, 2, 16)), torch.zeros((3, 2), dtype=torch.int32), i3, i3, i3, i3.view(3, 1, 1))
