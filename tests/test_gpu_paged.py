"""The paged K/V cache on the GPU against the float64 oracle: ringattn_cache_append,
ringattn_cache_read and ringattn_fwd_paged, through the C ABI."""
import math

import numpy as np
import pytest
import torch

from oracle import attention as oatt
from oracle import paged as opaged
from tests.gpu_util import dev
from tests.paged_util import Batch, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ra():
    from online_softmax_attention_zigzag_gb300 import ringattn
    ringattn.lib()
    torch.cuda.set_device(0)
    return ringattn


def _randn(shape, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(torch.bfloat16)


def _bits(t):
    return t.contiguous().view(torch.uint8 if t.element_size() == 1 else torch.int16 if t.element_size() == 2
                               else torch.int32).cpu()


def _attend(ra, B, q, out_dtype=torch.bfloat16, workspace=None, max_q=None, stream=None, **kw):
    """fwd_paged on NaN-filled outputs; returns (out, lse)."""
    total, Hq, d = q.shape
    out = torch.full((total, Hq, d), float("nan"), dtype=out_dtype, device=dev())
    lse = torch.full((total, Hq), float("nan"), device=dev())
    max_q = max_q or B.max_q
    if workspace is None:  # full of NaN: what it holds must not matter
        workspace = torch.full((ra.paged_workspace_bytes(total, len(B.seqs), Hq, B.hkv, d, max_q),), 255,
                               dtype=torch.uint8, device=dev())
    ra.fwd_paged(q, B.k_cache, B.v_cache, out, lse, *B.args(), workspace, max_q=max_q, stream=stream, **B.kw(), **kw)
    return out, lse


def _check_all(B, q, out, lse, p_eps=2.0 ** -8, **kw):
    cu = B.cu.tolist()
    for b, (n, L) in enumerate(B.seqs):
        k, v = B.kept(b)
        rows = slice(cu[b], cu[b + 1])
        # rows before position 0 see nothing: the oracle takes the last min(n, L) rows
        ref = opaged.attention(q[rows].double().cpu().numpy(), k, v, kw.get("causal", 1), kw.get("window", 0),
                               kw.get("sinks", 0))
        check(out[rows], lse[rows], ref, B.d, out.dtype == torch.bfloat16, f"sequence {b} ({n} of {L})", p_eps)
    assert torch.isnan(out[cu[-1]:].float()).all() and torch.isnan(lse[cu[-1]:]).all(), "a padding row was written"


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("hkv,d,page,seqs,layout", [
    (8, 128, 64, [(1, 1)], "plain"),                                    # one token, an empty cache
    (8, 128, 16, [(1, 777), (1, 64), (1, 65), (0, 9), (1, 16)], "plain"),   # a decoding step
    (3, 64, 48, [(130, 131), (17, 700), (96, 96)], "fused"),            # a slice of a fused projection
    (2, 128, 32, [(65, 65), (1, 300)], "heads"),                        # head-major rows
    (1, 64, 256, [(5, 3), (300, 300)], "plain"),                        # rows before position 0
])
def test_append_is_bit_exact(ra, e4m3, hkv, d, page, seqs, layout):
    B = Batch(seqs, hkv=hkv, d=d, page=page, e4m3=e4m3, device=dev(), seed=1, pad=3, fill=False, gap=8)
    want = Batch(seqs, hkv=hkv, d=d, page=page, e4m3=e4m3, device=dev(), seed=1, pad=3, fill=False, gap=8)
    hq = 4
    if layout == "fused":
        qkv = _randn((B.total, hq + 2 * hkv, d), 2).to(dev())
        kn, vn = qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    elif layout == "heads":
        kn, vn = (_randn((hkv, B.total, d), s).to(dev()).transpose(0, 1) for s in (3, 4))
    else:
        kn, vn = (_randn((B.total, hkv, d), s).to(dev()) for s in (5, 6))
    ra.cache_append(kn, vn, B.k_cache, B.v_cache, *B.args(), **B.kw())
    assert ra.sync_status() == ra.RA_OK
    cu = B.cu.tolist()
    for b, (n, L) in enumerate(seqs):
        page_i, row_i = want.places(b)
        m = min(n, L)
        page_i, row_i = page_i[L - m:], row_i[L - m:]
        for x, cache, scale in ((kn, want.k_cache, want.k_scale), (vn, want.v_cache, want.v_scale)):
            x = x[cu[b + 1] - m:cu[b + 1]]
            if e4m3:
                c, s = opaged.quantise(x.double().cpu().numpy())
                cache.view(torch.uint8)[page_i, :, row_i] = torch.from_numpy(c).float().to(torch.float8_e4m3fn).to(
                    dev()).view(torch.uint8)
                scale[page_i, :, row_i] = torch.from_numpy(s).float().to(dev())
            else:
                cache[page_i, :, row_i] = x
    # every row of the pool: the new ones as they should be, all others as they were
    assert torch.equal(_bits(B.k_cache), _bits(want.k_cache)) and torch.equal(_bits(B.v_cache), _bits(want.v_cache))
    if e4m3:
        assert torch.equal(_bits(B.k_scale), _bits(want.k_scale)) and torch.equal(_bits(B.v_scale), _bits(want.v_scale))


@pytest.mark.parametrize("d", [64, 128])
def test_append_quantises_the_whole_range(ra, d):
    """Zeros, one element alone, subnormals, the largest bf16 numbers, ties, infinities and NaN."""
    rows = [torch.zeros(d), torch.ones(d), torch.full((d,), 448.0), torch.full((d,), 450.0), torch.full((d,), 2.0 ** -133),
            torch.full((d,), 1.8 * 2.0 ** 127), torch.cat([torch.tensor([1e30]), torch.full((d - 1,), 1e-30)]),
            torch.linspace(-3, 3, d), torch.cat([torch.tensor([448.0]), torch.arange(1, d) * 2.0 ** -10]),
            torch.cat([torch.tensor([256.0]), 17.0 + torch.arange(1, d) * 0.5]),
            torch.cat([torch.full((d - 1,), 2.0), torch.tensor([float("inf")])]),
            torch.cat([torch.tensor([float("nan")]), torch.full((d - 1,), 2.0)]),
            torch.cat([torch.full((d // 2,), -float("inf")), torch.full((d // 2,), float("nan"))])]
    rows += list(torch.exp2(torch.arange(-140, 127).float())[:, None] * torch.linspace(-1, 1, d)[None])
    x = torch.stack(rows).to(torch.bfloat16)[:, None]
    n = len(rows)
    B = Batch([(n, n)], hkv=1, d=d, page=64, e4m3=True, device=dev(), fill=False)
    ra.cache_append(x.to(dev()), x.neg().to(dev()), B.k_cache, B.v_cache, *B.args(), **B.kw())
    ko, vo = (torch.empty((1, n, d), dtype=torch.bfloat16, device=dev()) for _ in range(2))
    ra.cache_read(B.k_cache, B.v_cache, ko, vo, *B.args(), **B.kw())
    assert ra.sync_status() == ra.RA_OK
    codes, scale = opaged.quantise(x.double().numpy())
    page, row = B.places(0)
    got_s = B.k_scale[page, :, row].double().cpu().numpy()
    assert np.array_equal(got_s, scale, equal_nan=True)
    got_c = B.k_cache.view(torch.uint8)[page, :, row].view(torch.float8_e4m3fn).double().cpu().numpy()
    assert np.array_equal(got_c, codes)
    got_c = B.v_cache.view(torch.uint8)[page, :, row].view(torch.float8_e4m3fn).double().cpu().numpy()
    assert np.array_equal(got_c, -codes)
    want = (codes * scale[..., None]).transpose(1, 0, 2)
    assert np.array_equal(ko.double().cpu().numpy(), want, equal_nan=True)
    assert np.array_equal(vo.double().cpu().numpy(), -want, equal_nan=True)


# ------------------------------------------------------------------ read
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("hkv,d,page,seqs", [
    (8, 128, 64, [(1, 1)]),
    (2, 64, 16, [(777, 777), (0, 40), (1, 33), (31, 65)]),
    (3, 128, 48, [(100, 1000), (4, 2), (5, 0)]),              # rows before position 0 read as zeros
])
def test_read_is_bit_exact(ra, e4m3, hkv, d, page, seqs):
    B = Batch(seqs, hkv=hkv, d=d, page=page, e4m3=e4m3, device=dev(), seed=7, pad=5, gap=16)
    ko, vo = (torch.full((hkv, B.total, d), float("nan"), dtype=torch.bfloat16, device=dev()) for _ in range(2))
    ra.cache_read(B.k_cache, B.v_cache, ko, vo, *B.args(), **B.kw())
    assert ra.sync_status() == ra.RA_OK
    cu = B.cu.tolist()
    for b, (n, L) in enumerate(seqs):
        for got, kept in zip((ko, vo), B.kept(b)):
            got = got[:, cu[b]:cu[b + 1]].double().cpu().numpy().transpose(1, 0, 2)
            m = min(n, L)
            assert np.array_equal(got[n - m:], kept[L - m:])
            assert not got[:n - m].any()
    assert torch.isnan(ko[:, cu[-1]:].float()).all() and torch.isnan(vo[:, cu[-1]:].float()).all()


def test_pages_that_are_none_are_dropped_and_read_as_zeros(ra):
    """Table entries outside the pool: nothing is written for them, zeros are read from them, and
    attention takes a zero key and value there."""
    Hq, hkv, d, page, L = 4, 2, 128, 32, 200
    B = Batch([(L, L)], hkv=hkv, d=d, page=page, e4m3=False, device=dev(), seed=9)
    bad = {1: -1, 3: B.n_pages, 5: 2 ** 31 - 1}
    for i, pg in bad.items():
        B.dtable[0, i] = pg
        B.k[0][i * page:(i + 1) * page] = 0
        B.v[0][i * page:(i + 1) * page] = 0
    before = B.k_cache.clone()
    x = torch.ones((L, hkv, d), dtype=torch.bfloat16, device=dev())
    ko, vo = (torch.empty((hkv, L, d), dtype=torch.bfloat16, device=dev()) for _ in range(2))
    ra.cache_read(B.k_cache, B.v_cache, ko, vo, *B.args())
    assert torch.equal(ko.cpu().transpose(0, 1), B.k[0]) and torch.equal(vo.cpu().transpose(0, 1), B.v[0])
    for n in (1, 40, 200):
        q = _randn((n, Hq, d), 10, d ** -0.5).to(dev())
        B1 = Batch([(n, L)], hkv=hkv, d=d, page=page, e4m3=False, device=dev(), seed=9, fill=False)
        B1.k_cache, B1.v_cache, B1.dtable, B1.k, B1.v = B.k_cache, B.v_cache, B.dtable, B.k, B.v
        out, lse = _attend(ra, B1, q)
        assert ra.sync_status() == ra.RA_OK
        _check_all(B1, q, out, lse)
    ra.cache_append(x, x, B.k_cache, B.v_cache, *B.args())
    assert ra.sync_status() == ra.RA_OK
    changed = (_bits(B.k_cache) != _bits(before)).flatten(1).any(1)
    assert int(changed.sum()) == -(-L // page) - len(bad)


# ------------------------------------------------------------------ attend
SHAPES = [(64, 8, 128), (8, 2, 64), (6, 2, 128), (4, 4, 64), (8, 1, 128), (14, 2, 64), (128, 1, 64)]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("hq,hkv,d", SHAPES)
@pytest.mark.parametrize("page", [16, 48, 128])
def test_decode(ra, e4m3, hq, hkv, d, page):
    """One new token a sequence: lengths around tiles and pages, 1 and 0 among them."""
    seqs = [(1, L) for L in (1, 2, 15, 16, 17, 127, 128, 129, 255, 1000)] + [(0, 5), (1, 0), (0, 0)]
    B = Batch(seqs, hkv=hkv, d=d, page=page, e4m3=e4m3, device=dev(), seed=11, pad=2)
    q = _randn((B.total, hq, d), 12, d ** -0.5).to(dev())
    out, lse = _attend(ra, B, q)
    assert ra.sync_status() == ra.RA_OK
    _check_all(B, q, out, lse)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("hq,hkv,d", SHAPES)
@pytest.mark.parametrize("n", [2, 5, 16, 33, 130])
def test_chunks(ra, e4m3, hq, hkv, d, n):
    """Several new tokens a sequence, ragged, from the first token on and over a context."""
    seqs = [(n, n), (n, n + 1), (1, 300), (max(1, n - 1), 513), (n, 2 * n + 260), (n, n // 2), (n, 0)]
    B = Batch(seqs, hkv=hkv, d=d, page=32, e4m3=e4m3, device=dev(), seed=13, pad=1, gap=16)
    q = _randn((B.total, hq, d), 14, d ** -0.5).to(dev())
    out, lse = _attend(ra, B, q)
    assert ra.sync_status() == ra.RA_OK
    _check_all(B, q, out, lse)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (7, 3), (128, 0), (100, 128), (129, 130), (1000, 4), (5000, 9)])
@pytest.mark.parametrize("n", [1, 3, 150])
def test_window_and_sinks(ra, e4m3, window, sinks, n):
    hq, hkv, d = 8, 2, 128
    seqs = [(n, max(n, L)) for L in (1, 130, 257, 700, 1400)] + [(n, n // 3)]
    B = Batch(seqs, hkv=hkv, d=d, page=16, e4m3=e4m3, device=dev(), seed=15)
    q = _randn((B.total, hq, d), 16, d ** -0.5).to(dev())
    kw = dict(window=window, sinks=sinks)
    out, lse = _attend(ra, B, q, **kw)
    assert ra.sync_status() == ra.RA_OK
    _check_all(B, q, out, lse, **kw)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("n", [1, 2, 70])
def test_without_the_causal_mask_and_fp32_out(ra, e4m3, n):
    hq, hkv, d = 8, 2, 64
    B = Batch([(n, L) for L in (n, n + 129, 600)], hkv=hkv, d=d, page=64, e4m3=e4m3, device=dev(), seed=17)
    q = _randn((B.total, hq, d), 18, d ** -0.5).to(dev())
    for causal in (0, 1):
        out, lse = _attend(ra, B, q, torch.float32, causal=causal)
        assert ra.sync_status() == ra.RA_OK
        _check_all(B, q, out, lse, causal=causal)


@pytest.mark.parametrize("std", [0.02, 1.0, 8.0])
@pytest.mark.parametrize("n", [1, 40])
def test_flat_and_peaked_softmax(ra, std, n):
    """Scores from nearly equal to one key taking all."""
    hq, hkv, d = 16, 2, 128
    for e4m3 in (False, True):
        B = Batch([(n, 3000), (n, 500)], hkv=hkv, d=d, page=64, e4m3=e4m3, device=dev(), seed=19)
        q = _randn((B.total, hq, d), 20, std).to(dev())
        out, lse = _attend(ra, B, q)
        assert ra.sync_status() == ra.RA_OK
        _check_all(B, q, out, lse)


@pytest.mark.parametrize("e4m3", [False, True])
def test_scales_far_apart(ra, e4m3):
    """Rows of K and V whose sizes lie many powers of two apart, in one tile."""
    hq, hkv, d, L = 8, 2, 128, 400
    for n in (1, 60):
        B = Batch([(n, L)], hkv=hkv, d=d, page=16, e4m3=e4m3, device=dev(), seed=21, fill=False)
        g = torch.Generator().manual_seed(22)
        for x in (B.k[0], B.v[0]):
            x.mul_(torch.exp2(torch.randint(-30, 1, (L, hkv, 1), generator=g).float()))
        B.v[0].mul_(2.0 ** 20)
        B.fill()
        q = _randn((n, hq, d), 23, 0.3).to(dev())
        out, lse = _attend(ra, B, q)
        assert ra.sync_status() == ra.RA_OK
        _check_all(B, q, out, lse)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("n,window", [(2, 0), (9, 0), (200, 0), (9, 40), (200, 100)])
def test_infinities_and_nan_that_a_row_does_not_see(ra, e4m3, bad, n, window):
    """K and V rows of NaN or infinity: rows that do not see them are as without them, rows that
    see one are not finite where the definition is not."""
    hq, hkv, d, L = 4, 2, 128, 420
    B = Batch([(n, L)], hkv=hkv, d=d, page=32, e4m3=e4m3, device=dev(), seed=25, fill=False)
    at = [L - n + 1, L - max(1, n // 2), L - 1] + ([L - n - window + 1] if window else [])
    at = sorted({a for a in at if L - n - window < a < L and a >= 0 and (window or a > L - n)})
    for a in at:
        B.k[0][a, 0, 5] = bad       # head 0: a bad key
        B.v[0][a, 1, 7] = bad       # head 1: a bad value
    B.fill()
    q = _randn((n, hq, d), 26, d ** -0.5).to(dev())
    out, lse = _attend(ra, B, q, window=window)
    assert ra.sync_status() == ra.RA_OK
    k, v = B.kept(0)
    clean = [x.copy() for x in (k, v)]
    for x in clean:
        x[at] = 0.0
    ref = opaged.attention(q.double().cpu().numpy(), *clean, True, window)
    see = opaged.visible(n, L, True, window)[:, at].any(1)
    idx = torch.from_numpy(np.nonzero(~see)[0]).to(dev())
    check(out[idx], lse[idx], [r[~see] for r in ref], d, True, "rows that see no bad key")
    o = out.double().cpu().numpy()[see]
    g = hq // hkv
    if e4m3:   # the whole row is stored as NaN
        assert np.isnan(o).all()
    elif bad != bad:
        assert np.isnan(o[:, :g]).all(), "a NaN key"
        assert np.isnan(o[:, g:, 7]).all(), "a NaN value"
    else:
        assert not np.isfinite(o[:, g:, 7]).any(), "an infinite value"
    if not e4m3:  # the other columns of a row that sees a bad value are those of the finite values
        v2 = v.copy()
        v2[:, 1, 7] = 0.0
        k2 = k.copy()
        k2[at, 0] = 0.0
        ref2 = opaged.attention(q.double().cpu().numpy(), k2, v2, True, window)
        keep = [c for c in range(d) if c != 7]
        check(out[:, g:, keep], lse[:, g:], [x[:, g:][..., keep] if x.ndim == 3 else x[:, g:] for x in ref2], d, True,
              "other columns")


def test_a_shared_prefix_and_strided_tensors(ra):
    """Two sequences whose tables name the same pages; q out of a fused projection, out and lse
    head-major, the table a slice."""
    hq, hkv, d, page, L = 8, 2, 128, 16, 333
    for n in (1, 50):
        B = Batch([(n, L), (n, L)], hkv=hkv, d=d, page=page, e4m3=False, device=dev(), seed=27, gap=32)
        shared = 10
        B.table[1, :shared] = B.table[0, :shared]
        B.k[1][:shared * page] = B.k[0][:shared * page]
        B.v[1][:shared * page] = B.v[0][:shared * page]
        wide = torch.full((2, B.table.shape[1] + 7), -5, dtype=torch.int32, device=dev())
        wide[:, 3:3 + B.table.shape[1]] = B.table.to(dev())
        B.dtable = wide[:, 3:3 + B.table.shape[1]]
        q = _randn((B.total, hq + 4, d), 28, d ** -0.5).to(dev())[:, 2:2 + hq]
        out = torch.full((hq, B.total, d), float("nan"), device=dev()).to(torch.bfloat16).transpose(0, 1)
        lse = torch.full((hq, B.total), float("nan"), device=dev()).transpose(0, 1)
        ws = torch.empty(ra.paged_workspace_bytes(B.total, 2, hq, hkv, d, n), dtype=torch.uint8, device=dev())
        ra.fwd_paged(q, B.k_cache, B.v_cache, out, lse, *B.args(), ws, max_q=n)
        assert ra.sync_status() == ra.RA_OK
        _check_all(B, q, out, lse)


@pytest.mark.parametrize("e4m3", [False, True])
def test_long_contexts(ra, e4m3):
    """Contexts that are cut and joined, beside short ones; sampled heads."""
    hq, hkv, d = 16, 2, 128
    for n in (1, 12, 300):
        B = Batch([(n, 20011), (1, 3), (n, 7000)], hkv=hkv, d=d, page=64, e4m3=e4m3, device=dev(), seed=29)
        q = _randn((B.total, hq, d), 30, d ** -0.5).to(dev())
        out, lse = _attend(ra, B, q)
        assert ra.sync_status() == ra.RA_OK
        _check_all(B, q, out, lse)
        again = _attend(ra, B, q)
        assert torch.equal(out, again[0]) and torch.equal(lse, again[1]), "the same call twice"


def test_many_sequences(ra):
    """More sequences than blocks, more than the copies keep in shared memory, most of them short."""
    hq, hkv, d = 4, 1, 64
    g = torch.Generator().manual_seed(31)
    L = torch.randint(1, 40, (1500,), generator=g).tolist()
    B = Batch([(1, x) for x in L], hkv=hkv, d=d, page=16, e4m3=False, device=dev(), seed=31)
    q = _randn((B.total, hq, d), 32, d ** -0.5).to(dev())
    out, lse = _attend(ra, B, q)
    _check_all(B, q, out, lse)
    new = _randn((B.total, hkv, d), 33).to(dev())
    ra.cache_append(new, new, B.k_cache, B.v_cache, *B.args())
    ko, vo = (torch.empty((hkv, B.total, d), dtype=torch.bfloat16, device=dev()) for _ in range(2))
    ra.cache_read(B.k_cache, B.v_cache, ko, vo, *B.args())
    assert ra.sync_status() == ra.RA_OK
    assert torch.equal(ko.transpose(0, 1), new) and torch.equal(vo.transpose(0, 1), new)


def test_a_pool_beyond_32_bit_offsets(ra):
    """Pages whose elements lie beyond 2^32 elements of the pool's start."""
    hq, hkv, d, page, L = 8, 8, 128, 64, 500
    n_pages = 2 ** 32 // (hkv * page * d) + 40
    for dtype in (torch.float8_e4m3fn, torch.bfloat16):
        e4m3 = dtype != torch.bfloat16
        B = Batch([(L, L)], hkv=hkv, d=d, page=page, e4m3=e4m3, device=dev(), seed=35, fill=False)
        B.k_cache, B.v_cache = (torch.empty((n_pages, hkv, page, d), dtype=dtype, device=dev()) for _ in range(2))
        if e4m3:
            B.k_scale, B.v_scale = (torch.empty((n_pages, hkv, page), device=dev()) for _ in range(2))
        k = -(-L // page)
        B.table[0, :k] = n_pages - 1 - torch.arange(k, dtype=torch.int32)
        B.dtable = B.table.to(dev())
        ra.cache_append(B.k[0].to(dev()), B.v[0].to(dev()), B.k_cache, B.v_cache, *B.args(), **B.kw())
        ko, vo = (torch.empty((hkv, L, d), dtype=torch.bfloat16, device=dev()) for _ in range(2))
        ra.cache_read(B.k_cache, B.v_cache, ko, vo, *B.args(), **B.kw())
        kept = B.kept(0)
        assert np.array_equal(ko.transpose(0, 1).double().cpu().numpy(), kept[0])
        assert np.array_equal(vo.transpose(0, 1).double().cpu().numpy(), kept[1])
        for n in (1, 200):
            q = _randn((n, hq, d), 36, d ** -0.5).to(dev())
            B.seqs, B.max_q, B.cu = [(n, L)], n, torch.tensor([0, n], dtype=torch.int32)
            B.dcu = B.cu.to(dev())
            out, lse = _attend(ra, B, q)
            assert ra.sync_status() == ra.RA_OK
            _check_all(B, q, out, lse)
        del B, ko, vo
        torch.cuda.empty_cache()


# ------------------------------------------------------------------ streams and graphs
def test_streams_graphs_and_two_calls_at_once(ra):
    hq, hkv, d = 8, 2, 128
    Bs = [Batch([(n, 4000), (1, 77)], hkv=hkv, d=d, page=32, e4m3=e, device=dev(), seed=41 + i)
          for i, (n, e) in enumerate([(1, False), (2, True), (100, False), (64, True)])]
    qs = [_randn((B.total, hq, d), 45 + i, d ** -0.5).to(dev()) for i, B in enumerate(Bs)]
    want = [_attend(ra, B, q) for B, q in zip(Bs, qs)]
    torch.cuda.synchronize()
    # every batch on a stream of its own, each with its workspace, several rounds in flight
    streams = [torch.cuda.Stream() for _ in Bs]
    got = []
    for _ in range(5):
        for B, q, st in zip(Bs, qs, streams):
            with torch.cuda.stream(st):
                got.append(_attend(ra, B, q))
    torch.cuda.synchronize()
    for i, (o, l) in enumerate(got):
        assert torch.equal(o, want[i % 4][0]) and torch.equal(l, want[i % 4][1])
    # the stream given explicitly
    st = streams[0]
    st.wait_stream(torch.cuda.current_stream())
    o, l = _attend(ra, Bs[2], qs[2], stream=st)
    st.synchronize()
    assert torch.equal(o, want[2][0]) and torch.equal(l, want[2][1])
    # captured once, replayed with other lengths: the device arrays are read at replay
    for B, q in zip(Bs, qs):
        out = torch.zeros((B.total, hq, d), dtype=torch.bfloat16, device=dev())
        lse = torch.zeros((B.total, hq), device=dev())
        ws = torch.empty(ra.paged_workspace_bytes(B.total, 2, hq, hkv, d, B.max_q), dtype=torch.uint8, device=dev())
        new = _randn((B.total, hkv, d), 49).to(dev())
        gr = torch.cuda.CUDAGraph()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side), torch.cuda.graph(gr, stream=side):
            ra.fwd_paged(q, B.k_cache, B.v_cache, out, lse, *B.args(), ws, max_q=B.max_q, **B.kw())
            ra.cache_append(new, new, B.k_cache, B.v_cache, *B.args(), **B.kw())
        for L0 in (4000, 1500, 131, 0):
            B.seqs[0] = (B.seqs[0][0], L0)
            B.dlen[0] = L0
            gr.replay()
            assert ra.sync_status() == ra.RA_OK
            k, v = B.kept(0)
            n = B.seqs[0][0]
            ref = opaged.attention(q[:n].double().cpu().numpy(), k[:L0], v[:L0])
            check(out[:n], lse[:n], ref, d, True, f"replay with length {L0}")
            for b in (0, 1):  # what the append of this replay wrote
                cu, L = B.cu.tolist(), B.seqs[b][1]
                m = min(cu[b + 1] - cu[b], L)
                B.k[b][L - m:L] = new[cu[b + 1] - m:cu[b + 1]].cpu()
                B.v[b][L - m:L] = new[cu[b + 1] - m:cu[b + 1]].cpu()


# ------------------------------------------------------------------ together, as they are used
@pytest.mark.parametrize("e4m3", [False, True])
def test_prefill_chunk_decode_and_back_to_the_ring(ra, e4m3):
    """A prompt goes through the ring, its K and V into the cache; a further chunk and then single
    tokens append and attend; every row equals the causal attention of the whole sequence over
    what the cache holds, and the cache read back feeds the ring."""
    hq, hkv, d, page, S0, chunk, steps = 8, 2, 128, 32, 512, 125, 3
    S = S0 + chunk + steps
    k, v = _randn((hkv, S, d), 51), _randn((hkv, S, d), 52)
    q = _randn((hq, S, d), 53, d ** -0.5)
    qd, kd, vd = q.to(dev()), k.to(dev()), v.to(dev())
    out0 = torch.empty((hq, S0, d), device=dev())
    lse0 = torch.empty((hq, S0), device=dev())
    first = [x[:, :S0].contiguous() for x in (qd, kd, vd)]
    ra.fwd_natural(*first, out0, lse0, c=2, causal=1, layout=1, kv_block=128)
    B = Batch([(S, S)], hkv=hkv, d=d, page=page, e4m3=e4m3, device=dev(), seed=54, fill=False)
    B.k[0], B.v[0] = k.transpose(0, 1), v.transpose(0, 1)
    at = 0
    rows = []
    for n in [S0, chunk] + [1] * steps:
        B.dcu = torch.tensor([0, n], dtype=torch.int32, device=dev())
        B.dlen = torch.tensor([at + n], dtype=torch.int32, device=dev())
        kn, vn, qn = (x[:, at:at + n].transpose(0, 1) for x in (kd, vd, qd))
        ra.cache_append(kn, vn, B.k_cache, B.v_cache, *B.args(), **B.kw())
        B.max_q = n
        rows.append(_attend(ra, B, qn, torch.float32))
        at += n
    assert ra.sync_status() == ra.RA_OK
    out, lse = (torch.cat([r[i] for r in rows]) for i in (0, 1))
    B.seqs = [(S, S)]
    ref = opaged.attention(q.double().numpy().transpose(1, 0, 2), *B.kept(0))
    check(out, lse, ref, d, False, "prompt, chunk and steps")
    if not e4m3:  # the ring saw the same K and V
        ro, rl = oatt.full_attention(q[:, :S0].double().numpy(), k[:, :S0].double().numpy(), v[:, :S0].double().numpy(), True)
        assert np.abs(out0.double().cpu().numpy() - ro).max() <= 2e-2
        check(out0.transpose(0, 1), lse0.transpose(0, 1), [x[:S0] for x in ref], d, False, "the ring's rows")
    # back to the ring: the whole cache as [Hkv, S, d], padded to the ring's tiles by another call
    n = S // 128 * 128
    B.dcu = torch.tensor([0, n], dtype=torch.int32, device=dev())
    B.dlen = torch.tensor([n], dtype=torch.int32, device=dev())
    ko, vo = (torch.empty((hkv, n, d), dtype=torch.bfloat16, device=dev()) for _ in range(2))
    ra.cache_read(B.k_cache, B.v_cache, ko, vo, *B.args(), **B.kw())
    o1, l1 = torch.empty((hq, n, d), device=dev()), torch.empty((hq, n), device=dev())
    ra.fwd_natural(qd[:, :n].contiguous(), ko, vo, o1, l1, c=1, causal=1, layout=0, kv_block=n)
    assert ra.sync_status() == ra.RA_OK
    check(o1.transpose(0, 1), l1.transpose(0, 1), [x[:n] for x in ref], d, False, "the ring over the cache")


def test_partial_results_merge(ra):
    """fp32 results over disjoint keys (the prompt's, the rest's) combine with ringattn_merge."""
    hq, hkv, d, L, cut = 8, 2, 64, 500, 300
    for n in (1, 30):
        B = Batch([(n, L)], hkv=hkv, d=d, page=20 * 16, e4m3=False, device=dev(), seed=61)
        q = _randn((n, hq, d), 62, d ** -0.5).to(dev())
        A = Batch([(n, cut)], hkv=hkv, d=d, page=16, e4m3=False, device=dev(), seed=63, fill=False)
        A.k[0], A.v[0] = B.k[0][:cut], B.v[0][:cut]
        A.fill()
        C = Batch([(n, L - cut)], hkv=hkv, d=d, page=48, e4m3=False, device=dev(), seed=64, fill=False)
        C.k[0], C.v[0] = B.k[0][cut:], B.v[0][cut:]
        C.fill()
        o, l = _attend(ra, A, q, torch.float32, causal=0)
        o2, l2 = _attend(ra, C, q, torch.float32, causal=1)
        ra.merge(o, l, o2, l2)
        assert ra.sync_status() == ra.RA_OK
        _check_all(B, q, o, l)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("n,L", [(3, 200), (60, 333), (60, 20), (3, 1)])
def test_largest_window_and_sinks(ra, e4m3, n, L):
    """A window (and sinks) of the type's largest value sees what no window sees, in rows before position 0 too."""
    hq, hkv, d = 4, 2, 128
    B = Batch([(n, L), (1, 300)], hkv=hkv, d=d, page=32, e4m3=e4m3, device=dev(), seed=71)
    q = _randn((B.total, hq, d), 72, d ** -0.5).to(dev())
    plain = _attend(ra, B, q, torch.float32)
    for window, sinks in ((2 ** 31 - 1, 0), (2 ** 31 - 1, 2 ** 31 - 1), (1, 2 ** 31 - 1)):
        o, l = _attend(ra, B, q, torch.float32, window=window, sinks=sinks)
        assert ra.sync_status() == ra.RA_OK
        assert torch.equal(o, plain[0]) and torch.equal(l, plain[1])


def test_call_longer_than_the_wait_limit(ra):
    """4.5e15 operations, more than two seconds at any rate this GPU has, over 2^30 keys (one page again and
    again): warps that have nothing to look over all that while must not take it for a hang.
    Scores are 0 and V is 0.5, so every sum is exact: out = 0.5, lse = log 2^30."""
    n, d, page = 8192, 128, 65536
    k = torch.randn((1, 1, page, d), device=dev()).to(torch.bfloat16)
    v = torch.full((1, 1, page, d), 0.5, device=dev(), dtype=torch.bfloat16)
    table = torch.zeros((1, 2 ** 30 // page), dtype=torch.int32, device=dev())
    cu = torch.tensor([0, n], dtype=torch.int32, device=dev())
    ln = torch.tensor([2 ** 30], dtype=torch.int32, device=dev())
    q = torch.zeros((n, 1, d), dtype=torch.bfloat16, device=dev())
    out, lse = torch.empty((n, 1, d), device=dev()), torch.empty((n, 1), device=dev())
    ws = torch.empty(ra.paged_workspace_bytes(n, 1, 1, 1, d, n), dtype=torch.uint8, device=dev())
    ra.fwd_paged(q, k, v, out, lse, table, cu, ln, ws, max_q=n, causal=0)
    assert ra.sync_status() == ra.RA_OK
    # (fp32: a few half steps of the quotient, and of a logarithm of 20.8)
    assert (out - 0.5).abs().max().item() <= 4 * 2.0 ** -24
    assert (lse - 30 * math.log(2)).abs().max().item() <= 4 * 2.0 ** -24 * 32


@pytest.mark.parametrize("e4m3", [False, True])
def test_sums_over_a_million_keys(ra, e4m3):
    """Equal weights and positive values over 2^20 keys (one page 16 times) in one block's hands.

    The tensor cores may truncate: a step of 2^-23 of the sum so far for every 16 keys, so half that of the
    whole sum on average.  Of 64k keys at a time that is 4096 / 2 steps; a few more for adding the 16
    sums and for the quotient."""
    n, L, d, page = 256 * torch.cuda.get_device_properties(0).multi_processor_count, 2 ** 20, 128, 65536
    dt = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    g = torch.Generator(device=dev()).manual_seed(81)
    v = (torch.rand((1, 1, page, d), device=dev(), generator=g) + 0.1).to(dt)
    k = torch.randn((1, 1, page, d), device=dev(), generator=g).to(dt)
    one = torch.ones((1, 1, page), device=dev()) if e4m3 else None
    table = torch.zeros((1, L // page), dtype=torch.int32, device=dev())
    cu = torch.tensor([0, n], dtype=torch.int32, device=dev())
    ln = torch.tensor([L], dtype=torch.int32, device=dev())
    q = torch.zeros((n, 1, d), dtype=torch.bfloat16, device=dev())
    out, lse = torch.empty((n, 1, d), device=dev()), torch.empty((n, 1), device=dev())
    ws = torch.empty(ra.paged_workspace_bytes(n, 1, 1, 1, d, n), dtype=torch.uint8, device=dev())
    ra.fwd_paged(q, k, v, out, lse, table, cu, ln, ws, max_q=n, causal=0, k_scale=one, v_scale=one)
    assert ra.sync_status() == ra.RA_OK
    want = v.double().mean(2)[0, 0]
    assert (out[:, 0].double() / want - 1).abs().max().item() <= (4096 / 2 + 32) * 2.0 ** -23


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("n", [20, 40])  # one unit of rows, and two
def test_long_items_whose_maximum_grows(ra, e4m3, n):
    """An item of 1040 tiles a block (the same pages for all), with scores that grow along the keys."""
    hq, d, L, nb = 4, 128, 133000, torch.cuda.get_device_properties(0).multi_processor_count
    B = Batch([(n, L)], hkv=1, d=d, page=512, e4m3=e4m3, device=dev(), seed=82, fill=False)
    B.k[0] = (B.k[0].float() * (0.5 + 3.5 * torch.arange(L)[:, None, None] / L)).to(torch.bfloat16)
    B.fill()
    q = _randn((nb * n, hq, d), 83, d ** -0.5)
    out, lse = torch.empty((nb * n, hq, d), device=dev()), torch.empty((nb * n, hq), device=dev())
    cu = torch.arange(0, nb * n + 1, n, dtype=torch.int32, device=dev())
    ws = torch.empty(ra.paged_workspace_bytes(nb * n, nb, hq, 1, d, n), dtype=torch.uint8, device=dev())
    ra.fwd_paged(q.to(dev()), B.k_cache, B.v_cache, out, lse, B.dtable.expand(nb, -1).contiguous(), cu, B.dlen.expand(nb).contiguous(),
                 ws, max_q=n, **B.kw())
    assert ra.sync_status() == ra.RA_OK
    for b in (0, nb - 1):
        rows = slice(b * n, (b + 1) * n)
        ref = opaged.attention(q[rows].double().numpy(), *B.kept(0))
        check(out[rows], lse[rows], ref, d, False, f"sequence {b}")


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [64, 128])
def test_outputs_on_16_byte_boundaries(ra, e4m3, out_dtype, d):
    """out rows that are 16-byte and not 32-byte aligned, in one unit of rows and in two; what lies between them stays."""
    hq, hkv, gap, step = 4, 1, 8, 16 // out_dtype.itemsize  # (strides are multiples of 8 elements in both types)
    for n in (25, 70):
        B = Batch([(n, 300), (3, 90)], hkv=hkv, d=d, page=16, e4m3=e4m3, device=dev(), seed=91)
        q = _randn((B.total, hq, d), 92, d ** -0.5).to(dev())
        buf = torch.full((B.total * hq * (d + gap) + step,), float("nan"), dtype=out_dtype, device=dev())
        out = buf[step:].view(B.total, hq, d + gap)[:, :, :d]
        assert out.data_ptr() % 32 == 16
        lse = torch.full((B.total, hq), float("nan"), device=dev())
        ws = torch.empty(ra.paged_workspace_bytes(B.total, 2, hq, hkv, d, n), dtype=torch.uint8, device=dev())
        ra.fwd_paged(q, B.k_cache, B.v_cache, out, lse, *B.args(), ws, max_q=n, **B.kw())
        assert ra.sync_status() == ra.RA_OK
        _check_all(B, q, out, lse)
        assert torch.isnan(buf[step:].view(B.total, hq, d + gap)[:, :, d:]).all() and torch.isnan(buf[:step]).all()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("n", [1, 2])
def test_one_long_sequence_among_short_ones(ra, e4m3, n):
    """Its pair lies in most of the shares while the others share theirs: one part joined of two, one of hundreds."""
    hq, hkv, d = 8, 1, 128
    g = torch.Generator().manual_seed(95)
    short = [int(x) for x in torch.randint(n, 300, (90,), generator=g)]
    B = Batch([(n, x) for x in short[:45]] + [(n, 60001)] + [(n, x) for x in short[45:]], hkv=hkv, d=d, page=32, e4m3=e4m3,
              device=dev(), seed=96)
    q = _randn((B.total, hq, d), 97, d ** -0.5).to(dev())
    o, l = _attend(ra, B, q, torch.float32)
    assert ra.sync_status() == ra.RA_OK
    # (few rows in bf16: P is two bf16 halves; in e4m3 fp16, 2^-11; the bound of one bf16 half covers both)
    _check_all(B, q, o, l)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("n,hq,hkv,L", [(14, 8, 2, 15041), (40, 8, 1, 50000), (300, 4, 1, 20000), (17, 128, 1, 4000)])
def test_few_long_items(ra, e4m3, n, hq, hkv, L):
    """Fewer items than blocks: shares of several tiles, blocks without any, an item in dozens of parts."""
    d = 128
    B = Batch([(n, L)], hkv=hkv, d=d, page=64, e4m3=e4m3, device=dev(), seed=98)
    q = _randn((n, hq, d), 99, d ** -0.5).to(dev())
    o, l = _attend(ra, B, q)
    assert ra.sync_status() == ra.RA_OK
    _check_all(B, q, o, l)
