"""ringattn_cache_weights: rows that add nothing (lse -inf) add nothing whatever they and the keys hold, on both sides of the
choice between its kernels, against the float64 oracle; and values that are no numbers come through where the formula has them."""
import numpy as np
import pytest
import torch

from oracle import evict as oevict
from tests.gpu_util import dev, f64
from tests.test_gpu_cache_weights import Run, ra  # noqa: F401

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")
# rows of a sequence; four query heads a KV head: kernels of one, two and more blocks of columns up to 24 rows in bf16 and 80
# in e4m3, then the tensor cores' units of 32 tokens, one of them, a few, a cut one
ROWS = [1, 3, 4, 5, 6, 7, 20, 21, 40, 200]


def keys(r, b=0):
    """Sequence b's keys as the pool holds them now, float64 [L, Hkv, d]."""
    pg, row = r.B.places(b)
    if not r.B.e4m3:
        return f64(r.B.k_cache[pg, :, row])
    codes = r.B.k_cache.view(torch.uint8)[pg, :, row].view(torch.float8_e4m3fn).float()
    return f64(codes) * f64(r.B.k_scale[pg, :, row])[..., None]


def compare(r, b=0):
    """As Run.check, with the keys that the pool holds; weights that are no numbers have to be none here too."""
    n, L = r.B.seqs[b]
    lo = int(r.B.cu[b])
    lse = f64(r.lse[lo:lo + n])
    with np.errstate(all="ignore"):
        want, size = oevict.add_weights(f64(r.old[b]), f64(r.q[lo:lo + n]), lse, keys(r, b), r.decay, *r.mask)
    pg, row = r.B.places(b)
    got = f64(r.w[pg, :, row])
    size = np.nan_to_num(size, nan=0.0, posinf=0.0)
    assert np.array_equal(np.isnan(got), np.isnan(want)), "NaN where there is none, or none where there is"
    assert np.array_equal(np.isinf(got), np.isinf(want))
    fin = np.isfinite(want)
    big = np.abs(lse[np.isfinite(lse)]).max() if np.isfinite(lse).any() else 0.0
    rel = ((r.d + 8) + 8) * 2.0 ** -23 * size + 2.0 ** -22 * big + 2.0 ** -20 + (n * r.hq / r.B.hkv + 16) * 2.0 ** -24
    worst = (np.abs(got - want)[fin] / (rel * np.abs(want) + 1e-37)[fin]).max()
    assert worst <= 1.0, f"off by {worst:.3g} of its bound"
    return got


def nan_key(r, b, j, h):
    """Key j of KV head h becomes NaN: its last element in bf16, its scale in e4m3."""
    pg, row = r.B.places(b)
    if r.B.e4m3:
        r.B.k_scale[pg[j], h, row[j]] = NAN
    else:
        r.B.k_cache[pg[j], h, row[j], -1] = NAN


@pytest.mark.parametrize("n", ROWS)
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("what", ["nan", "inf", "large"])
def test_whatever_a_row_without_an_lse_holds(ra, n, e4m3, d, what):
    r = Run([(n, 700), (1, 300)], hq=8, hkv=2, d=d, e4m3=e4m3, seed=n, decay=0.5)
    value = dict(nan=NAN, inf=INF, large=2.0 ** 100)[what]
    out = torch.zeros((n, 8), dtype=torch.bool)
    out[n // 2] = True
    out[0] = True
    out[:, 5] = True  # one head of every row
    if n == 1:
        out[0, :3] = False
    r.lse[:n][out] = -INF
    if what == "nan":
        r.q[:n][out] = value
    else:
        # (products of both signs, and beyond 2^60 where they are finite)
        r.q[:n][out] = value * torch.sign(r.q[:n][out].float()).to(torch.bfloat16)
    r.call(ra)
    assert ra.sync_status() == ra.RA_OK
    assert np.isfinite(compare(r)).all()
    compare(r, 1)


@pytest.mark.parametrize("n", ROWS)
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("hq,window", [(8, 0), (8, 150), (10, 150)])
def test_keys_that_only_rows_without_an_lse_see(ra, n, e4m3, hq, window):
    """The last key is NaN and the last row, the only one that sees it, has no lse: the key's weight is 0.  In bf16 a key
    that every row sees holds an infinity that gives the others' scores -inf, and theirs nothing."""
    r = Run([(n, 700)], hq=hq, hkv=2, d=64, page=16, e4m3=e4m3, seed=n, window=window)
    r.lse[n - 1] = -INF
    nan_key(r, 0, 699, 0)
    at = 0
    if not e4m3 and n > 1:
        at = 695 - n
        r.q[:, :, 3] = -1.0
        r.q[n - 1, :, 3] = torch.tensor([0.0, 1.0, -1.0, INF, NAN, 0.0, 2.0, -0.0, 3.0, -INF])[:hq].to(torch.bfloat16)
        pg, row = r.B.places(0)
        r.B.k_cache[pg[at], :, row[at], 3] = INF
    r.call(ra)
    assert ra.sync_status() == ra.RA_OK
    got = compare(r)
    assert got[699, 0] == 0.0 and np.isfinite(got).all()
    if at:
        assert np.array_equal(got[at], f64(r.old[0])[at]), "nothing is added"


@pytest.mark.parametrize("n", ROWS)
@pytest.mark.parametrize("e4m3", [False, True])
def test_all_rows_without_an_lse(ra, n, e4m3):
    r = Run([(n, 400), (n, 300)], hq=8, hkv=2, d=64, e4m3=e4m3, seed=3, decay=0.25)
    r.lse[:n] = -INF
    r.q[:n] = NAN
    r.call(ra)
    assert ra.sync_status() == ra.RA_OK
    got = compare(r)
    assert np.array_equal(got[:400 - n], 0.25 * f64(r.old[0])[:400 - n]) and not got[400 - n:].any()
    compare(r, 1)


@pytest.mark.parametrize("n", [7, 21, 200])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("causal", [0, 1])
def test_rows_without_an_lse_among_whole_units(ra, n, e4m3, causal):
    """Head by head and token by token, at the ends of units and of their halves: the other rows' bits do not change with
    what these hold."""
    r = Run([(n, 900)], hq=8, hkv=2, d=128, e4m3=e4m3, seed=n, causal=causal)
    for t in (0, 15, 16, 31, 32, 33, 63, 127, 128, n - 1):
        if t < n:
            r.lse[t, t % 8] = -INF
            r.lse[t, 7] = -INF
    res = []
    for value in (0.0, NAN, 2.0 ** 120):
        r.q[torch.isneginf(r.lse)] = value
        r.w.copy_(r.before)
        r.call(ra)
        assert ra.sync_status() == ra.RA_OK
        compare(r)
        res.append(r.w.clone())
    for x in res[1:]:
        assert torch.equal(x.view(torch.int32), res[0].view(torch.int32))
