"""ringattn_cache_weights: values that are no numbers, where the formula has them and where nobody sees them, against the float64
oracle."""
import numpy as np
import pytest
import torch

from tests.test_gpu_cache_weights import Run, ra  # noqa: F401
from tests.test_gpu_cache_weights_rows_left_out import INF, NAN, ROWS, compare, nan_key

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", ROWS)
@pytest.mark.parametrize("e4m3", [False, True])
def test_an_infinite_lse(ra, n, e4m3):
    """exp(s - inf) is 0 for a number s, and no number for a score that is none."""
    r = Run([(n, 300), (n, 200)], hq=8, hkv=2, d=64, e4m3=e4m3, seed=n)
    r.lse[0] = INF
    r.lse[n] = INF
    r.q[n, 1] = NAN
    r.call(ra)
    assert ra.sync_status() == ra.RA_OK
    assert np.isfinite(compare(r)).all()
    got = compare(r, 1)
    assert np.isnan(got[:200 - n + 1, 0]).all() and np.isfinite(got[:, 1]).all()


@pytest.mark.parametrize("n", ROWS)
@pytest.mark.parametrize("window", [0, 50])
def test_hidden_keys_of_e4m3_may_hold_anything(ra, n, window):
    """Scales that are no numbers behind a row's own position and before a window: no other key changes."""
    r = Run([(n, 400), (1, 90)], hq=8, hkv=2, d=64, page=16, e4m3=True, seed=8, window=window)
    pg, row = r.B.places(0)
    seen = np.ones((400, 2), dtype=bool)
    if window:
        nan_key(r, 0, 10, 0)
        r.B.k_scale[pg[11], 1, row[11]] = NAN
        r.B.k_scale[pg[12], :, row[12]] = INF
    if n > 1:  # the last row alone sees it
        r.B.k_scale[pg[399], 0, row[399]] = NAN
        seen[399, 0] = False
    r.call(ra)
    assert ra.sync_status() == ra.RA_OK
    got = compare(r)
    assert np.array_equal(np.isfinite(got), seen)
    compare(r, 1)
