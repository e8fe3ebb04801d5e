"""Infinities and NaN among the values that rows of a paged call see, against the definition: an
infinite value with a weight above zero makes the output that infinity, two of opposite signs or a NaN make it
NaN, and the other columns are those of the finite values."""
import numpy as np
import pytest
import torch

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


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [1, 2, 4, 40, 130])  # few rows (one group of 8, two) and chunks (one unit, two)
@pytest.mark.parametrize("causal", [0, 1])
def test_infinite_values_that_every_row_sees(ra, d, n, causal):
    """In a tile that all rows see whole and in the last one, whose end no row sees.  Scores 0 give weights
    that 16 bits hold exactly, others do not."""
    hq, hkv, L = 8, 2, 700
    for std in (0.0, d ** -0.5):
        B = Batch([(n, L)], hkv=hkv, d=d, page=32, e4m3=False, device=dev(), seed=3, fill=False)
        inf = float("inf")
        last = L - n - 1 if causal else L - 1
        B.v[0][100, 1, 3] = inf
        B.v[0][last, 1, 4] = inf
        B.v[0][200, 1, 5] = -inf
        B.v[0][50, 1, 6], B.v[0][60, 1, 6] = inf, -inf
        B.v[0][last, 1, 7] = float("nan")
        B.fill()
        q = (torch.randn((n, hq, d), generator=torch.Generator().manual_seed(4)) * std).to(torch.bfloat16).to(dev())
        out = torch.empty((n, hq, d), device=dev())
        lse = torch.empty((n, hq), device=dev())
        ws = torch.empty(ra.paged_workspace_bytes(n, 1, hq, hkv, d, n), dtype=torch.uint8, device=dev())
        ra.fwd_paged(q, B.k_cache, B.v_cache, out, lse, *B.args(), ws, max_q=n, causal=causal)
        assert ra.sync_status() == ra.RA_OK
        k, v = B.kept(0)
        clean = np.where(np.isfinite(v), v, 0.0)
        ref = opaged.attention(q.double().cpu().numpy(), k, clean, causal)
        g = hq // hkv
        check(out[:, :g], lse[:, :g], [x[:, :g] for x in ref], d, False, "the other head")
        keep = [0, 1, 2] + list(range(8, d))
        check(out[:, g:, keep], lse[:, g:], [x[:, g:][..., keep] if x.ndim == 3 else x[:, g:] for x in ref], d, False, "other columns")
        o = out[:, g:].cpu().numpy()
        assert np.isposinf(o[..., 3]).all() and np.isposinf(o[..., 4]).all(), "an infinite value"
        assert np.isneginf(o[..., 5]).all(), "a negative infinite value"
        assert np.isnan(o[..., 6]).all() and np.isnan(o[..., 7]).all(), "infinities of both signs, and a NaN"
