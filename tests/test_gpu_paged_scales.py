"""An e4m3 cache whose scales are no powers of two, as another program may have written it."""
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


def _bf16(x):
    return torch.from_numpy(x).float().to(torch.bfloat16).double().numpy()


@pytest.mark.parametrize("n", [1, 2, 20, 200])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("size", [1.0, 3e4, 1e-30])  # of V's scales; above 128 the chunk kernel takes them in two factors
def test_any_positive_scale(ra, n, d, size):
    """Few rows multiply with the scales in fp32; the chunk kernel rounds the scale to bf16 and then its product with the
    code; cache_read rounds the exact product."""
    hq, hkv, L = 8, 2, 900
    B = Batch([(n, L), (min(n, 3), 77)], hkv=hkv, d=d, page=32, e4m3=True, device=dev(), seed=1)
    g = torch.Generator().manual_seed(2)
    few = n * hq // hkv <= 16
    kept, exact = [], []
    for b in range(2):
        page, row = B.places(b)
        for x, cache, scale, f in ((B.k, B.k_cache, B.k_scale, 1.0), (B.v, B.v_cache, B.v_scale, size)):
            s = scale[page, :, row].cpu() * f * (0.5 + torch.rand(scale[page, :, row].shape, generator=g))
            scale[page, :, row] = s.to(dev())
            codes = cache.view(torch.uint8)[page, :, row].view(torch.float8_e4m3fn).double().cpu().numpy()
            s = s.double().numpy()[..., None]
            exact.append(codes * s)
            kept.append(codes * s if few else _bf16(codes * _bf16(s)))
    q = (torch.randn((B.total, hq, d), generator=g) * d ** -0.5).to(torch.bfloat16)
    out, lse = torch.empty((B.total, hq, d), device=dev()), torch.empty((B.total, hq), device=dev())
    ws = torch.empty(ra.paged_workspace_bytes(B.total, 2, hq, hkv, d, B.max_q), dtype=torch.uint8, device=dev())
    ra.fwd_paged(q.to(dev()), B.k_cache, B.v_cache, out, lse, *B.args(), ws, max_q=B.max_q, **B.kw())
    assert ra.sync_status() == ra.RA_OK
    cu = B.cu.tolist()
    for b in range(2):
        rows = slice(cu[b], cu[b + 1])
        ref = opaged.attention(q[rows].double().numpy(), kept[2 * b], kept[2 * b + 1] / size)
        # (few rows: a scale's logarithm is off by 2^-21 and a step of 2^-18 of its size, up to 128, moves p alike)
        check(out[rows].double() / size, lse[rows], ref, d, False, f"sequence {b}", 2.0 ** -11 + 2.0 ** -17 if few else 2.0 ** -8)
    # reading back: the product of code and scale, rounded once
    B.dcu = torch.tensor([0, L, L + 77], dtype=torch.int32, device=dev())
    ko, vo = (torch.empty((hkv, L + 77, d), dtype=torch.bfloat16, device=dev()) for _ in range(2))
    ra.cache_read(B.k_cache, B.v_cache, ko, vo, *B.args(), **B.kw())
    assert ra.sync_status() == ra.RA_OK
    for b, at in ((0, slice(0, L)), (1, slice(L, L + 77))):
        for got, x in ((ko, exact[2 * b]), (vo, exact[2 * b + 1])):
            assert np.array_equal(got[:, at].double().cpu().numpy().transpose(1, 0, 2), _bf16(x))
