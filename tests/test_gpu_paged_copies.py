"""cache_append and cache_read of large calls, whose kernels find the places of a block's tokens once and move four
pieces a thread: bit-exact, in ragged batches with padding, rows before position 0, pages that are none,
strided rows and last blocks of every size."""
import numpy as np
import pytest
import torch

from oracle import paged as opaged
from tests.gpu_util import dev
from tests.paged_util import Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ra():
    from online_softmax_attention_zigzag_gb300 import ringattn
    ringattn.lib()
    torch.cuda.set_device(0)
    return ringattn


def _large(total, hkv, d):
    """More pieces of 16 bytes than eight waves of full SMs take at one a thread."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return hkv * d // 8 * total > 8 * 2048 * sms


def _bits(t):
    return t.contiguous().view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("hkv,d,page,seqs,layout,pad", [
    (8, 128, 64, [(19999, 20100), (3, 2), (700, 9000), (0, 50), (1, 1)], "plain", 5),
    (3, 128, 48, [(33000, 33000), (20001, 20000)], "fused", 0),     # 21 tokens a block
    (8, 64, 16, [(1, 70)] * 40 + [(41001, 41007)], "heads", 1),
    (1, 64, 256, [(300001, 300300), (20007, 20007)], "plain", 63),   # 64 tokens a block, its largest number
    (40, 128, 32, [(4001, 4100), (5, 4)], "plain", 0),              # a token is more than a block moves at once
])
def test_large_calls_are_bit_exact(ra, e4m3, hkv, d, page, seqs, layout, pad):
    kw = dict(hkv=hkv, d=d, page=page, e4m3=e4m3, device=dev(), seed=1, pad=pad, fill=False, gap=8)
    B, want = Batch(seqs, **kw), Batch(seqs, **kw)
    assert _large(B.total, hkv, d)
    g = torch.Generator(device=dev()).manual_seed(2)
    rand = lambda *s: torch.randn(s, generator=g, device=dev()).to(torch.bfloat16)  # noqa: E731
    if layout == "fused":
        qkv = rand(B.total, 4 + 2 * hkv, d)
        kn, vn = qkv[:, 4:4 + hkv], qkv[:, 4 + hkv:]
    elif layout == "heads":
        kn, vn = (rand(hkv, B.total, d).transpose(0, 1) for _ in range(2))
    else:
        kn, vn = rand(B.total, hkv, d), rand(B.total, hkv, d)
    bad = seqs[0][1] // page // 2  # a page of the first sequence that is none
    hole = seqs[0][1] > 2 * page
    if hole:
        B.dtable[0, bad] = B.n_pages
    ra.cache_append(kn, vn, B.k_cache, B.v_cache, *B.args(), **B.kw())
    assert ra.sync_status() == ra.RA_OK
    cu = B.cu.tolist()
    stored = [torch.zeros((hkv, B.total, d), dtype=torch.bfloat16, device=dev()) for _ in range(2)]
    for x, cache, scale, out in ((kn, want.k_cache, want.k_scale, stored[0]), (vn, want.v_cache, want.v_scale, stored[1])):
        if e4m3:
            c, s = opaged.quantise(x.double().cpu().numpy())
            codes = torch.from_numpy(c.astype(np.float32)).to(dev()).to(torch.float8_e4m3fn)
            scales = torch.from_numpy(s.astype(np.float32)).to(dev())
            kept = (codes.float() * scales[..., None]).to(torch.bfloat16)
        else:
            kept = x
        for b, (n, L) in enumerate(seqs):
            m = min(n, L)
            pos = torch.arange(L - m, L)
            use = torch.ones(m, dtype=torch.bool) if not hole or b else pos // page != bad
            pg, row = (y[L - m:][use.to(dev())] for y in want.places(b))
            at = (torch.arange(cu[b + 1] - m, cu[b + 1])[use]).to(dev())
            if e4m3:
                cache.view(torch.uint8)[pg, :, row] = codes[at].view(torch.uint8)
                scale[pg, :, row] = scales[at]
            else:
                cache[pg, :, row] = x[at]
            out[:, at] = kept[at].transpose(0, 1)
    for a, b in ((B.k_cache, want.k_cache), (B.v_cache, want.v_cache)) + (
            ((B.k_scale, want.k_scale), (B.v_scale, want.v_scale)) if e4m3 else ()):
        assert torch.equal(_bits(a), _bits(b))
    ko, vo = (torch.full((hkv, B.total, d), float("nan"), dtype=torch.bfloat16, device=dev()) for _ in range(2))
    ra.cache_read(B.k_cache, B.v_cache, ko, vo, *B.args(), **B.kw())
    assert ra.sync_status() == ra.RA_OK
    for got, ref in zip((ko, vo), stored):
        assert torch.equal(got[:, :cu[-1]], ref[:, :cu[-1]])  # zeros where nothing is kept
        assert torch.isnan(got[:, cu[-1]:].float()).all()
