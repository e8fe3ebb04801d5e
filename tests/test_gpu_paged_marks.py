"""Long contexts whose every tile of values shows in out, and the precision that each kernel keeps of its
probabilities, in fp32 outputs."""
import numpy as np
import pytest
import torch

from oracle import paged as opaged
from tests.gpu_util import dev
from tests.paged_util import Batch, check


@pytest.fixture(scope="module")
def ra():
    from online_softmax_attention_zigzag_gb300 import ringattn
    ringattn.lib()
    torch.cuda.set_device(0)
    return ringattn


def _marked(L, hkv, d, seed):
    """Values around 1, tile t of 128 keys with 100 in column t % d: a tile that is lost, taken twice or put in
    another's place moves a column by a tenth of itself and more."""
    v = 1 + 0.1 * torch.randn((L, hkv, d), generator=torch.Generator().manual_seed(seed))
    j = torch.arange(L)
    v[j, :, (j // 128) % d] = 100.0
    return v.to(torch.bfloat16)


def _queries(n, hq, d, seed):
    return (torch.randn((n, hq, d), generator=torch.Generator().manual_seed(seed)) * d ** -0.5).to(torch.bfloat16)


def _attend(ra, B, q, **kw):
    total, hq, d = q.shape
    out, lse = torch.empty((total, hq, d), device=dev()), torch.empty((total, hq), device=dev())
    ws = torch.empty(ra.paged_workspace_bytes(total, len(B.seqs), hq, B.hkv, d, B.max_q), dtype=torch.uint8, device=dev())
    ra.fwd_paged(q.to(dev()), B.k_cache, B.v_cache, out, lse, *B.args(), ws, max_q=B.max_q, **B.kw(), **kw)
    assert ra.sync_status() == ra.RA_OK
    return out, lse


# n, hq, hkv, d, L, window, sinks: a part of hundreds, parts of items of one unit and of two
LONG = [(1, 8, 1, 128, 60001, 0, 0), (2, 8, 1, 64, 30000, 0, 0), (14, 8, 2, 128, 15041, 0, 0), (40, 8, 1, 128, 50000, 0, 0),
        (300, 4, 1, 128, 20000, 0, 0), (200, 8, 2, 64, 20011, 0, 0), (1, 8, 1, 128, 60001, 30000, 200), (60, 4, 1, 128, 40000, 20000, 300)]


@pytest.mark.gpu
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("n,hq,hkv,d,L,window,sinks", LONG)
def test_every_tile_of_a_long_context(ra, e4m3, n, hq, hkv, d, L, window, sinks):
    B = Batch([(n, 300), (n, L), (1, 40)], hkv=hkv, d=d, page=48, e4m3=e4m3, device=dev(), seed=3, fill=False)
    B.v[1] = _marked(L, hkv, d, 4)
    B.fill()
    q = _queries(B.total, hq, d, 5)
    out, lse = _attend(ra, B, q, window=window, sinks=sinks)
    cu = B.cu.tolist()
    for b in range(3):
        rows = slice(cu[b], cu[b + 1])
        ref = opaged.attention(q[rows].double().numpy(), *B.kept(b), True, window, sinks)
        check(out[rows], lse[rows], ref, d, False, f"sequence {b}")


@pytest.mark.parametrize("n,hq,hkv,d,L,window,sinks", LONG)
def test_a_lost_tile_would_show(n, hq, hkv, d, L, window, sinks):
    """Host: the same inputs with one tile's values missing, or two tiles changed over, in the reference."""
    n, hq = min(n, 4), hq // hkv
    k = torch.randn((L, 1, d), generator=torch.Generator().manual_seed(6)).double().numpy()
    v = _marked(L, 1, d, 4).double().numpy()
    q = _queries(n, hq, d, 5).double().numpy()
    ref = opaged.attention(q, k, v, True, window, sinks)
    out, lse = (torch.from_numpy(x) for x in ref[:2])
    check(out, lse, ref, d, False)
    first = (L - n - window) // 128 + 2 if window else 0
    for t in (first, (first + L // 128) // 2, L // 128 - 1):
        lost = v.copy()
        lost[t * 128:(t + 1) * 128] = 0
        swapped = v.copy()
        swapped[t * 128:(t + 1) * 128] = 1  # another tile's values: this one's mark is gone
        for wrong in (lost, swapped):
            with pytest.raises(AssertionError):
                check(out, lse, opaged.attention(q, k, wrong, True, window, sinks), d, False)


# What a probability is rounded to on its way to V.  Few rows, bf16: a half that is cut off leaves less than 2^-7
# of p, whose own half is off by 2^-8 of that, and the half is 2^-20 of p too large on purpose.  Few rows, e4m3: fp16, 2^-11.
P_EPS = {False: 2.0 ** -15 + 2.0 ** -20, True: 2.0 ** -11}


@pytest.mark.gpu
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("n,hq,hkv,d", [(1, 8, 1, 128), (2, 8, 1, 128), (1, 8, 2, 64), (4, 4, 1, 64)])
def test_precision_of_the_few_row_kernel(ra, e4m3, n, hq, hkv, d):
    """Values of one sign and small scores: what is lost of p is lost of out."""
    L = 1800
    B = Batch([(n, L), (n, 130)], hkv=hkv, d=d, page=32, e4m3=e4m3, device=dev(), seed=7, fill=False)
    for b in range(2):
        B.v[b] = (B.v[b].float().abs() + 0.5).to(torch.bfloat16)
    B.fill()
    q = (_queries(B.total, hq, d, 8).float() * 0.2).to(torch.bfloat16)
    out, lse = _attend(ra, B, q)
    cu = B.cu.tolist()
    for b in range(2):
        rows = slice(cu[b], cu[b + 1])
        ref = opaged.attention(q[rows].double().numpy(), *B.kept(b))
        check(out[rows], lse[rows], ref, d, False, f"sequence {b}", P_EPS[e4m3])


@pytest.mark.parametrize("e4m3", [False, True])
def test_a_coarser_probability_would_show(e4m3):
    """Host: p cut off to one bf16 half misses either bound."""
    n, hq, d, L = 1, 8, 128, 1800
    g = torch.Generator().manual_seed(9)
    k, v = torch.randn((L, 1, d), generator=g).double().numpy(), (torch.randn((L, 1, d), generator=g).abs() + 0.5).double().numpy()
    q = (_queries(n, hq, d, 8).float() * 0.2).double().numpy()
    ref = opaged.attention(q, k, v)
    s = q[0] @ k[:, 0].T
    p = np.exp(s - s.max(1, keepdims=True))
    x = torch.from_numpy(p).float()
    cut = (x.view(torch.int32) & -65536).view(torch.float32).double().numpy()  # a first half alone
    kept = p if not e4m3 else x.to(torch.float16).double().numpy()
    lse = torch.from_numpy(ref[1])

    def hold(p2):
        check(torch.from_numpy(p2 @ v[:, 0] / p.sum(1, keepdims=True))[None], lse, ref, d, False, p_eps=P_EPS[e4m3])

    hold(kept)
    with pytest.raises(AssertionError):
        hold(cut)
