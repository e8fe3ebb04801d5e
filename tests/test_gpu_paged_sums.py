"""Sums of the few-row paged kernel over millions of keys in one group of warps' hands, weights unequal
and values of one sign: the tensor cores truncate every addend, so nothing averages out."""
import math

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


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("n,std,d", [(1, 0.0, 128), (1, 0.3, 128), (2, 1.0, 128), (1, 3.0, 128), (1, 0.3, 64), (2, 3.0, 64)])
def test_millions_of_keys(ra, e4m3, n, std, d):
    """2^22 keys (one page 64 times) of as many sequences as there are groups of warps: every group has whole
    sequences.

    A group's sums end after 256 tiles of 128 keys.  In these every warp adds 1024 times (bf16: 32 keys as
    two products for each half of P; e4m3: 64 keys as four) 16 addends to a sum, each of the 17 cut off by
    less than 2^-23 of that sum; it grows from 0, so that is half as much of the whole on average.  P is kept to 2^-15
    at least (two bf16 halves) or 2^-11 (fp16), scores and exponentials to 2^-17 (sums of d = 128
    products below 2 in all, 2^-21 for the exponential); adding 128 of them up takes 2^-17."""
    hq, L, page = 8, 2 ** 22, 65536
    B = 4 * torch.cuda.get_device_properties(0).multi_processor_count
    dt = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    g = torch.Generator(device=dev()).manual_seed(101)
    v = (torch.rand((1, 1, page, d), device=dev(), generator=g) + 0.1).to(dt)
    k = torch.randn((1, 1, page, d), device=dev(), generator=g).to(dt)
    one = torch.ones((1, 1, page), device=dev()) if e4m3 else None
    table = torch.zeros((B, L // page), dtype=torch.int32, device=dev())
    cu = torch.arange(0, B * n + 1, n, dtype=torch.int32, device=dev())
    ln = torch.full((B,), L, dtype=torch.int32, device=dev())
    q = (torch.randn((B * n, hq, d), device=dev(), generator=g) * std * d ** -0.5).to(torch.bfloat16)
    out, lse = torch.empty((B * n, hq, d), device=dev()), torch.empty((B * n, hq), device=dev())
    ws = torch.empty(ra.paged_workspace_bytes(B * n, B, hq, 1, d, n), dtype=torch.uint8, device=dev())
    ra.fwd_paged(q, k, v, out, lse, table, cu, ln, ws, max_q=n, causal=0, k_scale=one, v_scale=one)
    assert ra.sync_status() == ra.RA_OK
    tol = 17 * 1024 / 2 * 2.0 ** -23 + (2.0 ** -11 if e4m3 else 2.0 ** -15) + 2.0 ** -17 + 2.0 ** -17
    for b in (0, B // 3, B - 1):
        rows = slice(b * n, (b + 1) * n)
        x = q[rows].double().reshape(n * hq, d) @ k[0, 0].double().T
        want = torch.softmax(x, 1) @ v[0, 0].double()
        off = (out[rows].double().reshape(n * hq, d) / want - 1).abs().max().item()
        assert off <= tol, f"sequence {b}: out off by {off:.3g}, {tol:.3g} allowed"
        want = torch.logsumexp(x, 1) + math.log(L // page)
        off = (lse[rows].double().reshape(-1) - want).abs().max().item()
        assert off <= 2.0 ** -16 + 2.0 ** -22 * want.abs().max().item()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("n,window,sinks", [(1, 0, 0), (2, 0, 0), (1, 60000, 200), (2, 50000, 1000)])
def test_stretches_whose_maximum_grows(ra, e4m3, n, window, sinks):
    """A part of 547 tiles for a group (the same pages for all its sequences), so three stretches, with scores that grow
    along the keys, or shrink; the sequence of another group in two parts; an infinite value in the first stretch."""
    hq, d, L = 8, 128, 70000
    B = 4 * torch.cuda.get_device_properties(0).multi_processor_count + 1  # (one more than groups: some parts are cut)
    for grow in (True, False):
        S = Batch([(n, L)], hkv=1, d=d, page=512, e4m3=e4m3, device=dev(), seed=82, fill=False)
        ramp = torch.arange(L)[:, None, None] / L
        S.k[0] = (S.k[0].float() * (0.5 + 3.5 * (ramp if grow else 1 - ramp))).to(torch.bfloat16)
        at = 150 if window else 20000  # (a sink)
        if not e4m3:
            S.v[0][at, 0, 9] = float("inf")
        S.fill()
        q = (torch.randn((B * n, hq, d), generator=torch.Generator().manual_seed(83)) * 0.3).to(torch.bfloat16)
        out, lse = torch.empty((B * n, hq, d), device=dev()), torch.empty((B * n, hq), device=dev())
        cu = torch.arange(0, B * n + 1, n, dtype=torch.int32, device=dev())
        ws = torch.full((ra.paged_workspace_bytes(B * n, B, hq, 1, d, n),), 255, dtype=torch.uint8, device=dev())
        ra.fwd_paged(q.to(dev()), S.k_cache, S.v_cache, out, lse, S.dtable.expand(B, -1).contiguous(), cu, S.dlen.expand(B).contiguous(),
                     ws, max_q=n, window=window, sinks=sinks, **S.kw())
        assert ra.sync_status() == ra.RA_OK
        k, v = S.kept(0)
        if not e4m3:
            v[at, 0, 9] = 0.0
        keep = [c for c in range(d) if c != 9]
        for b in (0, B - 1):
            rows = slice(b * n, (b + 1) * n)
            ref = opaged.attention(q[rows].double().numpy(), k, v, True, window, sinks)
            check(out[rows][..., keep], lse[rows], [x[..., keep] if x.ndim == 3 else x for x in ref], d, False, f"sequence {b}, {grow}")
            if not e4m3:
                assert torch.isposinf(out[rows][..., 9]).all()
