"""The calls around attention as they are used together: a prompt's projection normed and turned, kept in pages,
attended over, weighed and cut down, and the next tokens over what is left; and a training step through the ring."""
import numpy as np
import pytest
import torch

from oracle import backward as oback
from oracle import evict as oevict
from oracle import paged as opaged
from oracle import qk_norm as onorm
from tests.gpu_util import dev, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ra():
    from online_softmax_attention_zigzag_gb300 import ringattn
    ringattn.lib()
    torch.cuda.set_device(0)
    return ringattn


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device=dev())


def table(n, rot):
    a = torch.arange(n).double()[:, None] * 1e4 ** (-torch.arange(0, rot, 2).double() / rot)
    return torch.cat([a.cos(), a.sin()], 1).float().to(dev())


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_prompt_eviction_and_next_tokens(ra, e4m3, d):
    """A prompt of 333, cut down to 120 positions a head, then six tokens one by one.  Every step against the oracle on
    what the step before left on the device."""
    hq, hkv, page, S, keep, more = 8, 2, 32, 333, 120, 6
    g = torch.Generator().manual_seed(d)
    qkv = torch.randn((S + more, hq + 2 * hkv, d), generator=g).to(torch.bfloat16).to(dev())
    w = [(1 + 0.1 * torch.randn(d, generator=g)).to(torch.bfloat16).to(dev()) for _ in range(2)]
    cs = table(S + more, d)
    pages = -(-(S + more) // page)
    bt = torch.randperm(pages, generator=g).to(torch.int32)[None].to(dev())
    cache = [torch.zeros((pages, hkv, page, d), device=dev()).to(torch.float8_e4m3fn if e4m3 else torch.bfloat16) for _ in range(2)]
    scale = [torch.zeros((pages, hkv, page), device=dev()) if e4m3 else None for _ in range(2)]
    kw = dict(k_scale=scale[0], v_scale=scale[1])
    weights = torch.full((pages, hkv, page), float("nan"), device=dev())
    length = 0

    def step(a, b):
        nonlocal length
        n = b - a
        q = torch.empty((n, hq, d), dtype=torch.bfloat16, device=dev())
        k = torch.empty((n, hkv, d), dtype=torch.bfloat16, device=dev())
        pos = torch.arange(a, b, dtype=torch.int32, device=dev())
        ra.qk_norm_rope(qkv[a:b, :hq], qkv[a:b, hq:hq + hkv], q, k, pos, cs, q_weight=w[0], k_weight=w[1], q_scale=d ** -0.5)
        length += n
        cu, ln = ints(0, n), ints(length)
        ra.cache_append(k, qkv[a:b, hq + hkv:], *cache, bt, cu, ln, **kw)
        out, lse = torch.empty((n, hq, d), device=dev()), torch.empty((n, hq), device=dev())
        ws = torch.empty(ra.paged_workspace_bytes(n, 1, hq, hkv, d, n), dtype=torch.uint8, device=dev())
        ra.fwd_paged(q, *cache, out, lse, bt, cu, ln, ws, max_q=n, **kw)
        before = seen(weights)
        ra.cache_weights(q, lse, *cache, weights, bt, cu, ln, ws, max_q=n, decay=0.9, **kw)
        assert ra.sync_status() == ra.RA_OK
        z, _ = onorm.forward(f64(qkv[a:b, :hq]), f64(w[0]), f64(cs[a:b]), scale=d ** -0.5)
        assert np.abs(f64(q) - z).max() <= 2.0 ** -7 * np.abs(z).max()
        kk, vv = (f64(x) for x in (seen(cache[0], scale[0]), seen(cache[1], scale[1])))
        o, l, _, _ = opaged.attention(f64(q), kk, vv)
        assert np.abs(f64(out) - o).max() <= 2e-2 and np.abs(f64(lse) - l).max() <= 1e-3
        want, _ = oevict.add_weights(f64(before), f64(q), f64(lse), kk, 0.9)
        # scores of some units: 2^-23 (d + 16) of sum |q k| <= 16, the sum of n g probabilities, and so on, as in the
        # operator's own tests
        assert np.allclose(f64(seen(weights)), want, rtol=(d + 16) * 16 * 2.0 ** -23 + 4 * n * 2.0 ** -24 + 2.0 ** -18, atol=0)

    def seen(x, s=None):
        """Positions [0, length), as fp32."""
        p = torch.arange(length, device=dev())
        pg, row = bt[0].long()[p // page], p % page
        y = x.view(torch.uint8)[pg, :, row].view(x.dtype).float() if x.dtype is torch.float8_e4m3fn else x[pg, :, row].float()
        return y if s is None else y * s[pg, :, row][..., None]

    step(0, S)
    # a row's weights add up to 1: the prompt's rows, g heads of each
    assert np.allclose(f64(seen(weights)).sum(0), S * hq / hkv, rtol=1e-5)
    was = [f64(seen(cache[0], scale[0])), f64(seen(cache[1], scale[1])), f64(seen(weights))]
    new_len, kept = ints(0), torch.empty((1, hkv, keep), dtype=torch.int32, device=dev())
    ra.cache_evict(*cache, weights, bt, ints(length), ints(keep), new_len, kept, sinks=4, recent=16, **kw)
    assert ra.sync_status() == ra.RA_OK
    length = int(new_len)
    assert length == keep
    for h in range(hkv):
        j = oevict.stay(was[2][:, h].tolist(), keep, 4, 16)
        assert kept[0, h].tolist() == j
        for now, then in zip((seen(cache[0], scale[0]), seen(cache[1], scale[1]), seen(weights)), was):
            assert np.array_equal(f64(now)[:, h], then[j, h])
    for t in range(S, S + more):
        step(t, t + 1)
    assert length == keep + more


@pytest.mark.parametrize("d,inter", [(64, 0), (128, 1)])
def test_training_step_through_the_ring(ra, d, inter):
    """Projection -> norm and rotation, head-major -> ring attention and its backward -> gradients of the projection and
    of the weights, against the float64 gradients of the whole.  q and k are rounded to bf16 between the steps on both sides."""
    S, hq, hkv, c = 512, 4, 2, 2
    g = torch.Generator().manual_seed(d)
    qkv = torch.randn((S, hq + 2 * hkv, d), generator=g).to(torch.bfloat16).to(dev())
    w = [(1 + 0.1 * torch.randn(d, generator=g)).to(dev()) for _ in range(2)]
    cs, pos = table(S, d), torch.arange(S, dtype=torch.int32, device=dev())
    q, k = (torch.empty((h, S, d), dtype=torch.bfloat16, device=dev()) for h in (hq, hkv))
    scale = d ** -0.5
    kw = dict(q_weight=w[0], k_weight=w[1], q_scale=scale, interleaved=inter)
    ra.qk_norm_rope(qkv[:, :hq], qkv[:, hq:hq + hkv], q.transpose(0, 1), k.transpose(0, 1), pos, cs, **kw)
    v = qkv[:, hq + hkv:].transpose(0, 1).contiguous()
    ring = dict(c=c, causal=1, layout=1, kv_block=128)
    out, lse = ra.attention(q, k, v, **ring)
    dout = torch.randn((hq, S, d), generator=g).to(torch.bfloat16).to(dev())
    dq, dk, dv = ra.attention_backward(q, k, v, out, lse, dout, **ring)
    dqkv = torch.full_like(qkv, float("nan"))
    dw = [torch.empty(d, device=dev()) for _ in range(2)]
    ws = torch.empty(ra.qk_norm_rope_workspace_bytes(S, hq, hkv, d), dtype=torch.uint8, device=dev())
    ra.qk_norm_rope_bwd(qkv[:, :hq], qkv[:, hq:hq + hkv], dq.transpose(0, 1), dk.transpose(0, 1), dqkv[:, :hq], dqkv[:, hq:hq + hkv], pos, cs, ws,
                        dq_weight=dw[0], dk_weight=dw[1], **kw)
    assert ra.sync_status() == ra.RA_OK
    assert torch.isnan(dqkv[:, hq + hkv:]).all()
    gq, gk, _ = oback.attention_grad(*(f64(x) for x in (q, k, v, dout)), True, out=f64(out))
    aq, ak, _ = oback.grad_abs_sums(*(f64(x) for x in (q, k, v, dout)), True, out=f64(out))
    for i, (x, grad, ab, got, s) in enumerate(((qkv[:, :hq], gq, aq, dqkv[:, :hq], scale), (qkv[:, hq:hq + hkv], gk, ak, dqkv[:, hq:hq + hkv], 1.0))):
        dx, dwx, dx_abs, _ = onorm.backward(f64(x), f64(w[i]), f64(cs), grad.transpose(1, 0, 2), inter, scale=s)
        # the ring's gradients are off by 2^-8 of their terms' absolute sums; that goes through the same linear map
        _, _, err, dw_err = onorm.backward(f64(x), f64(w[i]), f64(cs), (2.0 ** -8 * ab + 1e-6 * ab.max()).transpose(1, 0, 2), inter, scale=s)
        tol = err + 2.0 ** -17 * dx_abs
        tol = tol + 2.0 ** -8 * (np.abs(dx) + tol)
        worst = (np.abs(f64(got) - dx) / tol).max()
        assert worst <= 1.0, f"d{'qk'[i]} off by {worst:.3g} of its bound"
        worst = (np.abs(f64(dw[i]) - dwx) / (dw_err + 2.0 ** -14 * np.abs(dwx) + 1e-4)).max()
        assert worst <= 1.0, f"d{'qk'[i]}_weight off by {worst:.3g} of its bound"
