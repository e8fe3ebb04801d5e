"""ringattn_qk_norm_rope and its backward pass over all of bf16's range, with and without an eps: rows whose squares, or whose
sum of squares, no fp32 holds."""
import numpy as np
import pytest
import torch

from oracle import qk_norm as onorm
from tests.gpu_util import dev, f64
from tests.test_gpu_qk_norm import BF, F32, Case, check_forward, ra  # noqa: F401

pytestmark = pytest.mark.gpu

EXPONENTS = [-133, -130, -126, -110, -100, -85, -80, -76, -75, -74, -70, -64, -63, -60, -45, -31, -30, -29, 0, 29, 30, 31, 40, 59, 60, 61,
             63, 64, 90, 110, 125]


def exponents(eps):
    """All of them; with an eps from 2^-60 on, those whose squares fp32 holds."""
    return [e for e in EXPONENTS if eps < 2.0 ** -60 or e <= 59]


def case(es, d, hq=3, hkv=2, seed=0, **kw):
    """A token an exponent, every head's row times 2 to it."""
    c = Case(len(es), hq, hkv, d, seed=seed, **kw)
    for x in c.x:
        for t, e in enumerate(es):
            # (in two steps: 2^-133 is no fp32 number to multiply by, and 2^125 times a row's largest, below 4, is one)
            x[t] = (x[t].double().clamp(-3.9, 3.9) * 2.0 ** e).to(BF)
        # a row of one small element among zeros, and one of a large element among small ones
        x[:, -1] = 0.0
        x[:, -1, 5] = torch.tensor([2.0 ** e for e in es]).to(BF)
        x[::2, -1, 6] = 2.0 ** -133
    return c


@pytest.mark.parametrize("eps", [0.0, 1e-45, 1e-38, 1e-30, 1e-19, 1e-6, 1e20, 1e38])
@pytest.mark.parametrize("d,rot", [(64, 32), (128, 128)])
@pytest.mark.parametrize("inter", [0, 1])
def test_forward(ra, eps, d, rot, inter):
    c = case(exponents(eps), d, rot=rot)
    eps = float(np.float32(eps))
    out = c.rows()
    ra.qk_norm_rope(*c.rows(c.x), *out, *c.args(), eps=eps, q_scale=0.5, interleaved=inter, **c.kw())
    assert ra.sync_status() == ra.RA_OK
    check_forward(c, out, inter, eps, 0.5)


@pytest.mark.parametrize("eps", [0.0, 1e-30, 1e-6])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("types", [(F32, F32), (BF, BF), (F32, BF)])
@pytest.mark.parametrize("inter", [0, 1])
def test_backward(ra, eps, d, types, inter):
    """Gradients of rows of size 2^e are of size 2^-e: bounds relative to the terms' absolute sum, as in the other tests, and
    half a step of the smallest numbers of fp32 and of bf16 (2^-149, 2^-133)."""
    eps = float(np.float32(eps))
    es = exponents(eps)
    c = case(es, d, rot=d // 2, w="fp32")
    for x in c.dz:
        for t, e in enumerate(es):
            if e < -100:
                x[t] *= 2.0 ** -30
    dz = [x.to(types[0]) for x in c.dz]
    grads = c.rows(dtype=types[1])
    dw = [torch.full((d,), float("nan"), device=dev()) for _ in range(2)]
    ws = torch.empty(ra.qk_norm_rope_workspace_bytes(c.T, 3, 2, d), dtype=torch.uint8, device=dev())
    ra.qk_norm_rope_bwd(*c.rows(c.x), *c.rows(dz, types[0]), *grads, *c.args(), ws, dq_weight=dw[0], dk_weight=dw[1], eps=eps, q_scale=0.5,
                        interleaved=inter, **c.kw())
    assert ra.sync_status() == ra.RA_OK
    for i in range(2):
        dx, dwx, dx_abs, dw_abs = onorm.backward(c.x[i].double().numpy(), c.w64(i), c.cs(), dz[i].double().numpy(), inter, eps, 0.5 if i == 0 else 1.0)
        # (a few products of fp32's smallest numbers: whole steps of 2^-149, times r where they come before it, at most 2^8 once x is about 1)
        tol = 2.0 ** -17 * dx_abs + 2.0 ** -140
        if types[1] is BF:
            tol = tol + 2.0 ** -8 * (np.abs(dx) + tol) + 2.0 ** -134
        worst = (np.abs(f64(grads[i]) - dx) / tol).max(axis=(1, 2))
        assert (worst <= 1.0).all(), [(e, float(w)) for e, w in zip(es, worst) if not w <= 1.0]
        worst = (np.abs(f64(dw[i]) - dwx) / ((2.0 ** -19 + 400 * 2.0 ** -24) * dw_abs + 1e-30)).max()
        assert worst <= 1.0, f"d{'qk'[i]}_weight off by {worst:.3g} of its bound"


def test_rows_far_out_change_no_others(ra):
    """Bits of ordinary rows, alone and with the others beside them in the same warps."""
    alone, mixed = Case(64, 6, 2, 64, 32, seed=3), Case(64, 6, 2, 64, 32, seed=3)
    for x in mixed.x:
        x[::3] = (x[::3].double() * 2.0 ** -90).to(BF)
        x[1::3, 1] = (x[1::3, 1].double() * 2.0 ** 80).to(BF)
    res = []
    for c in (alone, mixed):
        out, g = c.rows(), c.rows(dtype=F32)
        ra.qk_norm_rope(*c.rows(c.x), *out, *c.args(), eps=0.0, **c.kw())
        ra.qk_norm_rope_bwd(*c.rows(c.x), *c.rows(c.dz, F32), *g, *c.args(), eps=0.0, **c.kw())
        assert ra.sync_status() == ra.RA_OK
        res.append((*out, *g))
    for a, b in zip(*res):
        assert torch.equal(a[2::3], b[2::3]) and torch.equal(a[1::3, 0], b[1::3, 0])
        assert not torch.isnan(b.float()).any()


@pytest.mark.parametrize("eps", [0.0, 1e-30])
def test_rows_of_zeros(ra, eps):
    """0 / 0 without an eps, else zeros; the row beside them is as ever."""
    c = Case(4, 2, 1, 64, 32, seed=5)
    for x in c.x:
        x[[0, 2]] = 0.0
    out = c.rows()
    ra.qk_norm_rope(*c.rows(c.x), *out, *c.args(), eps=eps, **c.kw())
    assert ra.sync_status() == ra.RA_OK
    for i, o in enumerate(out):
        z = o[[0, 2]].float()
        assert torch.isnan(z).all() if eps == 0.0 else not z.any()
    c.x, c.pos, c.T = [x[[1, 3]] for x in c.x], c.pos[[1, 3]], 2
    check_forward(c, [o[[1, 3]] for o in out], 0, eps, 1.0)
