"""ringattn_qk_norm_rope and its backward pass against the float64 oracle."""
import numpy as np
import pytest
import torch

from oracle import qk_norm as onorm
from tests.gpu_util import dev, f64

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def ra():
    from online_softmax_attention_zigzag_gb300 import ringattn
    ringattn.lib()
    torch.cuda.set_device(0)
    return ringattn


class Case:
    """q, k, weights, table and positions; layout: "token" or "head" major rows, or slices of a fused projection."""

    def __init__(self, T, hq=4, hkv=2, d=128, rot=None, w="bf16", layout="token", n_pos=600, seed=0, std=1.0):
        g = torch.Generator().manual_seed(seed)
        self.T, self.hq, self.hkv, self.d, self.rot, self.layout = T, hq, hkv, d, d if rot is None else rot, layout
        self.n_pos = n_pos
        self.x = [(torch.randn((T, h, d), generator=g) * std).to(BF) for h in (hq, hkv)]
        a = torch.arange(n_pos).double()[:, None] * 1e4 ** (-torch.arange(0, self.rot, 2).double() / max(1, self.rot))
        self.table = torch.cat([a.cos(), a.sin()], 1).float()
        self.pos = torch.randint(0, n_pos, (T,), generator=g).to(torch.int32)
        self.w = [None, None]
        if w != "none":
            self.w = [(1 + 0.3 * torch.randn(d, generator=g)).to(BF if w == "bf16" else F32) for _ in range(2)]
        self.dz = [torch.randn((T, h, d), generator=g) for h in (hq, hkv)]

    def rows(self, xs=None, dtype=BF, layout=None):
        """Device tensors [T, H, d] in the case's layout, holding xs (NaN where None)."""
        layout = layout or self.layout
        xs = xs or [torch.full((self.T, h, self.d), float("nan")) for h in (self.hq, self.hkv)]
        if layout == "fused":
            f = torch.full((self.T, self.hq + 2 * self.hkv, self.d), float("nan"), dtype=dtype, device=dev())
            r = [f[:, :self.hq], f[:, self.hq:self.hq + self.hkv]]
        elif layout == "head":
            r = [torch.empty((x.shape[1], self.T, self.d), dtype=dtype, device=dev()).transpose(0, 1) for x in xs]
        else:
            r = [torch.empty(x.shape, dtype=dtype, device=dev()) for x in xs]
        for a, b in zip(r, xs):
            a.copy_(b.to(dtype))
        return r

    def kw(self):
        wd = [None if w is None else w.to(dev()) for w in self.w]
        return dict(q_weight=wd[0], k_weight=wd[1])

    def args(self):
        return self.pos.to(dev()), self.table.to(dev())

    def w64(self, i):
        return None if self.w[i] is None else self.w[i].double().numpy()

    def cs(self):
        return self.table[self.pos.long()].double().numpy()


def check_forward(c, out, inter, eps, scale):
    """fp32 arithmetic: every term x r c or x r s carries the rounding of the sum of squares (d / 8 + 8 additions, less
    than 2^-19 of it), of rsqrt (2^-22) and of six products and sums (2^-24 each): 2^-18 of the terms' absolute sum
    covers them; then one rounding to bf16, half a step of 2^-8."""
    for i, got in enumerate(out):
        want, mag = onorm.forward(c.x[i].double().numpy(), c.w64(i), c.cs(), inter, eps, scale if i == 0 else 1.0)
        tol = 2.0 ** -18 * mag
        tol = tol + 2.0 ** -8 * (np.abs(want) + tol) + 1e-30
        worst = (np.abs(f64(got) - want) / tol).max()
        assert worst <= 1.0, f"{'qk'[i]} off by {worst:.3g} of its bound"


@pytest.mark.parametrize("T", [1, 2, 15, 17, 130])
@pytest.mark.parametrize("d,rot", [(128, 128), (128, 32), (64, 64), (64, 16), (64, 0), (128, 112)])
@pytest.mark.parametrize("inter", [0, 1])
def test_forward(ra, T, d, rot, inter):
    c = Case(T, d=d, rot=rot, seed=T)
    q, k = c.rows(c.x)
    out = c.rows()
    ra.qk_norm_rope(q, k, *out, *c.args(), eps=1e-5, q_scale=0.3, interleaved=inter, **c.kw())
    assert ra.sync_status() == ra.RA_OK
    check_forward(c, out, inter, 1e-5, 0.3)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 1), (6, 2), (5, 5), (64, 8), (33, 3)])
@pytest.mark.parametrize("layouts", [("fused", "head"), ("head", "token"), ("token", "fused"), ("head", "head")])
@pytest.mark.parametrize("w", ["bf16", "fp32", "none"])
def test_forward_heads_layouts_and_weights(ra, hq, hkv, layouts, w):
    c = Case(37, hq, hkv, 64, 32, w=w, seed=hq)
    q, k = c.rows(c.x, layout=layouts[0])
    out = c.rows(layout=layouts[1])
    ra.qk_norm_rope(q, k, *out, *c.args(), eps=0.0, q_scale=-1.5, **c.kw())
    assert ra.sync_status() == ra.RA_OK
    check_forward(c, out, 0, 0.0, -1.5)
    if layouts[1] == "fused":
        assert torch.isnan(out[0]._base[:, hq + hkv:]).all(), "v's heads of the projection are left alone"


@pytest.mark.parametrize("T", [5000, 40000])
def test_forward_more_tokens_than_one_round_of_blocks(ra, T):
    c = Case(T, 8, 1, 64, 64, n_pos=T, seed=3)
    c.pos = torch.arange(T, dtype=torch.int32).flip(0)
    out = c.rows()
    ra.qk_norm_rope(*c.rows(c.x), *out, *c.args(), q_scale=0.125, **c.kw())
    assert ra.sync_status() == ra.RA_OK
    pick = np.r_[0:50, T // 2:T // 2 + 50, T - 50:T]
    sub = Case(len(pick), 8, 1, 64, 64, n_pos=T)
    sub.x, sub.w, sub.table, sub.pos = [x[pick] for x in c.x], c.w, c.table, c.pos[pick]
    check_forward(sub, [o[torch.from_numpy(pick).to(dev())] for o in out], 0, 1e-6, 0.125)
    # every token at once: what is turned keeps its length
    n = out[1].float().square().mean((1, 2))
    want = (c.x[1].float() / (c.x[1].float().square().mean(-1, keepdim=True) + 1e-6).sqrt() * c.w[1].float()).square().mean((1, 2)).to(dev())
    # (each element is off by 2^-8 of itself at most)
    assert ((n - want).abs() <= 2.0 ** -6 * want).all()


@pytest.mark.parametrize("inter", [0, 1])
def test_in_place(ra, inter):
    c = Case(77, 6, 2, 128, 64, layout="fused", seed=4)
    q, k = c.rows(c.x)
    ra.qk_norm_rope(q, k, q, k, *c.args(), interleaved=inter, q_scale=0.5, **c.kw())
    assert ra.sync_status() == ra.RA_OK
    check_forward(c, (q, k), inter, 1e-6, 0.5)


def test_zero_rows_and_large_and_small_ones(ra):
    c = Case(6, 2, 1, 64, 32, seed=5)
    for x in c.x:
        x[0] = 0.0
        x[1] *= 2.0 ** 40
        x[2] *= 2.0 ** -40
        x[3] = 2.0 ** -130  # subnormal in bf16
    out = c.rows()
    ra.qk_norm_rope(*c.rows(c.x), *out, *c.args(), **c.kw())
    assert ra.sync_status() == ra.RA_OK
    check_forward(c, out, 0, 1e-6, 1.0)
    assert not out[0][0].any() and not out[1][0].any()


def test_a_row_with_an_infinity_or_a_nan_spoils_no_other(ra):
    c = Case(33, 4, 2, 64, 64, seed=6)
    c.x[0][5, 2, 7], c.x[1][9, 1, 0] = float("inf"), float("nan")
    out = c.rows()
    ra.qk_norm_rope(*c.rows(c.x), *out, *c.args(), **c.kw())
    assert ra.sync_status() == ra.RA_OK
    bad = [torch.isnan(o).any(-1).cpu() for o in out]
    assert bad[0].nonzero().tolist() == [[5, 2]] and bad[1].nonzero().tolist() == [[9, 1]]
    c.x[0][5, 2], c.x[1][9, 1] = 0.0, 0.0
    out[0][5, 2], out[1][9, 1] = 0.0, 0.0
    check_forward(c, out, 0, 1e-6, 1.0)


@pytest.mark.parametrize("backward", [False, True])
def test_tokens_without_a_position_are_left_alone(ra, backward):
    c = Case(50, 3, 2, 64, 32, n_pos=40, seed=7)
    off = torch.zeros(50, dtype=torch.bool)
    off[[0, 7, 31, 49]] = True
    c.pos[off] = torch.tensor([-1, 40, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32)
    q, k = c.rows(c.x)
    out = c.rows()
    if backward:
        dw = [torch.full((64,), float("nan"), device=dev()) for _ in range(2)]
        ws = torch.empty(ra.qk_norm_rope_workspace_bytes(50, 3, 2, 64), dtype=torch.uint8, device=dev())
        ra.qk_norm_rope_bwd(q, k, *c.rows(c.dz, F32), *out, *c.args(), ws, dq_weight=dw[0], dk_weight=dw[1], **c.kw())
    else:
        ra.qk_norm_rope(q, k, *out, *c.args(), **c.kw())
    assert ra.sync_status() == ra.RA_OK
    for o in out:
        assert torch.isnan(o[off.to(dev())]).all() and not torch.isnan(o[~off.to(dev())]).any()
    on = ~off
    c.x, c.dz, c.pos, c.T = [x[on] for x in c.x], [x[on] for x in c.dz], c.pos[on], int(on.sum())
    out = [o[on.to(dev())] for o in out]
    if backward:
        check_backward(c, c.dz, out, dw, 0, 1e-6, 1.0, BF)
    else:
        check_forward(c, out, 0, 1e-6, 1.0)


def check_backward(c, dz, grads, dw, inter, eps, scale, dtype):
    """As check_forward: dx's terms carry two sums of d products and a dozen roundings, 2^-17 of their absolute sum.  dw
    adds up T H terms of 2^-19 in fp32, every one through fewer than T H / 16 + 300 additions (a thread's own, 32 threads', the
    blocks'), in a tree whose last 64 or fewer steps see the whole: (T H / 16 + 300) 2^-24 of the absolute sum."""
    for i in range(2):
        x = c.x[i].double().numpy()
        dx, dwx, dx_abs, dw_abs = onorm.backward(x, c.w64(i), c.cs(), dz[i].double().numpy(), inter, eps, scale if i == 0 else 1.0)
        tol = 2.0 ** -17 * dx_abs + 1e-30
        if dtype is BF:
            tol = tol + 2.0 ** -8 * (np.abs(dx) + tol)
        worst = (np.abs(f64(grads[i]) - dx) / tol).max()
        assert worst <= 1.0, f"d{'qk'[i]} off by {worst:.3g} of its bound"
        if dw[i] is not None:
            n = x.shape[0] * x.shape[1]
            worst = (np.abs(f64(dw[i]) - dwx) / ((2.0 ** -19 + (n / 16 + 300) * 2.0 ** -24) * dw_abs + 1e-30)).max()
            assert worst <= 1.0, f"d{'qk'[i]}_weight off by {worst:.3g} of its bound"


@pytest.mark.parametrize("T", [1, 16, 33, 300])
@pytest.mark.parametrize("d,rot", [(128, 128), (64, 32), (128, 16), (64, 0)])
@pytest.mark.parametrize("inter", [0, 1])
@pytest.mark.parametrize("types", [(F32, BF), (BF, BF), (F32, F32), (BF, F32)])
def test_backward(ra, T, d, rot, inter, types):
    c = Case(T, 6, 2, d, rot, w="fp32" if T % 2 else "bf16", seed=T)
    dz = [x.to(types[0]) for x in c.dz]
    grads = c.rows(dtype=types[1])
    dw = [torch.full((d,), float("nan"), device=dev()) for _ in range(2)]
    ws = torch.full((ra.qk_norm_rope_workspace_bytes(T, 6, 2, d),), 0xff, dtype=torch.uint8, device=dev())
    ra.qk_norm_rope_bwd(*c.rows(c.x), *c.rows(dz, types[0]), *grads, *c.args(), ws, dq_weight=dw[0], dk_weight=dw[1], eps=1e-3, q_scale=0.4,
                        interleaved=inter, **c.kw())
    assert ra.sync_status() == ra.RA_OK
    check_backward(c, dz, grads, dw, inter, 1e-3, 0.4, types[1])


@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 2), (64, 8), (5, 5)])
@pytest.mark.parametrize("layouts", [("fused", "head", "fused"), ("head", "token", "head")])
@pytest.mark.parametrize("w", ["none", "bf16"])
def test_backward_heads_and_layouts(ra, hq, hkv, layouts, w):
    c = Case(70, hq, hkv, 128, 64, w=w, seed=8)
    grads = c.rows(layout=layouts[2])
    # (a gradient of weights that are ones, and one that nobody asks for)
    dw = [torch.full((128,), float("nan"), device=dev()), None]
    ws = torch.empty(ra.qk_norm_rope_workspace_bytes(70, hq, hkv, 128), dtype=torch.uint8, device=dev())
    ra.qk_norm_rope_bwd(*c.rows(c.x, layout=layouts[0]), *c.rows(c.dz, F32, layouts[1]), *grads, *c.args(), ws, dq_weight=dw[0], q_scale=2.0, **c.kw())
    assert ra.sync_status() == ra.RA_OK
    check_backward(c, c.dz, grads, dw, 0, 1e-6, 2.0, BF)


def test_backward_without_weights_gradients_and_in_place(ra):
    c = Case(45, 4, 2, 64, 64, seed=9)
    g = c.rows(c.dz, F32)
    ra.qk_norm_rope_bwd(*c.rows(c.x), *g, *g, *c.args(), **c.kw())
    assert ra.sync_status() == ra.RA_OK
    check_backward(c, c.dz, g, [None, None], 0, 1e-6, 1.0, F32)


def test_backward_of_no_tokens_gives_weights_gradients_of_zero(ra):
    c = Case(0, 4, 2, 64, 64)
    dw = [torch.full((64,), float("nan"), device=dev()) for _ in range(2)]
    ws = torch.empty(ra.qk_norm_rope_workspace_bytes(0, 4, 2, 64), dtype=torch.uint8, device=dev())
    r = c.rows(c.x)
    ra.qk_norm_rope(*r, *r, *c.args(), **c.kw())
    ra.qk_norm_rope_bwd(*r, *r, *r, *c.args(), ws, dq_weight=dw[0], dk_weight=dw[1], **c.kw())
    assert ra.sync_status() == ra.RA_OK
    assert not dw[0].any() and not dw[1].any()


@pytest.mark.parametrize("inter", [0, 1])
def test_backward_against_differences_of_the_forward_oracle(ra, inter):
    """dx . e against (f(x + h e) - f(x - h e)) / 2h in float64, along random directions."""
    c = Case(9, 2, 1, 64, 32, w="fp32", seed=10)
    grads = c.rows(dtype=F32)
    ra.qk_norm_rope_bwd(*c.rows(c.x), *c.rows(c.dz, F32), *grads, *c.args(), q_scale=0.7, interleaved=inter, **c.kw())
    assert ra.sync_status() == ra.RA_OK
    r = np.random.default_rng(0)
    for i in range(2):
        x, dz = c.x[i].double().numpy(), c.dz[i].double().numpy()
        for _ in range(5):
            e = r.normal(size=x.shape)

            def f(h):
                return (onorm.forward(x + h * e, c.w64(i), c.cs(), inter, 1e-6, 0.7 if i == 0 else 1.0)[0] * dz).sum()

            want, got = (f(1e-5) - f(-1e-5)) / 2e-5, (f64(grads[i]) * e).sum()
            _, _, dx_abs, _ = onorm.backward(x, c.w64(i), c.cs(), dz, inter, 1e-6, 0.7 if i == 0 else 1.0)
            assert abs(want - got) <= 2.0 ** -17 * (dx_abs * np.abs(e)).sum() + 1e-6


def test_weights_gradients_are_the_same_bits_every_time_and_those_of_many_tokens(ra):
    T = 30000
    c = Case(T, 8, 2, 128, 128, seed=11)
    ws = torch.empty(ra.qk_norm_rope_workspace_bytes(T, 8, 2, 128), dtype=torch.uint8, device=dev())
    res = []
    ins, dz = c.rows(c.x), c.rows(c.dz, F32)
    for _ in range(3):
        dw = [torch.empty(128, device=dev()) for _ in range(2)]
        ra.qk_norm_rope_bwd(*ins, *dz, *c.rows(), *c.args(), ws, dq_weight=dw[0], dk_weight=dw[1], **c.kw())
        res.append(dw)
    assert ra.sync_status() == ra.RA_OK
    for a in res[1:]:
        assert torch.equal(a[0], res[0][0]) and torch.equal(a[1], res[0][1])
    cs = c.table.to(dev()).double()[c.pos.to(dev()).long()][:, None]
    for i in range(2):
        x, g = ins[i].double(), dz[i].double()
        a, b = g.chunk(2, -1)
        co, si = cs.chunk(2, -1)
        g = torch.cat([a * co + b * si, b * co - a * si], -1)
        terms = g * x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt()
        err = (res[0][i].double() - terms.sum((0, 1))).abs() / terms.abs().sum((0, 1))
        # a thread adds up at most T H / (blocks * 16) < 500 terms of 2^-19, then 16, then at most 1216 blocks' by 32 threads
        assert err.max() <= 2.0 ** -19 + (500 + 16 + 38 + 32) * 2.0 ** -24


def test_captured_and_on_another_stream(ra):
    c = Case(64, 8, 2, 128, 128, layout="fused", seed=12)
    q, k = c.rows(c.x)
    out, grads = c.rows(layout="head"), c.rows(layout="token")
    dw = [torch.empty(128, device=dev()) for _ in range(2)]
    ws = torch.empty(ra.qk_norm_rope_workspace_bytes(64, 8, 2, 128), dtype=torch.uint8, device=dev())
    pos, table = c.args()
    kw, dz = c.kw(), c.rows(c.dz, F32, "head")

    def both(**s):
        ra.qk_norm_rope(q, k, *out, pos, table, **kw, **s)
        ra.qk_norm_rope_bwd(q, k, *dz, *grads, pos, table, ws, dq_weight=dw[0], dk_weight=dw[1], **kw, **s)

    both()
    torch.cuda.synchronize()
    want = [x.clone() for x in (*out, *grads, *dw)]
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        both()
    for how in ("replay", "stream"):
        for x in (*out, *grads, *dw):
            x.fill_(float("nan"))
        torch.cuda.synchronize()
        if how == "replay":
            graph.replay()
        else:
            both(stream=s)
        torch.cuda.synchronize()
        for a, b in zip((*out, *grads, *dw), want):
            assert torch.equal(a, b), how
    # new inputs in the same places
    pos.copy_(pos.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    c.pos = c.pos.flip(0)
    check_forward(c, out, 0, 1e-6, 1.0)
    check_backward(c, c.dz, grads, dw, 0, 1e-6, 1.0, BF)


def test_rows_far_apart(ra):
    """Strides whose offsets pass 2^31 elements."""
    step = 2 ** 26
    big = torch.empty(33 * step + 4096, dtype=BF, device=dev())
    c = Case(34, 1, 1, 64, 64, seed=13)
    q = big.as_strided((34, 1, 64), (step, 64, 1))
    k = big.as_strided((34, 1, 64), (step, 64, 1), 1024)
    q.copy_(c.x[0])
    k.copy_(c.x[1])
    ra.qk_norm_rope(q, k, q, k, *c.args(), **c.kw())
    assert ra.sync_status() == ra.RA_OK
    check_forward(c, (q, k), 0, 1e-6, 1.0)
