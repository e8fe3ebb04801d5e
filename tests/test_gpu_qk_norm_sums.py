"""The weights' gradients of the norm over many tokens, against the additions that the kernels' own tree of sums makes."""
import pytest
import torch

from tests.gpu_util import dev
from tests.test_gpu_qk_norm import F32, Case, ra  # noqa: F401

pytestmark = pytest.mark.gpu


def additions(T, heads, all_heads, d):
    """Of a sum over T tokens of `heads` heads, one after the other: a thread's own terms (a group of four heads at most, the
    tokens that a block comes back for), the block's tokens, a thread's share of the blocks, 32 such shares."""
    groups = [-(-h // 4) for h in all_heads]
    tokens = 256 // (d // 8)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    along = min(-(-T // tokens), max(1, sms * 4 // sum(groups)))
    return min(heads, 4) * -(-(-(-T // tokens)) // along) + tokens + -(-(-(-heads // 4) * along) // 32) + 32


@pytest.mark.parametrize("T,hq,hkv,d", [(30000, 8, 2, 128), (100, 3, 1, 64), (70001, 4, 4, 64)])
@pytest.mark.parametrize("eps", [1e-6, 0.0])
def test_sums_carry_no_more_than_their_own_additions(ra, T, hq, hkv, d, eps):
    c = Case(T, hq, hkv, d, d, seed=11)
    ws = torch.empty(ra.qk_norm_rope_workspace_bytes(T, hq, hkv, d), dtype=torch.uint8, device=dev())
    ins, dz = c.rows(c.x), c.rows(c.dz, F32)
    dw = [torch.empty(d, device=dev()) for _ in range(2)]
    ra.qk_norm_rope_bwd(*ins, *dz, *c.rows(), *c.args(), ws, dq_weight=dw[0], dk_weight=dw[1], eps=eps, **c.kw())
    assert ra.sync_status() == ra.RA_OK
    cs = c.table.to(dev()).double()[c.pos.to(dev()).long()][:, None]
    for i, heads in enumerate((hq, hkv)):
        x, g = ins[i].double(), dz[i].double()
        a, b = g.chunk(2, -1)
        co, si = cs.chunk(2, -1)
        g = torch.cat([a * co + b * si, b * co - a * si], -1)
        terms = g * x / (x.square().mean(-1, keepdim=True) + eps).sqrt()
        # a term's own error: its rotation's two products and sum, the sum of squares, r, two products: 2^-19 of |a cos| + |b sin|
        size = torch.cat([(a * co).abs() + (b * si).abs(), (b * co).abs() + (a * si).abs()], -1) * (terms / g).abs().nan_to_num()
        bound = 2.0 ** -19 * size.sum((0, 1)) + additions(T, heads, (hq, hkv), d) * 2.0 ** -24 * terms.abs().sum((0, 1))
        assert ((dw[i].double() - terms.sum((0, 1))).abs() <= bound).all()
