"""Numbers that the C ABI cannot hold, on the host (no GPU): the binding refuses them by name and passes no other in their place."""
import pytest
import torch

from tests.test_more_operators_host import ra  # noqa: F401


@pytest.fixture
def host(monkeypatch):
    """Host tensors report device -1; with the current device taken as that, they are taken for its own."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)


@pytest.mark.parametrize("max_keep", [2 ** 31, 2 ** 32, 2 ** 32 + 7, 2 ** 40 + 1])
def test_a_list_of_kept_positions_longer_than_a_c_int(ra, host, max_keep):
    """(of no sequences, so that it takes no memory)"""
    cache = [torch.zeros((6, 2, 16, 64), dtype=torch.bfloat16) for _ in range(2)]
    none = torch.zeros(0, dtype=torch.int32)
    kept = torch.empty((0, 2, max_keep), dtype=torch.int32)
    with pytest.raises(ValueError, match="max_keep must be a 32-bit number"):
        ra.cache_evict(*cache, torch.zeros((6, 2, 16)), torch.zeros((0, 2), dtype=torch.int32), none, none, none, kept, stream=0)


@pytest.mark.parametrize("kw,error", [(dict(interleaved=2 ** 31), ValueError), (dict(interleaved=-2 ** 40), ValueError),
                                      (dict(eps=1e39), RuntimeError), (dict(q_scale=-1e300), RuntimeError)])
def test_norm_numbers(ra, host, kw, error):
    """(numbers that are none in fp32 reach the library as infinities, which it refuses)"""
    q, k = torch.zeros((5, 4, 64), dtype=torch.bfloat16), torch.zeros((5, 2, 64), dtype=torch.bfloat16)
    pos, table = torch.zeros(5, dtype=torch.int32), torch.zeros((9, 32))
    with pytest.raises(error, match="interleaved must be a 32-bit number|invalid argument"):
        ra.qk_norm_rope(q, k, q, k, pos, table, stream=0, **kw)
    with pytest.raises(error, match="interleaved must be a 32-bit number|invalid argument"):
        ra.qk_norm_rope_bwd(q, k, q, k, q, k, pos, table, stream=0, **kw)
