"""Norm and rotation, weights and eviction through the check build: no index check may fail, also where device arrays hold what
the header allows them to (pages that are none, lengths and positions of any value), and the results are bitwise those
of the normal library."""
import os
import re

import pytest
import torch

from tests.gpu_util import dev
from tests.paged_util import Batch
from tests.test_gpu_check_build import PKG, _binding
from tests.test_gpu_paged_check_build import _same


@pytest.fixture(scope="module")
def libs():
    torch.cuda.set_device(0)
    return _binding("libringattn.so", "ringattn_release_more"), _binding("libringattn_check.so", "ringattn_checked_more")


def test_every_site_is_used():
    """Host: the sites that these kernels declare are all checked somewhere, in each of their files."""
    read = lambda n: open(os.path.join(PKG, "csrc", n)).read()  # noqa: E731
    files = {n: read(n) for n in ("qk_norm.cu", "cache_weights.cu", "cache_weights_chunk.cu", "cache_evict.cu")}
    for n, text in files.items():
        assert "RA_CHECKED(" in text, n
    sites = re.findall(r"(kSite(?:Norm|Weights|Evict)\w+) = \d+", read("qk_norm.h") + read("cache_weights.h"))
    assert len(sites) >= 7
    for s in sites:
        assert any(re.search(r"RA_CHECKED\((?:[^;{]|\n)*?" + s, t) for t in files.values()), s


def _pool(B, hkv, page, seed):
    w = torch.rand((B.n_pages, hkv, page), generator=torch.Generator().manual_seed(seed)).to(dev())
    w[0, 0, 0] = float("nan")
    return w


@pytest.mark.gpu
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("hq,hkv,d,page,seqs,kw", [
    (8, 2, 128, 16, [(1, 1), (1, 700), (0, 5), (1, 0), (1, 129)], {}),               # few rows
    (8, 1, 64, 48, [(2, 2), (3, 1000), (1, 1), (2, 0)], {}),                          # more of them
    (14, 2, 128, 32, [(19, 9), (30, 400), (12, 5)], {}),                              # chunks
    (6, 2, 64, 128, [(150, 150), (70, 900), (90, 40)], {}),
    (8, 2, 128, 16, [(1, 1400), (1, 3)], dict(window=100, sinks=20)),
    (8, 2, 128, 48, [(70, 1400), (30, 30)], dict(window=300, sinks=17)),
    (8, 1, 128, 64, [(40, 20000), (3, 100)], {}),                                     # cut and joined
    (8, 1, 128, 64, [(200, 9000)], dict(causal=0)),
])
def test_weights(libs, e4m3, hq, hkv, d, page, seqs, kw):
    B = Batch(seqs, hkv=hkv, d=d, page=page, e4m3=e4m3, device=dev(), seed=5, pad=3, gap=16)
    for b, (n, L) in enumerate(seqs):
        if L > 2 * page:  # a page that is none, and a value that is no number
            B.dtable[b, 1] = -1
            p = int(B.table[b, (L - 1) // page])
            if e4m3:
                B.k_scale[p, 0, (L - 1) % page] = float("nan")
            else:
                B.k_cache[p, 0, (L - 1) % page, 3] = float("inf")
    g = torch.Generator().manual_seed(6)
    q = (torch.randn((B.total, hq, d), generator=g) * d ** -0.5).to(torch.bfloat16).to(dev())
    lse = (torch.randn((B.total, hq), generator=g) + 5).to(dev())

    def run(ra):
        w = _pool(B, hkv, page, 7)
        ws = torch.empty(ra.paged_workspace_bytes(B.total, len(seqs), hq, hkv, d, B.max_q), dtype=torch.uint8, device=dev())
        for decay in (0.5, 0.0):
            ra.cache_weights(q, lse, B.k_cache, B.v_cache, w, *B.args(), ws, max_q=B.max_q, decay=decay, **B.kw(), **kw)
        return [w]

    _same(libs, run)


@pytest.mark.gpu
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("hkv,d,page,lens,keep", [
    (8, 128, 16, [700, 1, 0, 33], [100, 5, 5, 33]),
    (3, 64, 48, [131, 1700, 20], [64, 900, 0]),
    (2, 128, 64, [40000, 9000], [20000, 10]),
    (40, 64, 16, [900] * 8, [300] * 8),  # a block a head
    (160, 64, 16, [9000], [500]),
])
def test_evict(libs, e4m3, hkv, d, page, lens, keep):
    def run(ra):
        B = Batch([(0, n) for n in lens], hkv=hkv, d=d, page=page, e4m3=e4m3, device=dev(), seed=8, gap=16)
        if lens[0] > 2 * page:
            B.dtable[0, 1] = B.n_pages
        w = _pool(B, hkv, page, 9)
        n = torch.empty(len(lens), dtype=torch.int32, device=dev())
        kept = torch.empty((len(lens), hkv, max(keep)), dtype=torch.int32, device=dev())
        ra.cache_evict(B.k_cache, B.v_cache, w, B.dtable, B.dlen, torch.tensor(keep, dtype=torch.int32, device=dev()), n, kept, sinks=2,
                       recent=7, **B.kw())
        caches = [x.view(torch.uint8) if e4m3 else x for x in (B.k_cache, B.v_cache)]
        return [*caches, w, n, kept] + ([B.k_scale, B.v_scale] if e4m3 else [])

    _same(libs, run)


@pytest.mark.gpu
@pytest.mark.parametrize("T,hq,hkv,d,rot,inter", [(1, 8, 2, 128, 128, 0), (333, 5, 1, 64, 32, 1), (2000, 64, 8, 128, 64, 0), (70, 3, 3, 64, 0, 0)])
def test_norm(libs, T, hq, hkv, d, rot, inter):
    g = torch.Generator().manual_seed(10)
    q, k, dq, dk = (torch.randn((T, h, d), generator=g).to(torch.bfloat16).to(dev()) for h in (hq, hkv, hq, hkv))
    wq, wk = (torch.rand(d, generator=g).to(dev()) for _ in range(2))
    cos_sin = torch.randn((50, rot), generator=g).to(dev())
    position = torch.randint(-3, 53, (T,), generator=g, dtype=torch.int32).to(dev())
    kw = dict(q_weight=wq, k_weight=wk, q_scale=0.3, interleaved=inter)

    def run(ra):
        outs = [torch.zeros_like(x) for x in (q, k)]
        ra.qk_norm_rope(q, k, *outs, position, cos_sin, **kw)
        grads = [torch.zeros_like(x) for x in (q, k)]
        dw = torch.empty((2, d), device=dev())
        ws = torch.empty(ra.qk_norm_rope_workspace_bytes(T, hq, hkv, d), dtype=torch.uint8, device=dev())
        ra.qk_norm_rope_bwd(q, k, dq, dk, *grads, position, cos_sin, ws, dq_weight=dw[0], dk_weight=dw[1], **kw)
        return [*outs, *grads, dw]

    _same(libs, run)
