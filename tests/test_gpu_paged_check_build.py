"""The paged cache through the check build: on valid batches, and on those whose device arrays hold what the header
allows them to (pages that are none, rows before position 0, padding), no index check may fail and the results are
bitwise those of the normal library."""
import os
import re

import pytest
import torch

from tests.gpu_util import dev
from tests.paged_util import Batch
from tests.test_gpu_check_build import PKG, _binding


@pytest.fixture(scope="module")
def libs():
    torch.cuda.set_device(0)
    return _binding("libringattn.so", "ringattn_release"), _binding("libringattn_check.so", "ringattn_checked")


def _bits(t):
    return t.contiguous().view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()]).cpu()


def _same(libs, run):
    res = []
    for ra in libs:
        out = run(ra)
        torch.cuda.synchronize()
        assert ra.sync_status() == ra.RA_OK, f"{ra.__name__}: site {ra.last_timeout()}" if hasattr(ra, "last_timeout") else ra.__name__
        res.append([_bits(t) for t in out])
    for a, b in zip(*res):
        assert torch.equal(a, b)


def test_every_site_is_used():
    """Host: the sites that the paged kernels declare are all checked somewhere, in each of their files."""
    read = lambda n: open(os.path.join(PKG, "csrc", n)).read()  # noqa: E731
    head = read("paged.h")
    sites = re.findall(r"(kSitePaged\w+) = \d+", head)
    assert len(sites) >= 6
    files = {n: read(n) for n in ("paged_cache.cu", "paged_decode.cu", "paged_chunk.cu")}
    for n, text in files.items():
        assert "RA_CHECKED(" in text, n
    for s in sites:
        assert any(re.search(r"RA_CHECKED\((?:[^;{]|\n)*?" + s, t) for t in (head, *files.values())), s


@pytest.mark.gpu
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("hq,hkv,d,page,seqs,kw", [
    (8, 2, 128, 16, [(1, 1), (1, 700), (0, 5), (1, 0), (1, 129)], {}),              # few rows, one group of 8
    (8, 1, 64, 48, [(2, 2), (2, 1000), (1, 1), (2, 0)], {}),                         # two groups
    (14, 2, 128, 32, [(9, 9), (3, 400), (9, 5)], {}),                                # one unit
    (6, 2, 64, 128, [(150, 150), (7, 900), (90, 40)], {}),                           # two units
    (8, 2, 128, 16, [(1, 1400), (1, 3)], dict(window=100, sinks=20)),
    (8, 2, 128, 48, [(70, 1400), (30, 30)], dict(window=300, sinks=17)),
    (8, 1, 128, 64, [(1, 30000)] + [(1, 40)] * 30, {}),                              # cut and joined
    (8, 1, 128, 64, [(40, 20000), (3, 100)], {}),
    (8, 1, 128, 64, [(200, 9000)], dict(causal=0)),
])
def test_attention(libs, e4m3, hq, hkv, d, page, seqs, kw):
    B = Batch(seqs, hkv=hkv, d=d, page=page, e4m3=e4m3, device=dev(), seed=5, pad=3, gap=16)
    for b, (n, L) in enumerate(seqs):
        if L > 2 * page:  # a page that is none, and values that are no numbers
            B.dtable[b, 1] = -1
            p = int(B.table[b, (L - 1) // page])
            if e4m3:
                B.v_scale[p, 0, (L - 1) % page] = float("nan")
            else:
                B.v_cache[p, 0, (L - 1) % page, 3] = float("inf")
    q = (torch.randn((B.total, hq, d), generator=torch.Generator().manual_seed(6)) * d ** -0.5).to(torch.bfloat16).to(dev())

    def run(ra):
        res = []
        for dt in (torch.bfloat16, torch.float32):
            out = torch.full((B.total, hq, d), float("nan"), dtype=dt, device=dev())
            lse = torch.full((B.total, hq), float("nan"), device=dev())
            ws = torch.empty(ra.paged_workspace_bytes(B.total, len(seqs), hq, hkv, d, B.max_q), dtype=torch.uint8, device=dev())
            ra.fwd_paged(q, B.k_cache, B.v_cache, out, lse, *B.args(), ws, max_q=B.max_q, **B.kw(), **kw)
            res += [out, lse]
        return res

    _same(libs, run)


@pytest.mark.gpu
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("hkv,d,page,seqs", [
    (8, 128, 16, [(1, 777), (1, 1), (0, 3), (5, 2)]),
    (3, 64, 48, [(130, 131), (17, 700)]),
    (8, 128, 64, [(20011, 20100), (3, 2), (700, 9000)]),  # the kernels of large calls
])
def test_append_and_read(libs, e4m3, hkv, d, page, seqs):
    g = torch.Generator().manual_seed(7)
    kn, vn = (torch.randn((sum(n for n, _ in seqs) + 3, hkv, d), generator=g).to(torch.bfloat16).to(dev()) for _ in range(2))

    def run(ra):
        B = Batch(seqs, hkv=hkv, d=d, page=page, e4m3=e4m3, device=dev(), seed=8, pad=3, fill=False, gap=8)
        if seqs[0][1] > 2 * page:
            B.dtable[0, 1] = B.n_pages
        ra.cache_append(kn, vn, B.k_cache, B.v_cache, *B.args(), **B.kw())
        ko, vo = (torch.full((hkv, B.total, d), float("nan"), dtype=torch.bfloat16, device=dev()) for _ in range(2))
        ra.cache_read(B.k_cache, B.v_cache, ko, vo, *B.args(), **B.kw())
        return [B.k_cache, B.v_cache, ko, vo] + ([B.k_scale, B.v_scale] if e4m3 else [])

    _same(libs, run)
