"""ringattn_cache_evict against the oracle: everything bit for bit."""
import numpy as np
import pytest
import torch

from oracle import evict as oevict
from tests.gpu_util import dev
from tests.paged_util import Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ra():
    from online_softmax_attention_zigzag_gb300 import ringattn
    ringattn.lib()
    torch.cuda.set_device(0)
    return ringattn


class Run:
    def __init__(self, lens, keep, *, hkv=2, d=64, page=16, e4m3=False, seed=0, gap=0, weights=None, max_keep=None, spare=2):
        self.B = Batch([(0, L) for L in lens], hkv=hkv, d=d, page=page, e4m3=e4m3, device=dev(), seed=seed, gap=gap, spare=spare)
        g = torch.Generator().manual_seed(seed + 1)
        self.lens, self.hkv, self.page = lens, hkv, page
        self.keep = torch.tensor(keep, dtype=torch.int32)
        w = torch.full((self.B.n_pages, hkv * page + 4 * (gap > 0)), float("nan"), device=dev())
        self.w = w.as_strided((self.B.n_pages, hkv, page), (w.shape[1], page, 1))
        self.weights = []
        for b, L in enumerate(lens):
            x = torch.rand((L, hkv), generator=g) if weights is None else weights(b, L)
            pg, row = self.B.places(b)
            if L:
                self.w[pg, :, row] = x.to(dev())
            self.weights.append(x)
        self.max_keep = max_keep or max(1, max(keep))
        self.kept = torch.full((len(lens), hkv, self.max_keep), -7, dtype=torch.int32, device=dev())
        self.out = torch.full((len(lens),), -7, dtype=torch.int32, device=dev())

    def pools(self):
        B = self.B
        r = [B.k_cache.view(torch.uint8) if B.e4m3 else B.k_cache, B.v_cache.view(torch.uint8) if B.e4m3 else B.v_cache, self.w]
        return r + ([B.k_scale, B.v_scale] if B.e4m3 else [])

    def call(self, ra, sinks=0, recent=0, out=None, stream=None):
        self.dkeep = self.keep.to(dev())
        ra.cache_evict(self.B.k_cache, self.B.v_cache, self.w, self.B.dtable, self.B.dlen, self.dkeep, self.out if out is None else out, self.kept,
                       sinks=sinks, recent=recent, stream=stream, **self.B.kw())

    def expect(self, sinks=0, recent=0):
        """(pools, kept, lengths) that the call has to leave."""
        pools = [x.clone() for x in self.pools()]
        kept = torch.full_like(self.kept, -1)
        for b, L in enumerate(self.lens):
            keep = max(0, min(int(self.keep[b]), self.max_keep))
            pg, row = self.B.places(b)
            for h in range(self.hkv):
                j = oevict.stay(self.weights[b][:, h].tolist(), keep, sinks, recent)
                kept[b, h, :len(j)] = torch.tensor(j, dtype=torch.int32)
                jt = torch.tensor(j, dtype=torch.long, device=dev())
                for new, old in zip(pools, self.pools()):
                    new[pg[:len(j)], h, row[:len(j)]] = old[pg[jt], h, row[jt]]
        return pools, kept, torch.tensor([min(L, max(0, min(int(k), self.max_keep))) for L, k in zip(self.lens, self.keep)], dtype=torch.int32, device=dev())

    def check(self, ra, sinks=0, recent=0, **kw):
        pools, kept, n = self.expect(sinks, recent)
        self.call(ra, sinks, recent, **kw)
        assert ra.sync_status() == ra.RA_OK
        assert torch.equal(self.kept, kept)
        assert torch.equal(kw.get("out", self.out), n)
        for x, y in zip(self.pools(), pools):
            bits = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[x.element_size()]
            assert torch.equal(x.contiguous().view(bits), y.contiguous().view(bits))


LENS = [0, 1, 15, 16, 17, 100, 333, 1000]


@pytest.mark.parametrize("d,e4m3", [(64, False), (128, False), (64, True), (128, True)])
@pytest.mark.parametrize("page", [16, 48, 256])
@pytest.mark.parametrize("sinks,recent", [(0, 0), (3, 10)])
def test_lengths(ra, d, e4m3, page, sinks, recent):
    Run(LENS, [5, 1, 7, 16, 16, 50, 100, 17], d=d, e4m3=e4m3, page=page, seed=d).check(ra, sinks, recent)


@pytest.mark.parametrize("keep", [0, 1, 2, 31, 32, 33, 499, 500, 501, 2 ** 31 - 1, -1, -2 ** 31])
def test_how_many_stay(ra, keep):
    Run([500, 40], [keep, 20], seed=1, hkv=3, max_keep=600).check(ra, 1, 4)


def test_at_most_max_keep(ra):
    Run([500, 40], [400, 20], seed=2, max_keep=33).check(ra)


@pytest.mark.parametrize("sinks,recent", [(0, 1), (1, 0), (50, 0), (0, 50), (25, 25), (30, 40), (2 ** 31 - 1, 0), (0, 2 ** 31 - 1), (7, 2 ** 31 - 1)])
def test_sinks_and_recent_ones(ra, sinks, recent):
    Run([300, 49, 50, 51], [50, 50, 50, 50], seed=3).check(ra, sinks, recent)


def test_weights_that_are_equal(ra):
    """Ties go to the lower position: few values, zeros of both signs, all the same."""
    g = torch.Generator().manual_seed(4)
    kinds = [lambda L: torch.randint(0, 3, (L, 2), generator=g).float(), lambda L: torch.zeros(L, 2),
             lambda L: torch.where(torch.rand((L, 2), generator=g) < 0.5, 0.0, -0.0), lambda L: torch.full((L, 2), 0.125)]
    for x in kinds:
        Run([700, 90], [101, 30], weights=lambda b, L: x(L), seed=5).check(ra)


def test_weights_of_every_kind(ra):
    """Negative ones, infinities, NaN of both signs, subnormals, neighbours in the last bit."""
    g = torch.Generator().manual_seed(6)

    def some(b, L):
        x = torch.randn((L, 2), generator=g) * torch.exp2(torch.randint(-140, 127, (L, 2), generator=g).float())
        x[::17], x[3::29], x[5::31] = float("inf"), -float("inf"), float("nan")
        x[7::41] = torch.tensor([0xffc00001 - 2 ** 32], dtype=torch.int32).view(torch.float32)
        x[11::13] = torch.nextafter(torch.ones(1), torch.full((1,), 2.0)) if b else 1.0
        x[12::13] = 1.0
        return x

    for keep in (1, 20, 60, 300, 640):
        Run([700, 660], [keep, keep], weights=some, seed=keep).check(ra)


def test_nothing_to_evict_changes_nothing(ra):
    r = Run([30, 17, 0], [30, 40, 1], seed=7)
    before = [x.clone() for x in r.pools()]
    r.check(ra, 2, 2)
    for x, y in zip(r.pools(), before):
        assert torch.equal(torch.nan_to_num(x.float()), torch.nan_to_num(y.float()))


@pytest.mark.parametrize("e4m3", [False, True])
def test_lengths_in_place_and_pages_apart(ra, e4m3):
    r = Run([400, 33, 210], [64, 40, 7], seed=8, gap=5, e4m3=e4m3)
    r.check(ra, 1, 3, out=r.B.dlen)


def test_again_and_again(ra):
    """Evicting from what was kept: the weights have moved along."""
    r = Run([900, 300], [400, 200], seed=9)
    r.check(ra, 2, 8, out=r.B.dlen)
    for keep in ([150, 150], [150, 90], [20, 1]):
        lens = r.B.dlen.tolist()
        for b, L in enumerate(lens):
            pg, row = r.B.places(b)
            r.weights[b] = r.w[pg[:L], :, row[:L]].cpu()
        r.lens = lens
        r.keep = torch.tensor(keep, dtype=torch.int32)
        r.check(ra, 2, 8, out=r.B.dlen)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("L,keep", [(5000, 1000), (40000, 3001), (150000, 20000), (70000, 69999)])
def test_long_ones(ra, e4m3, L, keep):
    """Against torch's stable sort."""
    hkv, d, page = 2, 64, 64
    g = torch.Generator(device=dev()).manual_seed(L)
    pages = -(-L // page)
    table = torch.randperm(pages, generator=g, device=dev()).to(torch.int32)[None]
    bits = [torch.randint(0, 256, (pages, hkv, page, d * (1 if e4m3 else 2)), generator=g, device=dev(), dtype=torch.uint8) for _ in range(2)]
    k, v = (x.view(torch.float8_e4m3fn if e4m3 else torch.bfloat16) for x in bits)
    sc = [torch.rand((pages, hkv, page), generator=g, device=dev()) if e4m3 else None for _ in range(2)]
    w = torch.rand((pages, hkv, page), generator=g, device=dev()) ** 8
    w.mul_(torch.rand(w.shape, generator=g, device=dev()) > 0.2)
    old = [x.clone() for x in bits + [w] + [s for s in sc if s is not None]]
    t = table[0].long()
    x = w[t].transpose(0, 1).reshape(hkv, -1)[:, :L].clone()
    x[:, :4], x[:, L - 64:] = float("inf"), float("inf")
    order = torch.sort(x, dim=1, descending=True, stable=True)[1][:, :keep].sort(1)[0]
    ln, kp = (torch.tensor([y], dtype=torch.int32, device=dev()) for y in (L, keep))
    kept = torch.empty((1, hkv, keep + 3), dtype=torch.int32, device=dev())
    ra.cache_evict(k, v, w, table, ln, kp, ln, kept, sinks=4, recent=64, k_scale=sc[0], v_scale=sc[1])
    assert ra.sync_status() == ra.RA_OK
    assert int(ln) == keep and torch.equal(kept[0, :, :keep].long(), order) and (kept[0, :, keep:] == -1).all()
    to = torch.arange(keep, device=dev())
    for got, was in zip(bits + [w] + [s for s in sc if s is not None], old):
        want = was.clone()
        for h in range(hkv):
            want[t[to // page], h, to % page] = was[t[order[h] // page], h, order[h] % page]
        assert torch.equal(got, want)


@pytest.mark.parametrize("L,keep,heads", [(17000, 900, 160), (40000, 20000, 1), (140000, 70001, 1), (30000, 1, 3), (5000, 4999, 200)])
@pytest.mark.parametrize("kind", ["ties", "zeros", "near"])
def test_long_ones_whose_weights_are_alike(ra, L, keep, heads, kind):
    """More equal ones than a block lists, stretches of several parts, thousands of keys whose first digits agree."""
    d, page = 64, 128
    g = torch.Generator(device=dev()).manual_seed(L + keep)
    pages = -(-L // page)
    table = torch.randperm(pages, generator=g, device=dev()).to(torch.int32)[None]
    k, v = (torch.zeros((pages, heads, page, d), device=dev(), dtype=torch.uint8).view(torch.float8_e4m3fn) for _ in range(2))
    sc = [torch.rand((pages, heads, page), generator=g, device=dev()) for _ in range(2)]
    w = torch.rand((pages, heads, page), generator=g, device=dev())
    if kind == "ties":
        w = (w * 4).floor()
    elif kind == "zeros":
        w = w * (w > 0.9)
    else:
        w = 1.0 + w * 1e-3
    t = table[0].long()
    x = w[t].transpose(0, 1).reshape(heads, -1)[:, :L]
    order = torch.sort(x, dim=1, descending=True, stable=True)[1][:, :keep].sort(1)[0]
    want = [s[t].transpose(0, 1).reshape(heads, -1)[:, :L].gather(1, order) for s in (w, *sc)]
    ln, kp = (torch.tensor([y], dtype=torch.int32, device=dev()) for y in (L, keep))
    kept = torch.empty((1, heads, keep), dtype=torch.int32, device=dev())
    ra.cache_evict(k, v, w, table, ln, kp, ln, kept, k_scale=sc[0], v_scale=sc[1])
    assert ra.sync_status() == ra.RA_OK
    assert int(ln) == keep and torch.equal(kept[0].long(), order)
    for s, y in zip((w, *sc), want):
        assert torch.equal(s[t].transpose(0, 1).reshape(heads, -1)[:, :keep], y)


def test_many_heads_and_sequences(ra):
    Run([(37 * b) % 90 for b in range(300)], [(11 * b) % 50 for b in range(300)], hkv=5, seed=10).check(ra, 1, 2)


def test_pages_that_the_table_does_not_name(ra):
    """They read as weight 0 and zeros, what would move there is dropped, nothing outside the pool is touched."""
    r = Run([200, 100], [60, 60], hkv=1, seed=11)
    bad = torch.tensor([-1, 2 ** 31 - 1, r.B.n_pages, -2 ** 31], dtype=torch.int32, device=dev())
    r.B.dtable[0, [1, 5, 6, 9]] = bad
    before = [x.clone() for x in r.pools()]
    w = r.weights[0][:, 0].clone()
    for e in (1, 5, 6, 9):
        w[16 * e:16 * e + 16] = 0.0
    j = oevict.stay(w.tolist(), 60)
    r.call(ra)
    assert ra.sync_status() == ra.RA_OK
    assert r.kept[0, 0].tolist() == j
    pg, row = r.B.places(0)
    for new, old in zip(r.pools(), before):
        want = old.clone()
        jt = torch.tensor(j, device=dev())
        src = old[pg[jt], 0, row[jt]].clone()
        src[torch.isin(jt // 16, torch.tensor([1, 5, 6, 9], device=dev()))] = 0
        for i in range(60):
            if i // 16 not in (1, 5, 6, 9) and j[i] != i:
                want[pg[i], 0, row[i]] = src[i]
        same = (new == want) | (torch.isnan(new.float()) & torch.isnan(want.float()))
        mine = torch.zeros_like(same)
        mine[pg, 0, row] = True
        assert (same | ~mine).all()


@pytest.mark.parametrize("lens", [[2 ** 31 - 1, -3, 100], [-2 ** 31, 2 ** 31 - 1, 7]])
def test_lengths_that_are_none(ra, lens):
    r = Run([100, 100, 100], [10, 20, 30], seed=12)
    r.B.dlen.copy_(torch.tensor(lens, dtype=torch.int32))
    r.B.dtable[r.B.dtable >= r.B.n_pages] = -1
    r.call(ra)
    assert ra.sync_status() == ra.RA_OK
    cap = r.B.table.shape[1] * 16
    assert r.out.tolist() == [min(max(0, min(L, cap)), k) for L, k in zip(lens, (10, 20, 30))]


def test_captured_and_on_another_stream(ra):
    r = Run([400, 900], [100, 77], seed=13)
    start = [x.clone() for x in r.pools()]
    pools, kept, n = r.expect(1, 5)
    s = torch.cuda.Stream()
    r.call(ra, 1, 5)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    keep = r.dkeep
    with torch.cuda.graph(graph, stream=s):
        ra.cache_evict(r.B.k_cache, r.B.v_cache, r.w, r.B.dtable, r.B.dlen, keep, r.out, r.kept, sinks=1, recent=5)
    for how in ("replay", "stream"):
        for x, y in zip(r.pools(), start):
            x.copy_(y)
        r.kept.fill_(-9)
        torch.cuda.synchronize()
        if how == "replay":
            graph.replay()
        else:
            r.call(ra, 1, 5, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(r.kept, kept) and torch.equal(r.out, n), how
        for x, y in zip(r.pools(), pools):
            assert torch.equal(torch.nan_to_num(x.float()), torch.nan_to_num(y.float())), how
    assert ra.sync_status() == ra.RA_OK


@pytest.mark.parametrize("hkv,lens,keep", [(160, [8192, 1], [700, 1]), (153, [8193], [4000]), (152, [16400], [300]), (80, [20000, 5000], [64, 2500])])
@pytest.mark.parametrize("kind", ["all kinds", "few values"])
def test_more_heads_than_the_gpu_has_sms(ra, hkv, lens, keep, kind):
    g = torch.Generator().manual_seed(31)
    r = Run(lens, keep, hkv=hkv, d=64, page=16, seed=31,
            weights=lambda b, L: torch.rand((L, hkv), generator=g) if kind == "all kinds" else torch.randint(0, 3, (L, hkv), generator=g).float())
    r.check(ra, sinks=3, recent=20)
