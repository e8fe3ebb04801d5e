"""ringattn_cache_weights against the float64 oracle."""
import numpy as np
import pytest
import torch

from oracle import evict as oevict
from oracle import paged as opaged
from tests.gpu_util import dev, f64
from tests.paged_util import Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ra():
    from online_softmax_attention_zigzag_gb300 import ringattn
    ringattn.lib()
    torch.cuda.set_device(0)
    return ringattn


class Run:
    """A batch, queries, their lse and the weights' pool; call() runs the library, check() compares everything."""

    def __init__(self, seqs, *, hq, hkv, d, page=32, e4m3=False, seed=0, std=1.0, pad=0, gap=0, max_q=None, causal=1, window=0, sinks=0,
                 decay=1.0, lse=None, old=None):
        self.B = Batch(seqs, hkv=hkv, d=d, page=page, e4m3=e4m3, device=dev(), seed=seed, pad=pad, gap=gap)
        self.hq, self.d, self.decay, self.mask = hq, d, decay, (causal, window, sinks)
        g = torch.Generator().manual_seed(seed + 1)
        self.q = (torch.randn((self.B.total, hq, d), generator=g) * (std * d ** -0.5)).to(torch.bfloat16)
        self.max_q = max_q or self.B.max_q
        self.lse = torch.zeros((self.B.total, hq))
        for b, (n, L) in enumerate(seqs):
            lo = int(self.B.cu[b])
            l = opaged.attention(f64(self.q[lo:lo + n]), *self.B.kept(b), causal, window, sinks)[1]
            self.lse[lo:lo + n] = torch.from_numpy(l).float()
        if lse is not None:
            self.lse = lse
        # what other positions of the pool hold must not matter, nor change
        shape = (self.B.n_pages, hkv, page)
        w = torch.full((shape[0], hkv * page + 4 * (gap > 0)), float("nan"), device=dev())
        self.w = w.as_strided(shape, (w.shape[1], page, 1))
        self.old = []
        for b, (n, L) in enumerate(seqs):
            x = torch.rand((L, hkv), generator=g) * 3 if old is None else old[b]
            if L > n:
                pg, row = self.B.places(b)
                self.w[pg[:L - n], :, row[:L - n]] = x[:L - n].to(dev())
            elif n == 0 and L:
                pg, row = self.B.places(b)
                self.w[pg, :, row] = x.to(dev())
            self.old.append(x)
        self.before = self.w.clone()

    def ws(self, ra):
        B = self.B
        n = ra.paged_workspace_bytes(B.total, len(B.seqs), self.hq, B.hkv, self.d, self.max_q)
        return torch.full((n,), 0xff, dtype=torch.uint8, device=dev())

    def call(self, ra, stream=None, ws=None, q=None, lse=None):
        causal, window, sinks = self.mask
        ra.cache_weights(self.q.to(dev()) if q is None else q, self.lse.to(dev()) if lse is None else lse, self.B.k_cache, self.B.v_cache, self.w,
                         *self.B.args(), self.ws(ra) if ws is None else ws, max_q=self.max_q, decay=self.decay, causal=causal, window=window,
                         sinks=sinks, stream=stream, **self.B.kw())

    def check(self, what=""):
        """A score is a sum of d exact products in fp32, (d + 8) steps of 2^-23 of sum |q k| at most (a step, not half of
        one: the tensor cores may truncate); its exponent is rounded in base 2 (steps of 2^-23 of |s| and |lse|, twice),
        ex2 is 2^-21 off at most.  So a weight is off by that share of itself, and the sum of c of them by c halves of a step more."""
        touched = torch.zeros_like(self.w, dtype=torch.bool)
        for b, (n, L) in enumerate(self.B.seqs):
            if n == 0 or L == 0:
                continue
            lo = int(self.B.cu[b])
            q, lse = f64(self.q[lo:lo + n]), f64(self.lse[lo:lo + n])
            k, _ = self.B.kept(b)
            want, size = oevict.add_weights(f64(self.old[b]), q, lse, k, self.decay, *self.mask)
            pg, row = self.B.places(b)
            got = f64(self.w[pg, :, row])
            touched[pg, :, row] = True
            big = np.abs(lse[np.isfinite(lse)]).max() if np.isfinite(lse).any() else 0.0
            rel = ((self.d + 8) + 8) * 2.0 ** -23 * size + 2.0 ** -22 * big + 2.0 ** -20 + (n * self.hq / self.B.hkv + 16) * 2.0 ** -24
            worst = (np.abs(got - want) / (rel * np.abs(want) + 1e-37)).max()
            assert worst <= 1.0, f"{what}, sequence {b}: off by {worst:.3g} of its bound"
        same = (self.w == self.before) | (torch.isnan(self.w) & torch.isnan(self.before))
        assert (same | touched).all(), "a place of no position has changed"


SEQS = [(1, 1), (1, 16), (1, 17), (1, 700), (1, 33), (0, 40), (1, 129), (0, 0), (1, 512)]


@pytest.mark.parametrize("hq,hkv,d", [(8, 1, 128), (8, 8, 64), (6, 2, 64), (64, 4, 128), (16, 2, 64), (5, 1, 128)])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("page", [16, 48])
def test_single_tokens(ra, hq, hkv, d, e4m3, page):
    r = Run(SEQS, hq=hq, hkv=hkv, d=d, page=page, e4m3=e4m3, seed=hq, pad=3)
    r.call(ra)
    assert ra.sync_status() == ra.RA_OK
    r.check()


@pytest.mark.parametrize("seqs", [[(2, 2), (3, 300), (1, 5)], [(17, 17), (40, 333), (3, 700), (1, 1), (0, 9)], [(130, 130), (129, 640), (1, 257)],
                                  [(300, 300)], [(5, 3), (40, 17)]])
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (6, 2, 64), (16, 1, 64), (5, 5, 128)])
@pytest.mark.parametrize("e4m3", [False, True])
def test_rows(ra, seqs, hq, hkv, d, e4m3):
    """Several rows a sequence, rows before position 0 among them."""
    r = Run(seqs, hq=hq, hkv=hkv, d=d, e4m3=e4m3, seed=3, decay=0.75)
    r.call(ra)
    assert ra.sync_status() == ra.RA_OK
    r.check()


@pytest.mark.parametrize("seqs", [[(1, 1000), (1, 90), (1, 128)], [(3, 500), (9, 140)], [(140, 900), (65, 65), (1, 400)]])
@pytest.mark.parametrize("window,sinks", [(1, 0), (64, 0), (100, 5), (130, 300), (300, 17), (5000, 3)])
@pytest.mark.parametrize("decay", [0.0, 0.5, 1.0])
@pytest.mark.parametrize("e4m3", [False, True])
def test_windows(ra, seqs, window, sinks, decay, e4m3):
    r = Run(seqs, hq=8, hkv=2, d=64, page=16, e4m3=e4m3, seed=4, window=window, sinks=sinks, decay=decay)
    r.call(ra)
    assert ra.sync_status() == ra.RA_OK
    r.check()


@pytest.mark.parametrize("n", [1, 7, 150])
@pytest.mark.parametrize("e4m3", [False, True])
def test_all_rows_see_all_keys(ra, n, e4m3):
    r = Run([(n, 333), (n, n)], hq=8, hkv=2, d=128, e4m3=e4m3, seed=5, causal=0)
    r.call(ra)
    assert ra.sync_status() == ra.RA_OK
    r.check()


@pytest.mark.parametrize("n", [1, 20, 200])
def test_decay_of_zero_reads_nothing(ra, n):
    r = Run([(n, 300)], hq=8, hkv=2, d=64, seed=6, decay=0.0, old=[torch.full((300, 2), float("nan"))])
    r.call(ra)
    assert ra.sync_status() == ra.RA_OK
    r.check()
    assert not torch.isnan(r.w[r.B.places(0)[0], :, r.B.places(0)[1]]).any()


@pytest.mark.parametrize("n", [1, 30, 200])
def test_rows_without_an_lse_add_nothing(ra, n):
    r = Run([(n, 300)], hq=8, hkv=2, d=64, seed=7)
    r.lse[0] = -float("inf")
    r.call(ra)
    assert ra.sync_status() == ra.RA_OK
    r.check()


@pytest.mark.parametrize("n", [1, 3, 200])
@pytest.mark.parametrize("window", [0, 50])
def test_keys_that_nobody_sees_may_hold_anything(ra, n, window):
    """NaN and infinities behind the last position, behind a row's own and before a window: no other key changes."""
    r = Run([(n, 400)], hq=8, hkv=2, d=64, page=16, seed=8, window=window)
    clean = [x.clone() for x in r.B.k]
    if window:
        r.B.k[0][10], r.B.k[0][100, 1, 5] = float("nan"), float("inf")
    if n > 1:
        r.B.k[0][399, 0] = float("nan")  # the last row alone sees it
    r.B.fill()
    r.call(ra)
    assert ra.sync_status() == ra.RA_OK
    if n > 1:
        pg, row = r.B.places(0)
        assert torch.isnan(r.w[pg[399], 0, row[399]])
        r.w[pg[399], 0, row[399]] = 0.0
        want, _ = oevict.add_weights(f64(r.old[0]), f64(r.q), f64(r.lse), f64(clean[0]), 1.0, *r.mask)
        got = f64(r.w[pg, :, row])
        got[399, 0] = want[399, 0]
        assert np.isfinite(got).all() and np.allclose(got, want, rtol=1e-3)
    else:
        r.B.k = clean
        r.check()


def test_large_scores_and_any_lse(ra):
    """Scores of some hundreds, an lse that is not theirs."""
    for n in (1, 40, 150):
        r = Run([(n, 300)], hq=4, hkv=1, d=128, seed=9, std=30.0)
        r.lse += torch.randn(r.lse.shape, generator=torch.Generator().manual_seed(1))
        r.call(ra)
        assert ra.sync_status() == ra.RA_OK
        r.check(str(n))


def test_scales_that_are_no_powers_of_two(ra):
    for n in (1, 3, 40, 150):
        r = Run([(n, 300), (n, n + 1)], hq=8, hkv=2, d=64, e4m3=True, seed=10)
        f = 0.5 + torch.rand(r.B.k_scale.shape, generator=torch.Generator().manual_seed(2)).to(dev())
        r.B.k_scale.mul_(f)
        kept = r.B.kept

        def scaled(b):
            pg, row = r.B.places(b)
            codes = r.B.k_cache.view(torch.uint8)[pg, :, row].view(torch.float8_e4m3fn).float()
            return f64(codes) * f64(r.B.k_scale[pg, :, row])[..., None], kept(b)[1]

        r.B.kept = scaled
        r.call(ra)
        assert ra.sync_status() == ra.RA_OK
        r.check(str(n))


@pytest.mark.parametrize("n", [1, 30, 140])
def test_strides(ra, n):
    """q out of a fused projection, lse head-major, pages further apart than their rows."""
    r = Run([(n, 200), (1, 77)], hq=8, hkv=2, d=64, seed=11, gap=3, page=16)
    q = torch.zeros((r.B.total, 12, 64), dtype=torch.bfloat16, device=dev())
    q[:, 2:10] = r.q.to(dev())
    lse = r.lse.to(dev()).t().contiguous().t()
    r.call(ra, q=q[:, 2:10], lse=lse)
    assert ra.sync_status() == ra.RA_OK
    r.check()


@pytest.mark.parametrize("n", [1, 30, 140])
def test_the_same_bits_every_time(ra, n):
    r = Run([(n, 900), (1, 500), (n, 640)], hq=16, hkv=2, d=128, seed=12)
    got = []
    for _ in range(4):
        r.w.copy_(r.before)
        r.call(ra)
        got.append(r.w.clone())
    assert ra.sync_status() == ra.RA_OK
    for x in got[1:]:
        assert torch.equal(x.view(torch.int32), got[0].view(torch.int32))
    r.check()


@pytest.mark.parametrize("n", [1, 20, 150])
def test_arrays_that_hold_anything(ra, n):
    """Lengths, rows and pages outside what there is: nothing outside the tensors is touched, other sequences are right."""
    r = Run([(n, 300), (n, 200), (n, 260)], hq=8, hkv=2, d=64, page=16, seed=13)
    pg, row = r.B.places(1)
    r.B.dtable[1] = torch.tensor([-1, 2 ** 31 - 1, r.B.n_pages, -2 ** 31] * 8, dtype=torch.int32, device=dev())[:r.B.dtable.shape[1]]
    r.call(ra)
    assert ra.sync_status() == ra.RA_OK
    assert torch.equal(torch.nan_to_num(r.w[pg, :, row]), torch.nan_to_num(r.before[pg, :, row])), "pages that the table does not name"
    r.B.seqs[1] = (0, 0)
    r.check()
    for lens in ([2 ** 31 - 1, -5, 300], [-2 ** 31, 2 ** 31 - 1, 2 ** 30]):
        r.B.dlen.copy_(torch.tensor(lens, dtype=torch.int32))
        r.call(ra)
    r.B.dlen.copy_(r.B.kv_len)
    for cu in ([5, -7, 2 ** 31 - 1, 3], [0, 2 ** 31 - 1, -2 ** 31, 1]):
        r.B.dcu.copy_(torch.tensor(cu, dtype=torch.int32))
        r.call(ra)
    assert ra.sync_status() == ra.RA_OK


@pytest.mark.parametrize("n", [1, 20, 150])
def test_captured_and_on_another_stream(ra, n):
    r = Run([(n, 400), (n, 231)], hq=8, hkv=2, d=128, seed=14)
    ws, q, lse = r.ws(ra), r.q.to(dev()), r.lse.to(dev())
    r.call(ra, ws=ws, q=q, lse=lse)
    torch.cuda.synchronize()
    want = r.w.clone()
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        r.call(ra, ws=ws, q=q, lse=lse)
    for how in ("replay", "stream"):
        r.w.copy_(r.before)
        ws.fill_(0x5a)
        torch.cuda.synchronize()
        if how == "replay":
            graph.replay()
        else:
            r.call(ra, stream=s, ws=ws, q=q, lse=lse)
        torch.cuda.synchronize()
        assert torch.equal(r.w.view(torch.int32), want.view(torch.int32)), how
    assert ra.sync_status() == ra.RA_OK


@pytest.mark.parametrize("n", [1, 2, 9, 40, 300])
@pytest.mark.parametrize("g", [1, 3, 7, 9, 33, 100, 128])
@pytest.mark.parametrize("e4m3", [False, True])
def test_query_heads_of_a_kv_head(ra, n, g, e4m3):
    """Units of the chunk kernel that 128 rows do not fill, head-major q."""
    r = Run([(n, n + 390), (1, 200), (n, n)], hq=2 * g, hkv=2, d=64, page=48, e4m3=e4m3, seed=g, decay=0.5)
    q = r.q.transpose(0, 1).contiguous().to(dev()).transpose(0, 1)
    r.call(ra, q=q)
    assert ra.sync_status() == ra.RA_OK
    r.check()


@pytest.mark.parametrize("n", [1, 5, 40, 200])
@pytest.mark.parametrize("batch", [40, 600])
def test_batches_of_all_sizes(ra, n, batch):
    """Sequences with and without rows, more of them than one part of shared memory holds."""
    seqs = [(n if b % 7 == 0 else b % 3, (61 * b) % 300 + 1) for b in range(batch)]
    seqs = [(min(a, L), L) for a, L in seqs]
    r = Run(seqs, hq=4, hkv=1, d=64, page=16, seed=n, window=100, sinks=3, decay=0.5)
    r.call(ra)
    assert ra.sync_status() == ra.RA_OK
    r.check()


@pytest.mark.parametrize("n", [1, 7, 60, 200])
@pytest.mark.parametrize("max_q", [1, 5, 33, 150])
def test_rows_behind_max_q_do_not_count(ra, n, max_q):
    seqs = [(n, 300), (min(n, 3), 100)]
    r = Run(seqs, hq=8, hkv=2, d=64, seed=16, max_q=max_q)
    lse = r.lse.clone()
    for b in range(2):
        r.lse[int(r.B.cu[b]) + max_q:int(r.B.cu[b + 1])] = -float("inf")
    r.call(ra, lse=lse.to(dev()))
    assert ra.sync_status() == ra.RA_OK
    r.check()


@pytest.mark.parametrize("n", [1, 6, 60, 200])
def test_rows_of_zeros_and_of_very_different_sizes(ra, n):
    """e4m3 scales from 2^-120 (rows of zeros) to 2^40; keys that some lse makes large weights of."""
    r = Run([(n, 300)], hq=8, hkv=2, d=128, e4m3=True, seed=17, std=0.0)
    k = r.B.k[0]
    k[10:40] = 0.0
    k[50:60] *= 2.0 ** -70
    k[60:70] *= 2.0 ** 40
    k[70] = 2.0 ** -133
    r.B.fill()
    r.q = (torch.randn(r.q.shape, generator=torch.Generator().manual_seed(18)) * 2.0 ** -40).to(torch.bfloat16)
    r.lse = torch.randn(r.lse.shape, generator=torch.Generator().manual_seed(19)) * 5
    r.call(ra)
    assert ra.sync_status() == ra.RA_OK
    r.check()


@pytest.mark.parametrize("n", [1, 6, 60, 200])
@pytest.mark.parametrize("e4m3", [False, True])
def test_lse_of_every_size(ra, n, e4m3):
    """Far from the scores: weights of nothing and of infinity, as the definition has them in fp32."""
    r = Run([(n, 300)], hq=8, hkv=2, d=64, e4m3=e4m3, seed=20)
    for at, x in ((0, 1e4), (1, 1e9), (2, 3e38), (3, float("inf")), (4, 200.0)):
        r.lse[:, at] = x  # heads of the first KV head and the first of the second add nothing
    r.call(ra)
    assert ra.sync_status() == ra.RA_OK
    r.check()
    r.w.copy_(r.before)
    r.lse[:, 7] = -1e5
    r.call(ra)
    pg, row = r.B.places(0)
    w = r.w[pg, :, row]
    assert torch.isinf(w[:300 - n + 1, 1]).all() and not torch.isinf(w[:, 0]).any()


def test_many_sequences(ra):
    """More of them than threads, as many as a call takes, most without rows."""
    seqs = [(1, 1 + (7 * b) % 40) if b % 5 == 0 else (0, 3) for b in range(4096)]
    r = Run(seqs, hq=2, hkv=1, d=64, page=16, seed=15)
    r.call(ra)
    assert ra.sync_status() == ra.RA_OK
    r.check()


@pytest.mark.parametrize("n,L,hq,hkv,e4m3", [(1, 70000, 8, 1, False), (1, 40000, 16, 1, True), (300, 9000, 8, 2, False), (2, 30000, 64, 8, True),
                                             (1100, 1100, 8, 1, True), (64, 20000, 64, 1, False), (2000, 5000, 6, 2, False)])
@pytest.mark.parametrize("window", [0, 1500])
def test_long_ones_against_torch_in_64_bits(ra, n, L, hq, hkv, e4m3, window):
    """Every position of long sequences; bounds as in Run.check, with the whole batch's largest sums."""
    g = torch.Generator(device=dev()).manual_seed(n)
    d, page = 128, 64
    pages = -(-L // page)
    table = torch.randperm(pages, generator=g, device=dev()).to(torch.int32)[None]
    k = torch.randn((pages, hkv, page, d), generator=g, device=dev()).to(torch.bfloat16)
    scale = None
    if e4m3:
        k = (k.float() * 40).to(torch.float8_e4m3fn)
        scale = torch.exp2(torch.randint(-9, -5, (pages, hkv, page), generator=g, device=dev()).float())
    v = torch.zeros_like(k)
    q = (torch.randn((n, hq, d), generator=g, device=dev()) * d ** -0.5).to(torch.bfloat16)
    w = torch.rand((pages, hkv, page), generator=g, device=dev())
    cu, ln = torch.tensor([0, n], dtype=torch.int32, device=dev()), torch.tensor([L], dtype=torch.int32, device=dev())
    ws = torch.empty(ra.paged_workspace_bytes(n, 1, hq, hkv, d, n), dtype=torch.uint8, device=dev())
    lse = torch.full((n, hq), 8.0, device=dev())
    t = table[0].long()
    old = w[t].transpose(0, 1).reshape(hkv, -1)[:, :L].double()
    ra.cache_weights(q, lse, k, v, w, table, cu, ln, ws, max_q=n, decay=0.5, window=window, sinks=9 if window else 0, k_scale=scale, v_scale=scale)
    assert ra.sync_status() == ra.RA_OK
    kk = k.double() if scale is None else k.double() * scale.double()[..., None]
    kk = kk[t].transpose(0, 1).reshape(hkv, -1, d)[:, :L]
    got = w[t].transpose(0, 1).reshape(hkv, -1)[:, :L].double()
    j = torch.arange(L, device=dev())
    want = torch.where(j < L - n, 0.5 * old, torch.zeros_like(old))
    size = 0.0
    for h in range(hq):
        for lo in range(0, n, 256):
            i = torch.arange(L - n + lo, L - n + min(n, lo + 256), device=dev())[:, None]
            see = j <= i
            if window:
                see = see & ((j > i - window) | (j < 9))
            s = q[lo:lo + 256, h].double() @ kk[h // (hq // hkv)].T
            want[h // (hq // hkv)] += torch.where(see, torch.exp(s - 8.0), 0.0).sum(0)
            size = max(size, float((q[lo:lo + 256, h].double().abs() @ kk[h // (hq // hkv)].abs().T).max()))
    rel = (d + 16) * 2.0 ** -23 * size + 2.0 ** -22 * 8 + 2.0 ** -20 + (n * hq / hkv + 16) * 2.0 ** -24
    worst = float(((got - want).abs() / (rel * want.abs() + 1e-37)).max())
    assert worst <= 1.0, f"off by {worst:.3g} of its bound"


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("page,hq,hkv,d,seqs", [
    (16, 16, 2, 64, [(16, 1500), (17, 900), (16, 300), (33, 1100)]),     # one unit of 128 rows, two, one, three
    (128, 8, 4, 128, [(64, 3000), (65, 2000), (64, 128), (64, 70)]),     # the same with all pairs of two tiles, then one tile
    (48, 32, 2, 128, [(8, 6000), (24, 3000), (16, 257), (9, 255)]),
    (256, 6, 1, 64, [(21, 5000), (22, 5000), (43, 129), (84, 2100)]),    # units of 126 rows
])
@pytest.mark.parametrize("window", [0, 700])
def test_few_units_see_every_pair_of_tiles(ra, page, hq, hkv, d, seqs, window, e4m3):
    r = Run(seqs, hq=hq, hkv=hkv, d=d, page=page, e4m3=e4m3, seed=23, decay=0.5, window=window, sinks=4 if window else 0)
    r.call(ra)
    assert ra.sync_status() == ra.RA_OK
    r.check()


@pytest.mark.parametrize("batch", [223, 224, 225, 257])
def test_batches_whose_shares_leave_shared_memory(ra, batch):
    seqs = [(14 + b % 5, 14 + b % 5 + 37 * (b % 11)) for b in range(batch)]
    r = Run(seqs, hq=8, hkv=1, d=64, page=16, seed=24)
    r.call(ra)
    assert ra.sync_status() == ra.RA_OK
    r.check()


@pytest.mark.parametrize("n", [1, 30, 300])
def test_two_calls_at_once(ra, n):
    """Batches, pools and workspaces of their own on two streams, again and again."""
    runs = [Run([(n, n + 2000), (n, n + 90)], hq=8, hkv=2, d=64, page=16, e4m3=s == 1, seed=25 + s) for s in range(2)]
    want = []
    for r in runs:
        r.call(ra)
        torch.cuda.synchronize()
        want.append(r.w.clone())
    args = [(r.ws(ra), r.q.to(dev()), r.lse.to(dev())) for r in runs]
    streams = [torch.cuda.Stream() for _ in runs]
    torch.cuda.synchronize()
    for r in runs:
        r.w.copy_(r.before)
    torch.cuda.synchronize()
    for k in range(6):
        for r, s, (ws, q, lse) in zip(runs, streams, args):
            with torch.cuda.stream(s):
                r.w.copy_(r.before)
                r.call(ra, stream=s, ws=ws, q=q, lse=lse)
    torch.cuda.synchronize()
    assert ra.sync_status() == ra.RA_OK
    for r, w in zip(runs, want):
        assert torch.equal(torch.nan_to_num(r.w, nan=-1.0), torch.nan_to_num(w, nan=-1.0))


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("n", [1, 40, 300])
def test_pages_far_apart(ra, e4m3, n):
    """Pages whose places pass 32 bits, in elements and in bytes: weights and eviction give what they give with pages side by side."""
    r = Run([(n, n + 200), (min(n, 7), 150)], hq=8, hkv=2, d=64, page=64, e4m3=e4m3, seed=27)
    pages = r.B.n_pages
    near = [r.B.k_cache, r.B.v_cache, r.w] + ([r.B.k_scale, r.B.v_scale] if e4m3 else [])
    apart = (2 ** 32 + 4096) // (pages - 1) // 64 * 64 + 64  # elements: the last page lies behind 2^32 of them
    far = []
    for x in near:
        base = torch.empty(apart * (pages - 1) + x[0].numel(), dtype=x.dtype, device=dev())
        y = base.as_strided(x.shape, (apart, *x.stride()[1:]))
        y.view(torch.uint8 if e4m3 and x.element_size() == 1 else x.dtype).copy_(x.view(torch.uint8 if e4m3 and x.element_size() == 1 else x.dtype))
        far.append(y)
    keep, lens = (torch.tensor(v, dtype=torch.int32, device=dev()) for v in ((70, 60), (0, 0)))
    res = []
    for pools in (near, far):
        kw = dict(k_scale=pools[3], v_scale=pools[4]) if e4m3 else {}
        ra.cache_weights(r.q.to(dev()), r.lse.to(dev()), *pools[:3], *r.B.args(), r.ws(ra), max_q=r.max_q, **kw)
        kept = torch.empty((2, 2, 70), dtype=torch.int32, device=dev())
        ra.cache_evict(*pools[:3], r.B.dtable, r.B.dlen, keep, lens, kept, sinks=1, recent=5, **kw)
        torch.cuda.synchronize()
        assert ra.sync_status() == ra.RA_OK
        res.append([kept] + [x.contiguous().view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[x.element_size()]) for x in pools])
    for a, b in zip(*res):
        assert torch.equal(a, b)
