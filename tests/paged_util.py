"""A small host model of a paged batch for the paged-cache tests: pools, tables and sequences
on the host, their device copies, and error bounds."""
from __future__ import annotations

import numpy as np
import torch

from oracle import paged as opaged


class Batch:
    """Sequences (n rows, length L) over a pool with a shuffled block table.

    The pool starts full of NaN, so that rows nobody wrote show up when they are read; pages that
    the table does not name stay that way."""

    def __init__(self, seqs, *, hkv, d, page, e4m3, device, seed=0, spare=2, pad=0, fill=True, gap=0):
        g = torch.Generator().manual_seed(seed)
        self.seqs, self.hkv, self.d, self.page, self.e4m3 = list(seqs), hkv, d, page, e4m3
        n = [r for r, _ in seqs]
        need = [-(-max(L, 1) // page) for _, L in seqs]
        self.n_pages = sum(need) + spare
        order = torch.randperm(self.n_pages, generator=g).to(torch.int32)
        self.table = torch.full((len(seqs), max(need) + 1), 2 ** 30, dtype=torch.int32)
        at = 0
        for b, k in enumerate(need):
            self.table[b, :k] = order[at:at + k]
            at += k
        self.cu = torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32)
        self.kv_len = torch.tensor([L for _, L in seqs], dtype=torch.int32)
        self.total = sum(n) + pad
        self.max_q = max(1, max(n))
        # every sequence's K and V, bf16 [L, hkv, d]
        self.k = [torch.randn((L, hkv, d), generator=g).to(torch.bfloat16) for _, L in seqs]
        self.v = [torch.randn((L, hkv, d), generator=g).to(torch.bfloat16) for _, L in seqs]
        dt = torch.uint8 if e4m3 else torch.bfloat16
        shape = (self.n_pages, hkv * page + gap, d)

        def pool():  # pages `gap` rows apart; 0x7f is an e4m3 NaN
            x = torch.full(shape, 0x7f, dtype=dt) if e4m3 else torch.full(shape, float("nan"), dtype=dt)
            x = x.to(device)
            x = x.view(torch.float8_e4m3fn) if e4m3 else x
            return x.as_strided((self.n_pages, hkv, page, d), (shape[1] * d, page * d, d, 1))

        self.k_cache, self.v_cache = pool(), pool()
        self.k_scale = self.v_scale = None
        if e4m3:
            s = torch.full((2, self.n_pages, hkv, page), float("nan"), device=device)
            self.k_scale, self.v_scale = s[0], s[1]
        self.device = device
        self.dtable, self.dcu, self.dlen = (x.to(device) for x in (self.table, self.cu, self.kv_len))
        if fill:
            self.fill()

    def places(self, b):
        L = self.seqs[b][1]
        pos = torch.arange(L)
        return self.table[b, pos // self.page].long().to(self.device), (pos % self.page).to(self.device)

    def fill(self):
        """Every position's K and V into the pool, by plain indexing (no library call)."""
        for b in range(len(self.seqs)):
            page, row = self.places(b)
            for x, cache, scale in ((self.k[b], self.k_cache, self.k_scale), (self.v[b], self.v_cache, self.v_scale)):
                if self.e4m3:
                    codes, s = opaged.quantise(x.double().numpy())
                    c8 = torch.from_numpy(codes).float().to(torch.float8_e4m3fn).to(self.device)
                    cache.view(torch.uint8)[page, :, row] = c8.view(torch.uint8)
                    scale[page, :, row] = torch.from_numpy(s).float().to(self.device)
                else:
                    cache[page, :, row] = x.to(self.device)

    def kept(self, b):
        """K and V of sequence b as the pool holds them, float64 [L, hkv, d]."""
        if not self.e4m3:
            return self.k[b].double().numpy(), self.v[b].double().numpy()
        res = []
        for x in (self.k[b], self.v[b]):
            c, s = opaged.quantise(x.double().numpy())
            res.append(c * s[..., None])
        return res

    def kw(self):
        return dict(k_scale=self.k_scale, v_scale=self.v_scale)

    def args(self):
        return self.dtable, self.dcu, self.dlen


def out_bound(ref, d, out_bf16, p_eps=2.0 ** -8):
    """Element bounds of (out, lse) for oracle.paged.attention's results.

    A score is a sum of d exact products kept in fp32: its error is at most (d + 8) steps of
    2^-23 (a step and not half of one: the tensor cores may truncate) of sum |q k|.  p = 2^x
    carries that, 2^-21 of the hardware's exponential and its argument's rounding (a step of
    2^-23 of |x| <= 1.5 (|s| + |max|), so at most 3 sum |q k|), and half a step of its 16-bit
    type (bf16: 2^-8); out divides two such sums, so twice all that of sum p |v|, plus fp32
    sums (2^-18 covers up to 32 steps), and half a bf16 step (2^-8) of the result."""
    out, lse, mag, size = ref
    score = ((d + 8) + 6) * 2.0 ** -23 * size + 2.0 ** -21
    tol = (2 * (p_eps + score[..., None]) + 2.0 ** -18) * mag * 1.02
    if out_bf16:
        tol = tol + 2.0 ** -8 * (np.abs(out) + tol)
    lse_fin = np.where(np.isfinite(lse), np.abs(lse), 0.0)
    return tol + 1e-30, score + 2.0 ** -18 + 2.0 ** -22 * lse_fin


def check(got_out, got_lse, ref, d, out_bf16, what="", p_eps=2.0 ** -8):
    """Both outputs of one sequence, [n, Hq, d] and [n, Hq] tensors, within the bounds."""
    out, lse = ref[0], ref[1]
    o, l = got_out.double().cpu().numpy(), got_lse.double().cpu().numpy()
    to, tl = out_bound(ref, d, out_bf16, p_eps)
    assert np.array_equal(np.isneginf(l), np.isneginf(lse)), what
    fin = np.isfinite(lse)
    assert np.isfinite(o).all(), what
    worst = (np.abs(o - out) / to).max() if o.size else 0.0
    assert worst <= 1.0, f"{what}: out off by {worst:.3g} of its bound"
    worst = (np.abs(l[fin] - lse[fin]) / tl[fin]).max() if fin.any() else 0.0
    assert worst <= 1.0, f"{what}: lse off by {worst:.3g} of its bound"
