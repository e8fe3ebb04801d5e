"""Batches whose device arrays are not the host's: a max_q that is no sequence's number of rows, arrays that change
under a captured graph, and arrays that hold anything."""
import random

import numpy as np
import pytest
import torch

from oracle import paged as opaged
from tests.gpu_util import dev
from tests.paged_util import Batch, check


@pytest.fixture(scope="module")
def ra():
    from online_softmax_attention_zigzag_gb300 import ringattn
    ringattn.lib()
    torch.cuda.set_device(0)
    return ringattn


def _queries(n, hq, d, seed):
    return (torch.randn((n, hq, d), generator=torch.Generator().manual_seed(seed)) * d ** -0.5).to(torch.bfloat16)


# ------------------------------------------------------------------ max_q
@pytest.mark.gpu
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("ns,max_q", [((1, 5, 3), 2), ((1, 5, 3), 4), ((1, 2, 0), 4), ((1, 5, 3), 40), ((1, 5, 3), 2 ** 31 - 1),
                                      ((200, 1, 33), 7), ((200, 1, 33), 130), ((300, 20, 7), 33), ((20, 3, 1), 5000)])
def test_max_q_below_and_above_the_rows(ra, e4m3, ns, max_q):
    """Rows at and behind max_q stay as they were, the others are those of the whole batch."""
    hq, hkv, d = 8, 2, 128
    B = Batch([(n, L) for n, L in zip(ns, (700, 333, 90))], hkv=hkv, d=d, page=32, e4m3=e4m3, device=dev(), seed=1, pad=2)
    q = _queries(B.total, hq, d, 2)
    for kw in ({}, dict(window=100, sinks=5)):
        out = torch.full((B.total, hq, d), float("nan"), device=dev())
        lse = torch.full((B.total, hq), float("nan"), device=dev())
        ws = torch.full((ra.paged_workspace_bytes(B.total, 3, hq, hkv, d, max_q),), 255, dtype=torch.uint8, device=dev())
        ra.fwd_paged(q.to(dev()), B.k_cache, B.v_cache, out, lse, *B.args(), ws, max_q=max_q, **B.kw(), **kw)
        assert ra.sync_status() == ra.RA_OK
        cu = B.cu.tolist()
        for b, (n, L) in enumerate(B.seqs):
            m = min(n, max_q)
            ref = opaged.attention(q[cu[b]:cu[b + 1]].double().numpy(), *B.kept(b), True, kw.get("window", 0), kw.get("sinks", 0))
            check(out[cu[b]:cu[b] + m], lse[cu[b]:cu[b] + m], [x[:m] for x in ref], d, False, f"sequence {b}")
            assert torch.isnan(out[cu[b] + m:cu[b + 1]]).all() and torch.isnan(lse[cu[b] + m:cu[b + 1]]).all()
        assert torch.isnan(out[cu[-1]:]).all()


# ------------------------------------------------------------------ a graph over batches of other shapes
@pytest.mark.gpu
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("max_q", [4, 64])
def test_a_graph_whose_rows_change(ra, e4m3, max_q):
    """Captured once for 96 token rows and up to 6 sequences; cu, kv_len and the table change between replays."""
    hq, hkv, d, page, total, batch = 8, 2, 128, 32, 96, 6
    pool = Batch([(1, 900)] * batch, hkv=hkv, d=d, page=page, e4m3=e4m3, device=dev(), seed=3)
    cu = torch.zeros(batch + 1, dtype=torch.int32, device=dev())
    ln = torch.zeros(batch, dtype=torch.int32, device=dev())
    q = _queries(total, hq, d, 4)
    g = torch.Generator().manual_seed(5)
    kn, vn = (torch.randn((total, hkv, d), generator=g).to(torch.bfloat16) for _ in range(2))
    qd, kd, vd = q.to(dev()), kn.to(dev()), vn.to(dev())
    out, lse = torch.empty((total, hq, d), device=dev()), torch.empty((total, hq), device=dev())
    ws = torch.empty(ra.paged_workspace_bytes(total, batch, hq, hkv, d, max_q), dtype=torch.uint8, device=dev())
    gr, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side), torch.cuda.graph(gr, stream=side):
        ra.cache_append(kd, vd, pool.k_cache, pool.v_cache, pool.dtable, cu, ln, **pool.kw())
        ra.fwd_paged(qd, pool.k_cache, pool.v_cache, out, lse, pool.dtable, cu, ln, ws, max_q=max_q, **pool.kw())
    r = random.Random(6)
    for rows in ([1] * 6, [0, max_q, 1, 0, 3, 2], [0] * 6, [max_q] + [0] * 5, [1, 1, 0, 0, 0, 0]):
        lens = [max(n, r.randint(0, 900)) for n in rows]
        cu.copy_(torch.tensor(np.concatenate([[0], np.cumsum(rows)]), dtype=torch.int32))
        ln.copy_(torch.tensor(lens, dtype=torch.int32))
        out.fill_(float("nan"))
        lse.fill_(float("nan"))
        torch.cuda.synchronize()
        gr.replay()
        torch.cuda.synchronize()
        assert ra.sync_status() == ra.RA_OK
        at = 0
        for b, (n, L) in enumerate(zip(rows, lens)):
            pool.k[b][L - n:L], pool.v[b][L - n:L] = kn[at:at + n], vn[at:at + n]
            k, v = pool.kept(b)
            if n:
                ref = opaged.attention(q[at:at + n].double().numpy(), k[:L], v[:L])
                check(out[at:at + n], lse[at:at + n], ref, d, False, f"{rows}: sequence {b}")
            at += n
        assert torch.isnan(out[at:]).all() and torch.isnan(lse[at:]).all()


# ------------------------------------------------------------------ arrays that hold anything
ANY_CU = [[0, 10, 4, 12, 20], [-5, 3, 7, 11, 15], [0, 5, 2 ** 31 - 1, 9, 20], [20, 15, 10, 5, 0], [0, 20, 0, 20, 0], [-2 ** 31, 2 ** 31 - 1, 3, 8, 8],
          [7, 7, 7, 7, 7], [30, 40, 50, 60, 70], [3, 6, 9, 12, 15]]
ANY_LEN = [-1, 2 ** 31 - 1, -2 ** 31, 321, 500, 160, 3, 0]


def _seq(cu, lens, b, total, most):
    """A sequence's rows and length as the header clamps them."""
    q0 = min(max(cu[b], 0), total)
    n = min(max(cu[b + 1], q0), total) - q0
    return q0, n, min(max(lens[b], 0), most)


@pytest.mark.parametrize("total,item,max_q", [(20, 16, 20), (20, 1, 20), (20, 2, 5), (300, 32, 2 ** 20), (1000, 7, 999)])
def test_lists_of_items_stay_within_their_room(total, item, max_q):
    """Host: the chunk kernel's list of items, made as paged_plan_kernel makes it, for arrays that hold anything: no
    more items than there is room for, every item of rows inside the tensors."""
    r = random.Random(total)
    cases = [list(c) for c in ANY_CU] + [[r.choice([r.randint(-9, total + 9), r.randint(-2 ** 31, 2 ** 31 - 1)]) for _ in range(9)]
                                         for _ in range(200)]
    for cu in cases:
        B = len(cu) - 1
        room = total // item + B
        seqs = [_seq(cu, [0] * B, b, total, 1) for b in range(B)]
        pairs = [-(-min(n, max_q) // item) for _, n, _ in seqs]
        base, at = [], 0
        for n in pairs:  # exclusive sums, cut off
            base.append(min(at, room))
            at += n
        E = min(at, room)
        base.append(E)
        assert base == sorted(base) and base[0] == 0
        for e in range(E):
            lo, hi = 0, B  # the kernel's search
            while hi - lo > 1:
                mid = (lo + hi) // 2
                if base[mid] <= e:
                    lo = mid
                else:
                    hi = mid
            assert base[lo] <= e < base[lo + 1]
            q0, n, _ = seqs[lo]
            ta = (e - base[lo]) * item
            tb = min(n, max_q, ta + item)
            assert 0 <= ta < tb and q0 + tb <= total


@pytest.mark.gpu
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("cu", ANY_CU)
@pytest.mark.parametrize("max_q", [2, 20])  # few rows, and a chunk
def test_arrays_that_hold_anything(ra, e4m3, cu, max_q):
    """Rows and lengths are clamped: a row that one sequence alone has is that sequence's, one that none has stays as it
    was, and nothing around the tensors changes."""
    hq, hkv, d, page, total = 8, 1, 64, 16, 20
    for first in (0, 4):
        lens = ANY_LEN[first:first + 4]
        B = Batch([(1, 320)] * 4, hkv=hkv, d=d, page=page, e4m3=e4m3, device=dev(), seed=7)
        most = 320  # positions that the narrowed table has
        table = B.dtable[:, :most // page].contiguous()
        dcu, dlen = torch.tensor(cu, dtype=torch.int32, device=dev()), torch.tensor(lens, dtype=torch.int32, device=dev())
        q = _queries(total, hq, d, 8)
        guard = 40
        bout = torch.full((total + 2 * guard, hq, d), float("nan"), device=dev())
        blse = torch.full((total + 2 * guard, hq), float("nan"), device=dev())
        out, lse = bout[guard:guard + total], blse[guard:guard + total]
        ws = torch.empty(ra.paged_workspace_bytes(total, 4, hq, hkv, d, max_q), dtype=torch.uint8, device=dev())
        ra.fwd_paged(q.to(dev()), B.k_cache, B.v_cache, out, lse, table, dcu, dlen, ws, max_q=max_q, **B.kw())
        assert ra.sync_status() == ra.RA_OK
        owners = [[] for _ in range(total)]
        for b in range(4):
            q0, n, L = _seq(cu, lens, b, total, most)
            for t in range(min(n, max_q)):
                owners[q0 + t].append(b)
        for b in range(4):
            q0, n, L = _seq(cu, lens, b, total, most)
            mine = [t for t in range(min(n, max_q)) if owners[q0 + t] == [b]]
            if not mine:
                continue
            k, v = B.kept(b)
            ref = opaged.attention(q[q0:q0 + n].double().numpy(), k[:L], v[:L])
            at = [q0 + t for t in mine]
            check(out[at], lse[at], [x[mine] for x in ref], d, False, f"sequence {b}")
        none = [t for t in range(total) if not owners[t]]
        assert torch.isnan(out[none]).all() and torch.isnan(lse[none]).all()
        for x in (bout, blse):
            assert torch.isnan(x[:guard]).all() and torch.isnan(x[guard + total:]).all()
        # the copies: what a search over such a cu finds is not specified; nothing outside the tensors is touched, and the pages
        # that the table does not name stay as they were
        x = torch.ones((total, hkv, d), dtype=torch.bfloat16, device=dev())
        named = torch.zeros(B.n_pages, dtype=torch.bool)
        named[B.table[:, :most // page].flatten().long()] = True
        before = B.k_cache.view(torch.uint8)[~named.to(dev())].clone()
        ra.cache_append(x, x, B.k_cache, B.v_cache, table, dcu, dlen, **B.kw())
        buf = torch.full((total * hkv * d + 4096,), float("nan"), dtype=torch.bfloat16, device=dev())
        ko, vo = buf[1024:1024 + total * d].view(hkv, total, d), torch.empty((hkv, total, d), dtype=torch.bfloat16, device=dev())
        ra.cache_read(B.k_cache, B.v_cache, ko, vo, table, dcu, dlen, **B.kw())
        assert ra.sync_status() == ra.RA_OK
        assert torch.equal(B.k_cache.view(torch.uint8)[~named.to(dev())], before)
        assert torch.isnan(buf[:1024]).all() and torch.isnan(buf[1024 + total * d:]).all()
