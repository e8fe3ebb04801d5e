"""Measured cases of the paged key/value cache: writing it, reading it back, and attending over it.

The cache is a pool of pages.  ``k_cache`` and ``v_cache`` are [n_pages, Hkv, page_size, d], bf16
or e4m3 with one power-of-two fp32 scale per (page, head, row) in ``k_scale`` / ``v_scale``
[n_pages, Hkv, page_size].  A batch of B sequences is described by ``block_table`` [B, max_pages]
(int32; page of every page_size positions), ``cu`` [B + 1] (int32; rows of sequence b are
cu[b] .. cu[b+1]) and ``kv_len`` [B] (int32; its length with those rows): row t of sequence b is
position kv_len[b] - (cu[b+1] - cu[b]) + t.

* ``append``: k_new, v_new [total, Hkv, d] go to their positions' places (quantised for e4m3).
* ``read``:   the rows come back as bf16, head-major [Hkv, total, d], as the ring entry points take them.
* ``attend``: q [total, Hq, d] over the keys of its sequence: j <= i (or all, without the causal
  mask), and with a window W only j > i - W or j < sinks; out [total, Hq, d] bf16, lse [total, Hq].
  No 1/sqrt(d) scale is applied: q comes scaled.
"""
from __future__ import annotations

import math
import random

import torch

own = False

E4M3_MAX = 448.0
MIN_EXP = -120  # smallest scale exponent, so that every stored value is a bf16 number


# ------------------------------------------------------------------ cases
def _case(op, name=None, **kw):
    c = dict(op=op, batch=1, rows_lo=1, rows_hi=1, ctx_lo=0, ctx_hi=0, hq=64, hkv=8, d=128, page=64, dtype="bf16",
             causal=1, window=0, sinks=0, fused=False)
    c.update(kw)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one decoding step of 64 sequences: one new token each, quantised
        _case("append", "append_decode_e4m3_b64", batch=64, ctx_lo=100, ctx_hi=16384, dtype="e4m3"),
        # a whole 32k prompt written at once after the ring's prefill, quantised
        _case("append", "append_prompt_e4m3_32k", rows_lo=32768, rows_hi=32768, dtype="e4m3"),
        # prompts of a batch, odd lengths, sliced out of a fused q/k/v projection, kept in bf16
        _case("append", "append_ragged_bf16_d64", batch=17, rows_lo=33, rows_hi=2049, ctx_hi=700, hq=8, hkv=8, d=64,
              page=48, fused=True),
        # a 128k context handed back to the ring, from 8 bits
        _case("read", "read_e4m3_128k", rows_lo=131072, rows_hi=131072, hq=32, dtype="e4m3"),
        # the contexts of a batch of short conversations, small pages, bf16
        _case("read", "read_ragged_bf16_d64", batch=33, rows_lo=1, rows_hi=1500, ctx_hi=300, hq=8, hkv=8, d=64, page=16),
        # the smallest call: one conversation's next token
        _case("attend", "decode_b1_777", ctx_lo=776, ctx_hi=776, page=16),
        # a serving batch's next tokens, lengths all over the range
        _case("attend", "decode_b64_16k", batch=64, ctx_lo=200, ctx_hi=16384),
        # few very long contexts in 8 bits: the cache's bytes are all there is
        _case("attend", "decode_e4m3_b8_128k", batch=8, ctx_lo=100000, ctx_hi=131071, hq=32, dtype="e4m3"),
        # long contexts under a sliding window with first tokens that stay visible
        _case("attend", "decode_window_e4m3_b48", batch=48, ctx_lo=3000, ctx_hi=32768, dtype="e4m3", window=4096, sinks=4),
        # several proposed tokens of each sequence checked at once
        _case("attend", "verify_t8_b16_32k", batch=16, rows_lo=8, rows_hi=8, ctx_lo=1000, ctx_hi=32768),
        # a large chunk of a long prompt
        _case("attend", "chunk_4096_of_32k", rows_lo=4096, rows_hi=4096, ctx_lo=28672, ctx_hi=28672),
        # chunks and single tokens in one batch, odd sizes and pages, in 8 bits, windowed
        _case("attend", "mixed_e4m3_window_b12", batch=12, rows_lo=1, rows_hi=1023, ctx_hi=9000, hq=32, page=48,
              dtype="e4m3", window=2500, sinks=17),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "read", "attend", "attend", "attend"])
    hq, hkv, d = rng.choice([(64, 8, 128), (32, 8, 128), (8, 2, 128), (8, 8, 64), (16, 16, 128), (6, 2, 64), (8, 1, 128)])
    c = _case(op, hq=hq, hkv=hkv, d=d, page=rng.choice([16, 32, 48, 64, 128, 256]), dtype=rng.choice(["bf16", "e4m3"]),
              batch=_log(rng, 1, 128), fused=rng.random() < 0.3)
    if op == "attend":
        kind = rng.choice(["decode", "decode", "few", "chunk"])
        c["rows_hi"] = {"decode": 1, "few": _log(rng, 2, 32), "chunk": _log(rng, 33, 4096)}[kind]
        c["ctx_hi"] = _log(rng, 16, 131072)
        c["causal"] = 0 if rng.random() < 0.1 else 1
        if c["causal"] and rng.random() < 0.4:
            c["window"], c["sinks"] = _log(rng, 16, 8192), rng.choice([0, 1, 4, 64, 200])
        # no more than the largest listed case's scores, and padded keys of 8 GB in 32 bits
        while c["batch"] > 1 and (c["batch"] * hq * c["rows_hi"] * (c["ctx_hi"] + c["rows_hi"]) > 64 * 4096 * 32768 or
                                  c["batch"] * hkv * d * (c["ctx_hi"] + c["rows_hi"]) > 2 ** 31):
            c["batch"] = max(1, c["batch"] // 2)
        while hq * c["rows_hi"] * (c["ctx_hi"] + c["rows_hi"]) > 64 * 4096 * 32768:
            c["ctx_hi"] //= 2
    else:
        c["rows_hi"] = _log(rng, 1, 131072)
        c["ctx_hi"] = _log(rng, 1, 4096)
        while c["batch"] > 1 and c["batch"] * c["rows_hi"] * hkv * d > 131072 * 8 * 128:
            c["batch"] = max(1, c["batch"] // 2)
        while c["rows_hi"] * hkv * d > 131072 * 8 * 128:
            c["rows_hi"] //= 2
    c["rows_lo"] = rng.choice([1, c["rows_hi"], (c["rows_hi"] + 1) // 2])
    c["ctx_lo"] = rng.choice([0, c["ctx_hi"], c["ctx_hi"] // 2])
    return c


def _lengths(case):
    """(rows, total length) of every sequence: a function of the case alone, so that work() knows them."""
    r = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    rows = [r.randint(case["rows_lo"], case["rows_hi"]) for _ in range(case["batch"])]
    # the spread of a serving batch: lengths over the whole range, one at its end
    ctx = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["batch"])]
    rows[-1], ctx[-1] = case["rows_hi"], case["ctx_hi"]
    return rows, [a + b for a, b in zip(rows, ctx)]


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    rows, lens = _lengths(case)
    B, P, Hq, Hkv, d = case["batch"], case["page"], case["hq"], case["hkv"], case["d"]
    pages = [-(-n // P) for n in lens]
    n_pages = sum(pages) + 3
    order = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    # pages of sequence b: the next ones of a random order; entries behind its last page are not valid pages
    first = torch.tensor([0] + pages[:-1], device=dev).cumsum(0)
    slot = torch.arange(max(pages), device=dev)
    used = slot[None] < torch.tensor(pages, device=dev)[:, None]
    table = torch.where(used, order[(first[:, None] + slot[None]).clamp(max=n_pages - 1)], torch.full_like(order[:1], -1))
    total = sum(rows)
    s = dict(case=case, max_q=max(rows), block_table=table.to(torch.int32).contiguous(),
             cu=torch.tensor([0] + rows, device=dev).cumsum(0).to(torch.int32),
             kv_len=torch.tensor(lens, device=dev, dtype=torch.int32))
    shape = (n_pages, Hkv, P, d)
    e4m3 = case["dtype"] == "e4m3"
    s["k_scale"] = s["v_scale"] = None
    if case["op"] == "append":
        for n in "kv":
            s[n + "_cache"] = torch.zeros(shape, dtype=torch.float8_e4m3fn if e4m3 else torch.bfloat16, device=dev)
            if e4m3:
                s[n + "_scale"] = torch.zeros(shape[:3], device=dev)
    else:
        for n in "kv":
            x = torch.empty(shape, dtype=torch.bfloat16, device=dev).normal_(generator=g)
            if e4m3:
                s[n + "_scale"] = torch.exp2(torch.randint(-9, -5, shape[:3], generator=g, device=dev).float())
                x.mul_(40.0)
                s[n + "_cache"] = x.to(torch.float8_e4m3fn)
            else:
                s[n + "_cache"] = x
    if case["op"] == "append":
        if case["fused"]:  # one projection's output, [total, (Hq + 2 Hkv) d]
            qkv = torch.empty((total, Hq + 2 * Hkv, d), dtype=torch.bfloat16, device=dev).normal_(generator=g)
            s["k_new"], s["v_new"] = qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        else:
            s["k_new"], s["v_new"] = (torch.empty((total, Hkv, d), dtype=torch.bfloat16, device=dev).normal_(generator=g)
                                      for _ in range(2))
    elif case["op"] == "read":
        s["k_out"], s["v_out"] = (torch.empty((Hkv, total, d), dtype=torch.bfloat16, device=dev) for _ in range(2))
    else:
        q = torch.empty((total, Hq + 2 * Hkv if case["fused"] else Hq, d), dtype=torch.bfloat16, device=dev)
        q = q.normal_(std=d ** -0.5, generator=g)[:, :Hq]
        s["q"] = q
        s["out"] = torch.empty((total, Hq, d), dtype=torch.bfloat16, device=dev)
        s["lse"] = torch.empty((total, Hq), device=dev)
    return s


# ------------------------------------------------------------------ plain forms
def _places(s):
    """Of every row: its sequence, its position, and the page and the row in the page that hold it."""
    cu, n = s["cu"].long(), s["kv_len"].long()
    rows = cu[1:] - cu[:-1]
    seq = torch.repeat_interleave(torch.arange(len(n), device=n.device), rows)
    pos = torch.arange(len(seq), device=n.device) - cu[seq] + (n - rows)[seq]
    P = s["case"]["page"]
    return seq, pos, s["block_table"][seq, pos // P].long(), pos % P


def _quantise(x):
    """bf16 rows -> (e4m3 codes, fp32 scales): the smallest power of two that brings the row's largest to 448."""
    m, e = torch.frexp(x.float().abs().amax(-1))
    e = (torch.where(m <= 0.875, e - 9, e - 8)).clamp(min=MIN_EXP)
    return (x.float() * torch.ldexp(torch.ones_like(m), -e)[..., None]).to(torch.float8_e4m3fn), torch.ldexp(torch.ones_like(m), e)


def _plain_append(s):
    _, _, page, row = _places(s)
    if s["case"]["dtype"] == "e4m3":
        (k, ks), (v, vs) = _quantise(s["k_new"]), _quantise(s["v_new"])
        s["k_cache"].view(torch.uint8)[page, :, row] = k.view(torch.uint8)
        s["v_cache"].view(torch.uint8)[page, :, row] = v.view(torch.uint8)
        s["k_scale"][page, :, row], s["v_scale"][page, :, row] = ks, vs
    else:
        s["k_cache"][page, :, row], s["v_cache"][page, :, row] = s["k_new"], s["v_new"]


def _fetch(s, n, page, row):
    """The cache's rows at these places in 32 bits, [..., Hkv, d]."""
    if s["case"]["dtype"] == "e4m3":
        x = s[n + "_cache"].view(torch.uint8)[page, :, row].view(torch.float8_e4m3fn).float()
        return x.mul_(s[n + "_scale"][page, :, row][..., None])
    return s[n + "_cache"][page, :, row].float()


def _plain_read(s):
    _, _, page, row = _places(s)
    s["k_out"].copy_(_fetch(s, "k", page, row).transpose(0, 1))
    s["v_out"].copy_(_fetch(s, "v", page, row).transpose(0, 1))


def _plain_attend(s):
    c = s["case"]
    P, Hkv, d = c["page"], c["hkv"], c["d"]
    g = c["hq"] // Hkv
    cu, n = s["cu"].long(), s["kv_len"].long()
    rows = cu[1:] - cu[:-1]
    T, L = s["max_q"], s["block_table"].shape[1] * P
    # the sequences padded to the longest, [B, Hkv, L, d] in 32 bits
    at = torch.arange(L, device=n.device)
    page = s["block_table"].long()[:, at // P].clamp(min=0)
    row = (at % P).expand_as(page)
    k = _fetch(s, "k", page, row).transpose(1, 2)
    t = torch.arange(T, device=n.device)
    src = (cu[:-1, None] + t).clamp(max=len(s["q"]) - 1)
    q = s["q"][src].float().view(len(n), T, Hkv, g, d).permute(0, 2, 1, 3, 4).reshape(len(n), Hkv, T * g, d)
    x = (q @ k.transpose(2, 3)).view(len(n), Hkv, T, g, L)
    del k
    i = (n - rows)[:, None] + t
    seen = (at < n[:, None]).expand(len(n), L)[:, None].expand(-1, T, -1)
    if c["causal"]:
        seen = seen & (at <= i[:, :, None])
    if c["window"]:
        seen = seen & ((at > i[:, :, None] - c["window"]) | (at < c["sinks"]))
    x.masked_fill_(~seen[:, None, :, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    x.sub_(top).exp_()
    z = x.sum(-1, keepdim=True)
    v = _fetch(s, "v", page, row).transpose(1, 2)
    o = (x.view(len(n), Hkv, T * g, L) @ v).view(len(n), Hkv, T, g, d).div_(z)
    lse = (top + z.log())[..., 0]
    mine = t < rows[:, None]
    s["out"].copy_(o.permute(0, 2, 1, 3, 4).reshape(len(n), T, c["hq"], d)[mine])
    s["lse"].copy_(lse.permute(0, 2, 1, 3).reshape(len(n), T, c["hq"])[mine])


def run(state):
    s, c = state, state["case"]
    if own:
        from online_softmax_attention_zigzag_gb300 import ringattn as ra
        kw = dict(k_scale=s["k_scale"], v_scale=s["v_scale"])
        if c["op"] == "append":
            ra.cache_append(s["k_new"], s["v_new"], s["k_cache"], s["v_cache"], s["block_table"], s["cu"], s["kv_len"], **kw)
        elif c["op"] == "read":
            ra.cache_read(s["k_cache"], s["v_cache"], s["k_out"], s["v_out"], s["block_table"], s["cu"], s["kv_len"], **kw)
        else:
            if "workspace" not in s:  # scratch that a program allocates once and keeps
                n = ra.paged_workspace_bytes(len(s["q"]), c["batch"], c["hq"], c["hkv"], c["d"], s["max_q"])
                s["workspace"] = torch.empty(n, dtype=torch.uint8, device=s["q"].device)
            ra.fwd_paged(s["q"], s["k_cache"], s["v_cache"], s["out"], s["lse"], s["block_table"], s["cu"], s["kv_len"],
                         s["workspace"], max_q=s["max_q"], causal=c["causal"], window=c["window"], sinks=c["sinks"], **kw)
    elif c["op"] == "append":
        _plain_append(s)
    elif c["op"] == "read":
        _plain_read(s)
    else:
        _plain_attend(s)
    if c["op"] == "append":
        out = {"k": s["k_cache"], "v": s["v_cache"]}
        return out if c["dtype"] == "bf16" else out | {"k_scale": s["k_scale"], "v_scale": s["v_scale"]}
    if c["op"] == "read":
        return {"k": s["k_out"], "v": s["v_out"]}
    return {"out": s["out"], "lse": s["lse"]}


# ------------------------------------------------------------------ what a pass cannot do without
def _seen(case, rows, length):
    """(keys that some row sees, visible pairs) of one sequence."""
    base, W, sinks = length - rows, case["window"], case["sinks"]
    if not case["causal"]:
        return length, rows * length
    if not W:
        return length, rows * base + rows * (rows + 1) // 2
    pairs = 0
    for i in range(base, length):
        lo = max(0, i - W + 1)
        pairs += i + 1 - lo + min(sinks, lo)
    lo = max(0, base - W + 1)
    return length - lo + min(sinks, lo), pairs


def work(case):
    rows, lens = _lengths(case)
    Hq, Hkv, d = case["hq"], case["hkv"], case["d"]
    kept = 2 * Hkv * (d + 4 if case["dtype"] == "e4m3" else 2 * d)  # bytes of one position's K and V in the cache
    total = sum(rows)
    if case["op"] != "attend":
        return {"bytes": total * (kept + 4 * Hkv * d), "flops": 0}
    keys, pairs = (sum(x) for x in zip(*(_seen(case, r, n) for r, n in zip(rows, lens))))
    return {"bytes": keys * kept + total * Hq * (4 * d + 4), "flops": 4.0 * pairs * Hq * d}


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    rows, lens = _lengths(case)
    P, Hq, Hkv, d = case["page"], case["hq"], case["hkv"], case["d"]
    table, e4m3 = s["block_table"].cpu(), case["dtype"] == "e4m3"
    if case["op"] == "append":
        pool = {n: s[n + "_cache"].double() for n in "kv"}
        scale = {n: s[n + "_scale"].double() for n in "kv"} if e4m3 else None
        for n in "kv":
            x = s[n + "_new"].double()
            if e4m3:
                # a power of two 2^e with amax <= 448 2^e < 2 amax; values to the nearest of 4 significant bits, the
                # even one in the middle, in steps of 2^-9 at least
                top = x.abs().amax(-1)
                e = torch.ceil(torch.log2(top / E4M3_MAX)).clamp(min=MIN_EXP)
                x = x / torch.exp2(e)[..., None]
                step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
                x = torch.round(x / step) * step
            at = 0
            for b, (r, length) in enumerate(zip(rows, lens)):
                pos = torch.arange(length - r, length)
                page = table[b, pos // P].long().to(x.device)
                row = (pos % P).to(x.device)
                pool[n][page, :, row] = x[at:at + r]
                if e4m3:
                    scale[n][page, :, row] = torch.exp2(e[at:at + r])
                at += r
        out = {"k": pool["k"], "v": pool["v"]}
        return out | {"k_scale": scale["k"], "v_scale": scale["v"]} if e4m3 else out

    def sequence(n, b, lo, hi):
        """Positions [lo, hi) of sequence b, [Hkv, hi - lo, d]."""
        pg = table[b, lo // P:-(-hi // P)].long().to(s["cu"].device)
        x = s[n + "_cache"].view(torch.uint8)[pg].view(torch.float8_e4m3fn).double() if e4m3 else s[n + "_cache"][pg].double()
        if e4m3:
            x = x * s[n + "_scale"][pg].double()[..., None]
        x = x.transpose(0, 1).reshape(Hkv, -1, d)
        return x[:, lo - lo // P * P:][:, :hi - lo]

    if case["op"] == "read":
        return {n: torch.cat([sequence(n, b, length - r, length) for b, (r, length) in enumerate(zip(rows, lens))], 1) for n in "kv"}
    if 4.0 * Hq * d * sum(r * n for r, n in zip(rows, lens)) > 1e13:
        return None
    out = torch.empty((len(s["q"]), Hq, d), dtype=torch.float64, device=s["q"].device)
    lse = torch.empty((len(s["q"]), Hq), dtype=torch.float64, device=s["q"].device)
    at = 0
    for b, (r, length) in enumerate(zip(rows, lens)):
        k, v = sequence("k", b, 0, length), sequence("v", b, 0, length)
        j = torch.arange(length, device=k.device)
        i = torch.arange(length - r, length, device=k.device)[:, None]
        dead = torch.zeros((r, length), dtype=torch.bool, device=k.device)
        if case["causal"]:
            dead |= j > i
        if case["window"]:
            dead |= (j <= i - case["window"]) & (j >= case["sinks"])
        for h in range(Hq):
            x = s["q"][at:at + r, h].double() @ k[h // (Hq // Hkv)].T
            x[dead] = -math.inf
            lse[at:at + r, h] = torch.logsumexp(x, 1)
            out[at:at + r, h] = torch.exp(x - lse[at:at + r, h, None]) @ v[h // (Hq // Hkv)]
        at += r
    return {"out": out, "lse": lse}
