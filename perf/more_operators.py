"""Measured cases of what stands around attention: the norm and rotation of q and k before it, with their
gradients, and the eviction of a paged cache's positions by the attention weight they have had.

* ``norm``:     q [total, Hq, d] and k [total, Hkv, d], bf16, each row x (one token and head) to
                rotate(w * x / sqrt(mean(x^2) + eps)), q's times ``q_scale``; w [d] of q and of k, or none.  Pairs
                (j, j + rot / 2), or (2 j, 2 j + 1) when interleaved, are turned by the angle whose cosine and sine are
                ``cos_sin[position, j]`` and ``cos_sin[position, rot / 2 + j]``; elements from rot on are not turned.
* ``norm_bwd``: gradients with respect to q, k and both w, given those of the results.
* ``weights``:  [n_pages, Hkv, page_size] fp32, one a cached position and KV head: decay * its value (0 for the batch's
                own rows' positions) + the sum over the batch's rows that see it, and the query heads of the KV head, of
                exp(q.k - lse).
* ``evict``:    of every sequence's positions keep[b] stay, for every KV head: the first ``sinks``, the last ``recent``,
                then those of the largest weight (of equal ones the lowest position).  They move to the front, in
                order, with K, V, scales and weights; ``kept`` [B, Hkv, max_keep] says which ones (-1 behind them).

The cache: ``k_cache``, ``v_cache`` [n_pages, Hkv, page_size, d], bf16 or e4m3 with fp32 scales a row;
``block_table`` [B, max_pages], ``cu`` [B + 1] and ``kv_len`` [B] int32; row t of sequence b is position
kv_len[b] - (cu[b + 1] - cu[b]) + t and sees j <= its own position, with a window W only j > i - W or j < sinks.
"""
from __future__ import annotations

import math
import random

import torch

own = False

EPS = 1e-6


# ------------------------------------------------------------------ cases
def _norm(op, name=None, **kw):
    c = dict(op=op, total=1, hq=64, hkv=8, d=128, rot=128, interleaved=0, fused=True, head_major=False, far=1 << 15, w="bf16",
             grad="fp32")
    c.update(kw)
    if name:
        c["name"] = name
    return c


def _cache(op, name=None, **kw):
    c = dict(op=op, batch=1, rows_lo=1, rows_hi=1, ctx_lo=0, ctx_hi=0, hq=64, hkv=8, d=128, page=64, dtype="bf16", window=0,
             sinks=0, decay=1.0, keep=0, recent=0)
    c.update(kw)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one decoding step of 64 sequences, far into their contexts: latency
        _norm("norm", "norm_decode_b64", total=64, far=1 << 17),
        # a whole 32k prompt out of a fused projection, head-major for the ring
        _norm("norm", "norm_prompt_32k", total=32768, head_major=True),
        # packed prompts of a small model: half of a head turned, neighbours as pairs, odd number of tokens
        _norm("norm", "norm_ragged_d64", total=4111, hq=6, hkv=2, d=64, rot=32, interleaved=1, w="fp32"),
        # training at 32k: the ring backward's fp32 gradients, head-major, into the fused projection's
        _norm("norm_bwd", "norm_bwd_32k", total=32768, head_major=True),
        # a short training sequence, gradients in bf16
        _norm("norm_bwd", "norm_bwd_ragged_d64", total=1021, hq=8, hkv=8, d=64, rot=64, interleaved=1, w="fp32", grad="bf16"),
        # one decoding step of a serving batch, lengths all over the range
        _cache("weights", "weights_decode_b64_16k", batch=64, ctx_lo=200, ctx_hi=16384),
        # few very long contexts in 8 bits: the cache's bytes are all there is
        _cache("weights", "weights_decode_e4m3_b8_128k", batch=8, ctx_lo=100000, ctx_hi=131071, hq=32, dtype="e4m3"),
        # a large chunk of a long prompt, whose rows alone weigh what is kept
        _cache("weights", "weights_chunk_4096_of_32k", rows_lo=4096, rows_hi=4096, ctx_lo=28672, ctx_hi=28672, decay=0.0),
        # chunks and single tokens in one batch, odd sizes and pages, 8 bits, a window, old weight fading
        _cache("weights", "weights_mixed_e4m3_b12", batch=12, rows_hi=1023, ctx_hi=9000, hq=32, page=48, dtype="e4m3",
               window=2500, sinks=17, decay=0.95),
        # a serving batch's contexts of up to 16k cut down to 2k
        _cache("evict", "evict_b16_16k_to_2k", batch=16, ctx_lo=4000, ctx_hi=16383, keep=2048, sinks=4, recent=256),
        # one very long prompt in 8 bits, an eighth of it kept
        _cache("evict", "evict_e4m3_128k_to_16k", ctx_lo=131071, ctx_hi=131071, hq=32, dtype="e4m3", keep=16384, recent=1024),
        # short conversations, small pages, some already short enough
        _cache("evict", "evict_small_d64", batch=5, ctx_lo=60, ctx_hi=700, hq=8, hkv=2, d=64, page=16, keep=250, sinks=1, recent=33),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "weights", "weights", "evict"])
    hq, hkv, d = rng.choice([(64, 8, 128), (32, 8, 128), (8, 2, 128), (8, 8, 64), (16, 16, 128), (6, 2, 64), (8, 1, 128)])
    if op in ("norm", "norm_bwd"):
        total = _log(rng, 1, 65536)
        total = min(total, 32768 * 72 * 128 // ((hq + hkv) * d))
        return _norm(op, total=total, hq=hq, hkv=hkv, d=d, rot=rng.choice([d, d, d // 2, 16]), interleaved=rng.choice([0, 1]),
                     fused=rng.random() < 0.6, head_major=rng.random() < 0.5, far=_log(rng, 128, 1 << 18),
                     w=rng.choice(["bf16", "fp32", "none"]), grad=rng.choice(["fp32", "bf16"]))
    c = _cache(op, hq=hq, hkv=hkv, d=d, page=rng.choice([16, 32, 48, 64, 128, 256]), dtype=rng.choice(["bf16", "e4m3"]),
               batch=_log(rng, 1, 128), ctx_hi=_log(rng, 16, 131072))
    if op == "weights":
        kind = rng.choice(["decode", "decode", "few", "chunk"])
        c["rows_hi"] = {"decode": 1, "few": _log(rng, 2, 32), "chunk": _log(rng, 33, 4096)}[kind]
        c["decay"] = rng.choice([0.0, 1.0, round(rng.uniform(0.5, 0.99), 2)])
        if rng.random() < 0.3:
            c["window"], c["sinks"] = _log(rng, 16, 8192), rng.choice([0, 1, 4, 64, 200])
    # no more than the largest listed case's scores, and padded keys of 8 GB in 32 bits
    while c["batch"] > 1 and (c["batch"] * hq * c["rows_hi"] * (c["ctx_hi"] + c["rows_hi"]) > 64 * 4096 * 32768 or
                              c["batch"] * hkv * d * (c["ctx_hi"] + c["rows_hi"]) > 2 ** 31):
        c["batch"] = max(1, c["batch"] // 2)
    while hq * c["rows_hi"] * (c["ctx_hi"] + c["rows_hi"]) > 64 * 4096 * 32768:
        c["ctx_hi"] //= 2
    c["rows_lo"] = rng.choice([1, c["rows_hi"], (c["rows_hi"] + 1) // 2])
    c["ctx_lo"] = rng.choice([0, c["ctx_hi"], c["ctx_hi"] // 2])
    if op == "evict":
        c["keep"] = max(1, min(_log(rng, 8, 32768), c["ctx_hi"] * rng.randint(1, 9) // 10))
        c["sinks"] = rng.randint(0, min(8, c["keep"] // 4))
        c["recent"] = rng.randint(0, c["keep"] // 2)
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
def _prepare_norm(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    T, Hq, Hkv, d, rot = case["total"], case["hq"], case["hkv"], case["d"], case["rot"]
    s = dict(case=case, q_scale=d ** -0.5)
    # the table of a model, made once in 64 bits; positions of a packed batch: runs that start anywhere below `far`
    n = case["far"]
    angle = torch.arange(n, device=dev, dtype=torch.float64)[:, None] * 1e4 ** (-torch.arange(0, rot, 2, device=dev).double() / rot)
    s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
    run = max(1, T // 7)
    start = torch.randint(0, n, (T // run + 1,), generator=g, device=dev)
    at = torch.arange(T, device=dev)
    s["position"] = ((start[at // run] + at % run) % n).to(torch.int32)
    for name, h, ch in (("q", Hq, 0), ("k", Hkv, Hq)):
        if case["fused"]:  # one projection's output, [total, (Hq + 2 Hkv), d]
            if "qkv" not in s:
                s["qkv"] = torch.empty((T, Hq + 2 * Hkv, d), dtype=torch.bfloat16, device=dev).normal_(generator=g)
            s[name] = s["qkv"][:, ch:ch + h]
        else:
            s[name] = torch.empty((T, h, d), dtype=torch.bfloat16, device=dev).normal_(generator=g)
        s[name + "_weight"] = None
        if case["w"] != "none":
            w = torch.empty(d, device=dev).normal_(1.0, 0.2, generator=g)
            s[name + "_weight"] = w.to(torch.bfloat16) if case["w"] == "bf16" else w

        def rows(dtype):
            x = torch.empty((h, T, d) if case["head_major"] else (T, h, d), dtype=dtype, device=dev)
            return x.transpose(0, 1) if case["head_major"] else x

        if case["op"] == "norm":
            s[name + "_out"] = rows(torch.bfloat16)
        else:
            s["d" + name + "_out"] = rows(torch.float32 if case["grad"] == "fp32" else torch.bfloat16).normal_(generator=g)
            s["d" + name + "_weight"] = None if case["w"] == "none" else torch.empty(d, device=dev)
    if case["op"] == "norm_bwd":
        dqkv = torch.empty((T, Hq + 2 * Hkv, d), dtype=torch.bfloat16, device=dev)
        s["dq"], s["dk"] = (dqkv[:, :Hq], dqkv[:, Hq:Hq + Hkv]) if case["fused"] else (torch.empty_like(s["q"]), torch.empty_like(s["k"]))
    return s


def prepare(case, seed):
    if case["op"] in ("norm", "norm_bwd"):
        return _prepare_norm(case, seed)
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
    for n in "kv":
        x = torch.empty(shape, dtype=torch.bfloat16, device=dev).normal_(generator=g)
        if e4m3:
            s[n + "_scale"] = torch.exp2(torch.randint(-9, -5, shape[:3], generator=g, device=dev).float())
            x.mul_(40.0)
            s[n + "_cache"] = x.to(torch.float8_e4m3fn)
        else:
            s[n + "_cache"] = x
        del x
    # what earlier steps left: most positions near nothing, a few with much, some with nothing at all
    w = torch.empty(shape[:3], device=dev).normal_(-4.0, 2.0, generator=g).exp_()
    s["weights"] = w.mul_(torch.empty_like(w).uniform_(generator=g) > 0.1)
    if case["op"] == "evict":
        s["keep"] = torch.full((B,), case["keep"], dtype=torch.int32, device=dev)
        s["kept"] = torch.empty((B, Hkv, case["keep"]), dtype=torch.int32, device=dev)
        s["new_len"] = torch.empty(B, dtype=torch.int32, device=dev)
        return s
    s["q"] = torch.empty((total, Hq, d), dtype=torch.bfloat16, device=dev).normal_(std=d ** -0.5, generator=g)
    # lse as attention leaves it for such q and k: log of the keys a row sees, and half the scores' variance
    i = torch.cat([torch.arange(n - r, n, device=dev) for r, n in zip(rows, lens)]).double()
    seen = i + 1
    if case["window"]:
        seen = torch.minimum(seen, torch.full_like(seen, case["window"] + case["sinks"]))
    noise = torch.empty((total, Hq), device=dev).normal_(std=0.05, generator=g)
    s["lse"] = seen.log().float()[:, None] + (0.05 if e4m3 else 0.5) + noise
    return s


# ------------------------------------------------------------------ plain forms
def _pairs(x, case):
    """The two elements of every pair that is turned, and the rest."""
    rot = case["rot"]
    y, rest = x[..., :rot], x[..., rot:]
    return (y[..., 0::2], y[..., 1::2], rest) if case["interleaved"] else (y[..., :rot // 2], y[..., rot // 2:], rest)


def _unpair(a, b, rest, case):
    y = torch.stack([a, b], -1).flatten(-2) if case["interleaved"] else torch.cat([a, b], -1)
    return torch.cat([y, rest], -1)


def _plain_norm(s, name, scale):
    c = s["case"]
    x = s[name].float()
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    if s[name + "_weight"] is not None:
        y = y * s[name + "_weight"].float()
    a, b, rest = _pairs(y * scale, c)
    cos, sin = s["cos_sin"][s["position"].long()][:, None].chunk(2, -1)
    s[name + "_out"].copy_(_unpair(a * cos - b * sin, b * cos + a * sin, rest, c))


def _plain_norm_bwd(s, name, scale):
    c = s["case"]
    a, b, rest = _pairs(s["d" + name + "_out"].float() * scale, c)
    cos, sin = s["cos_sin"][s["position"].long()][:, None].chunk(2, -1)
    u = _unpair(a * cos + b * sin, b * cos - a * sin, rest, c)
    x = s[name].float()
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    n = x * r
    if s[name + "_weight"] is not None:
        s["d" + name + "_weight"].copy_((u * n).flatten(0, 1).sum(0))
        u = u * s[name + "_weight"].float()
    s["d" + name].copy_(r * (u - n * (u * n).mean(-1, keepdim=True)))


def _all_places(s):
    """Pages and rows of every sequence's positions, padded to the longest, [B, L], and which are positions."""
    P = s["case"]["page"]
    at = torch.arange(s["block_table"].shape[1] * P, device=s["kv_len"].device)
    page = s["block_table"].long()[:, at // P].clamp(min=0)
    return at, page, (at % P).expand_as(page), at < s["kv_len"].long()[:, None]


def _plain_weights(s):
    c = s["case"]
    Hkv, d = c["hkv"], c["d"]
    g = c["hq"] // Hkv
    cu, n = s["cu"].long(), s["kv_len"].long()
    rows = cu[1:] - cu[:-1]
    T = s["max_q"]
    at, page, row, mine = _all_places(s)
    L = len(at)
    if c["dtype"] == "e4m3":
        k = s["k_cache"].view(torch.uint8)[page, :, row].view(torch.float8_e4m3fn).float()
        k = k.mul_(s["k_scale"][page, :, row][..., None]).transpose(1, 2)
    else:
        k = s["k_cache"][page, :, row].float().transpose(1, 2)
    t = torch.arange(T, device=n.device)
    src = (cu[:-1, None] + t).clamp(max=len(s["q"]) - 1)
    q = s["q"][src].float().view(len(n), T, Hkv, g, d).permute(0, 2, 1, 3, 4).reshape(len(n), Hkv, T * g, d)
    lse = s["lse"][src].view(len(n), T, Hkv, g).permute(0, 2, 1, 3).reshape(len(n), Hkv, T * g, 1)
    x = q @ k.transpose(2, 3)
    del k
    x.sub_(lse).exp_()
    i = (n - rows)[:, None] + t
    seen = mine[:, None] & (at <= i[:, :, None]) & (t < rows[:, None])[:, :, None]
    if c["window"]:
        seen = seen & ((at > i[:, :, None] - c["window"]) | (at < c["sinks"]))
    add = x.view(len(n), Hkv, T, g, L).masked_fill_(~seen[:, None, :, None], 0.0).sum((2, 3))
    old = s["weights"][page, :, row].transpose(1, 2) * c["decay"]
    new = torch.where(at < (n - rows)[:, None, None], old, torch.zeros_like(old)) + add
    s["weights"][page[mine], :, row[mine]] = new.transpose(1, 2)[mine]


def _plain_evict(s):
    c = s["case"]
    n, keep = s["kv_len"].long(), s["keep"].long()
    at, page, row, mine = _all_places(s)
    forced = mine & ((at < c["sinks"]) | (at >= n[:, None] - c["recent"]))
    w = s["weights"][page, :, row].transpose(1, 2).masked_fill(forced[:, None], math.inf).masked_fill(~mine[:, None], -math.inf)
    order = torch.sort(w, dim=-1, descending=True, stable=True)[1]
    rank = torch.empty_like(order).scatter_(2, order, at.expand_as(order).contiguous())
    stay = mine[:, None] & (rank < keep[:, None, None])
    b, h, j = stay.nonzero(as_tuple=True)
    to = (stay.cumsum(-1) - 1)[b, h, j]
    s["kept"].fill_(-1)
    s["kept"][b, h, to] = j.to(torch.int32)
    frm, dst = (page[b, j], h, row[b, j]), (page[b, to], h, row[b, to])
    for name in ("k_cache", "v_cache", "k_scale", "v_scale", "weights"):
        x = s[name]
        if x is not None:
            x = x.view(torch.uint8) if name.endswith("cache") and c["dtype"] == "e4m3" else x
            x[dst] = x[frm]
    s["new_len"].copy_(torch.minimum(n, keep))


def run(state):
    s, c = state, state["case"]
    kw = dict(k_scale=s["k_scale"], v_scale=s["v_scale"]) if "k_scale" in s else {}
    if own:
        from online_softmax_attention_zigzag_gb300 import ringattn as ra
        if c["op"] == "norm":
            ra.qk_norm_rope(s["q"], s["k"], s["q_out"], s["k_out"], s["position"], s["cos_sin"], q_weight=s["q_weight"],
                            k_weight=s["k_weight"], eps=EPS, q_scale=s["q_scale"], interleaved=c["interleaved"])
        elif c["op"] == "norm_bwd":
            if "workspace" not in s:  # scratch that a program allocates once and keeps
                nbytes = ra.qk_norm_rope_workspace_bytes(c["total"], c["hq"], c["hkv"], c["d"])
                s["workspace"] = torch.empty(nbytes, dtype=torch.uint8, device=s["q"].device)
            ra.qk_norm_rope_bwd(s["q"], s["k"], s["dq_out"], s["dk_out"], s["dq"], s["dk"], s["position"], s["cos_sin"],
                                s["workspace"], q_weight=s["q_weight"], k_weight=s["k_weight"], dq_weight=s["dq_weight"],
                                dk_weight=s["dk_weight"], eps=EPS, q_scale=s["q_scale"], interleaved=c["interleaved"])
        elif c["op"] == "weights":
            if "workspace" not in s:  # the one that attention over the same rows takes
                nbytes = ra.paged_workspace_bytes(len(s["q"]), c["batch"], c["hq"], c["hkv"], c["d"], s["max_q"])
                s["workspace"] = torch.empty(nbytes, dtype=torch.uint8, device=s["q"].device)
            ra.cache_weights(s["q"], s["lse"], s["k_cache"], s["v_cache"], s["weights"], s["block_table"], s["cu"], s["kv_len"],
                             s["workspace"], max_q=s["max_q"], decay=c["decay"], window=c["window"], sinks=c["sinks"], **kw)
        else:
            ra.cache_evict(s["k_cache"], s["v_cache"], s["weights"], s["block_table"], s["kv_len"], s["keep"], s["new_len"],
                           s["kept"], sinks=c["sinks"], recent=c["recent"], **kw)
    elif c["op"] == "norm":
        _plain_norm(s, "q", s["q_scale"])
        _plain_norm(s, "k", 1.0)
    elif c["op"] == "norm_bwd":
        _plain_norm_bwd(s, "q", s["q_scale"])
        _plain_norm_bwd(s, "k", 1.0)
    elif c["op"] == "weights":
        _plain_weights(s)
    else:
        _plain_evict(s)
    if c["op"] == "norm":
        return {"q": s["q_out"], "k": s["k_out"]}
    if c["op"] == "norm_bwd":
        return {n: s[n] for n in ("dq", "dk", "dq_weight", "dk_weight")}
    if c["op"] == "weights":
        return {"weights": s["weights"]}
    return {n: s[n] for n in ("k_cache", "v_cache", "k_scale", "v_scale", "weights", "kept", "new_len")}


# ------------------------------------------------------------------ what a pass cannot do without
def _seen(case, rows, length):
    """(keys that some row sees, visible pairs) of one sequence."""
    base, W, sinks = length - rows, case["window"], case["sinks"]
    if not W:
        return length, rows * base + rows * (rows + 1) // 2
    pairs = 0
    for i in range(base, length):
        lo = max(0, i - W + 1)
        pairs += i + 1 - lo + min(sinks, lo)
    lo = max(0, base - W + 1)
    return length - lo + min(sinks, lo), pairs


def work(case):
    Hq, Hkv, d = case["hq"], case["hkv"], case["d"]
    if case["op"] in ("norm", "norm_bwd"):
        # a position's row of the table is read once however many tokens have it
        per = 4 if case["op"] == "norm" else 4 + (4 if case["grad"] == "fp32" else 2)
        return {"bytes": case["total"] * ((Hq + Hkv) * d * per + 4) + min(case["total"], case["far"]) * case["rot"] * 4, "flops": 0}
    rows, lens = _lengths(case)
    kept = d + 4 if case["dtype"] == "e4m3" else 2 * d  # bytes of one position's K or V of one head
    if case["op"] == "evict":
        n = sum(min(x, case["keep"]) for x in lens)
        moved = sum(case["keep"] for x in lens if x > case["keep"])
        return {"bytes": Hkv * (4 * sum(lens) + 4 * n + moved * (4 * kept + 8)), "flops": 0}
    keys, pairs = (sum(x) for x in zip(*(_seen(case, r, n) for r, n in zip(rows, lens))))
    # every weight is written, and read unless nothing of it stays; with decay 1 those that nobody sees stay as they are
    touched = keys if case["decay"] == 1.0 else sum(lens)
    return {"bytes": Hkv * (keys * kept + touched * (8 if case["decay"] else 4)) + sum(rows) * Hq * (2 * d + 4),
            "flops": 2.0 * pairs * Hq * d}


# ------------------------------------------------------------------ the definition in 64 bits
def _exact_norm(case, seed):
    s = prepare(case, seed)
    c, rot = s["case"], case["rot"]
    table = s["cos_sin"][s["position"].long()].double()
    turn = torch.complex(table[:, :rot // 2].contiguous(), table[:, rot // 2:].contiguous())[:, None]

    def forward(x, w, scale):
        y = x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS)
        y = y * w if w is not None else y
        if c["interleaved"]:
            z = torch.view_as_complex(y[..., :rot].reshape(*y.shape[:2], rot // 2, 2).contiguous()) * turn
            turned = torch.view_as_real(z).flatten(2)
        else:
            z = torch.complex(y[..., :rot // 2].contiguous(), y[..., rot // 2:rot].contiguous()) * turn
            turned = torch.cat([z.real, z.imag], -1)
        return torch.cat([turned, y[..., rot:]], -1) * scale

    out = {}
    for name, scale in (("q", s["q_scale"]), ("k", 1.0)):
        x, w = s[name].double(), s[name + "_weight"]
        w = None if w is None else w.double()
        if c["op"] == "norm":
            out[name] = forward(x, w, scale)
            continue
        x.requires_grad_()
        if w is not None:
            w.requires_grad_()
        y = forward(x, w, scale)
        got = torch.autograd.grad(y, [x] + ([w] if w is not None else []), s["d" + name + "_out"].double())
        out["d" + name], out["d" + name + "_weight"] = got[0], got[1] if w is not None else None
    return out


def exact(case, seed):
    if case["op"] in ("norm", "norm_bwd"):
        return _exact_norm(case, seed)
    s = prepare(case, seed)
    rows, lens = _lengths(case)
    P, Hq, Hkv, d = case["page"], case["hq"], case["hkv"], case["d"]
    table, e4m3 = s["block_table"].cpu(), case["dtype"] == "e4m3"
    dev = s["kv_len"].device

    def places(b, length):
        pos = torch.arange(length)
        return table[b, pos // P].long().to(dev), (pos % P).to(dev)

    if case["op"] == "evict":
        # one head after the other, on the host: the positions by (forced first, weight, position)
        names = [n for n in ("k_cache", "v_cache", "k_scale", "v_scale", "weights") if s[n] is not None]
        new = {n: s[n].view(torch.uint8).clone() if e4m3 and n.endswith("cache") else s[n].clone() for n in names}
        old = {n: x.clone() for n, x in new.items()}
        kept = torch.full((case["batch"], Hkv, case["keep"]), -1, dtype=torch.int32)
        for b, length in enumerate(lens):
            page, row = places(b, length)
            w = s["weights"][page, :, row].double().cpu().numpy()
            m = min(length, case["keep"])
            for h in range(Hkv):
                x = w[:, h].copy()
                x[:case["sinks"]] = math.inf
                if case["recent"]:
                    x[max(0, length - case["recent"]):] = math.inf
                chosen = sorted((-x).argsort(kind="stable")[:m].tolist())
                kept[b, h, :m] = torch.tensor(chosen, dtype=torch.int32)
                j = torch.tensor(chosen, device=dev)
                for n in names:
                    new[n][page[:m], h, row[:m]] = old[n][page[j], h, row[j]]
        out = {n: (x.view(torch.float8_e4m3fn) if x.dtype == torch.uint8 else x).double() for n, x in new.items()}
        out.update(kept=kept, new_len=torch.tensor([min(x, case["keep"]) for x in lens], dtype=torch.int32))
        return {n: out.get(n) for n in ("k_cache", "v_cache", "k_scale", "v_scale", "weights", "kept", "new_len")}
    if 2.0 * Hq * d * sum(r * n for r, n in zip(rows, lens)) > 1e13:
        return None
    out = s["weights"].double()
    at, g = 0, Hq // Hkv
    for b, (r, length) in enumerate(zip(rows, lens)):
        page, row = places(b, length)
        j = torch.arange(length, device=dev)
        i = torch.arange(length - r, length, device=dev)[:, None]
        dead = j > i
        if case["window"]:
            dead = dead | ((j <= i - case["window"]) & (j >= case["sinks"]))
        for h in range(Hkv):
            k = s["k_cache"].view(torch.uint8)[page, h, row].view(torch.float8_e4m3fn).double() if e4m3 else s["k_cache"][page, h, row].double()
            if e4m3:
                k = k * s["k_scale"][page, h, row].double()[:, None]
            add = torch.zeros(length, dtype=torch.float64, device=dev)
            for x in range(h * g, (h + 1) * g):
                p = torch.exp(s["q"][at:at + r, x].double() @ k.T - s["lse"][at:at + r, x].double()[:, None])
                add += p.masked_fill_(dead, 0.0).sum(0)
            old = out[page, h, row] * case["decay"]
            old[length - r:] = 0.0
            out[page, h, row] = old + add
        at += r
    return {"weights": out}
