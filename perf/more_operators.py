"""Cases of a longer context in the same memory: a K/V cache in 4 bits (``kv_append``, ``kv_read``, ``kv_attend``),
attention whose scores are capped, biased by distance or masked by document (``kv_attend``), the attention
weight that each cached token has collected (``kv_weigh``) and the eviction of the tokens that collected
least (``kv_evict``).

``run`` computes an operator in elementary torch operations in 32 bits where ``own`` is false, and
through the package's entry points where it is true.  Head counts 32 / 8 of 128 are the q/k/v
projections 4096 -> 4096 / 1024 / 1024 that the benchmark runs; the others are generic.
"""
import math
import random

import torch

own = False

_DEV = "cuda" if torch.cuda.is_available() else "cpu"
_BLOCK = 32  # elements of one scale

# what a case of attention or of collected weight has, where it says nothing else
_SCORES = {"order": "head", "window": 0, "cap": 0.0, "slopes": False, "starts": False, "moved": False}


def listed():
    heads = {"heads": 32, "kv": 8, "dim": 128}
    return [
        # a decode step of 64 sequences into a 4-bit cache
        {"name": "append_64_a4", "op": "append", "fmt": "a4", "n": 64, "kv": 8, "dim": 128, "page": 64, "order": "token", "fused": False},
        # a prompt chunk of odd length into a 4-bit cache, as columns of one q/k/v result
        {"name": "append_4097_a4", "op": "append", "fmt": "a4", "n": 4097, "kv": 8, "dim": 128, "page": 16, "order": "head", "fused": True},
        # one short chat over a 4-bit cache: latency
        {"name": "attend_1x512_a4", "op": "attend", "fmt": "a4", "n_seq": 1, **heads, **_SCORES, "page": 16, "min_len": 512, "max_len": 512, "lens": 1},
        # a batch of unlike lengths in a 4-bit cache
        {"name": "attend_64_ragged_a4", "op": "attend", "fmt": "a4", "n_seq": 64, **heads, **_SCORES, "page": 16, "min_len": 1, "max_len": 8192, "lens": 2},
        # one long document in a 4-bit cache: the split over the length
        {"name": "attend_1x131071_a4", "op": "attend", "fmt": "a4", "n_seq": 1, **heads, **_SCORES, "page": 64, "min_len": 131071, "max_len": 131071, "lens": 3},
        # layers whose logits are capped, wide heads, under a sliding window
        {"name": "attend_16_capped_bf16", "op": "attend", "fmt": "bf16", "n_seq": 16, "heads": 16, "kv": 8, "dim": 256, **_SCORES, "page": 32,
         "min_len": 1000, "max_len": 16384, "lens": 4, "window": 4096, "cap": 50.0},
        # a bias that grows with distance, over sequences that hold several documents (some slots idle, some documents just begun)
        {"name": "attend_32_bias_q8", "op": "attend", "fmt": "q8", "n_seq": 32, "heads": 32, "kv": 32, "dim": 128, **_SCORES, "page": 16,
         "min_len": 0, "max_len": 4096, "lens": 5, "slopes": True, "starts": True},
        # what one token's attention adds to a short chat's cached tokens: latency
        {"name": "weigh_1x2048_bf16", "op": "weigh", "fmt": "bf16", "n_seq": 1, **heads, **_SCORES, "page": 16, "min_len": 2048, "max_len": 2048, "lens": 6},
        # the same for a batch of unlike lengths in a 4-bit cache
        {"name": "weigh_64_ragged_a4", "op": "weigh", "fmt": "a4", "n_seq": 64, **heads, **_SCORES, "page": 16, "min_len": 1, "max_len": 8192, "lens": 7},
        # a decode step at a fixed cache size: one token of each sequence makes room for the new one
        {"name": "evict_64_step_bf16", "op": "evict", "fmt": "bf16", "n_seq": 64, "kv": 8, "dim": 128, "page": 16, "order": "head",
         "min_len": 1025, "max_len": 1025, "lens": 8, "keep": 1024, "first": 4, "recent": 256, "moved": True},
        # one long prompt cut to an eighth
        {"name": "evict_1x32768_bf16", "op": "evict", "fmt": "bf16", "n_seq": 1, "kv": 8, "dim": 128, "page": 64, "order": "head",
         "min_len": 32768, "max_len": 32768, "lens": 9, "keep": 4096, "first": 4, "recent": 64, "moved": False},
        # a batch of prompts of unlike lengths cut to a size; the shortest stay as they are
        {"name": "evict_32_prompts_q8", "op": "evict", "fmt": "q8", "n_seq": 32, "kv": 8, "dim": 128, "page": 16, "order": "token",
         "min_len": 500, "max_len": 8192, "lens": 10, "keep": 2048, "first": 4, "recent": 512, "moved": False},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "scores", "scores", "weigh", "weigh", "evict", "evict"])
    page = rng.choice([8, 16, 16, 24, 32, 64, 128])
    order, fmt = rng.choice(["head", "token"]), rng.choice(["bf16", "q8", "a4"])
    if op in ("append", "evict"):
        kv, dim = rng.choice([(8, 128), (8, 64), (4, 128), (1, 256), (2, 96), (12, 64)])
        if op == "append":
            return {"op": op, "fmt": "a4", "n": _log_int(rng, 1, 16384), "kv": kv, "dim": dim, "page": page, "order": order,
                    "fused": rng.random() < 0.5}
        longest = _log_int(rng, 16, 32768)
        keep = _log_int(rng, 8, longest)
        return {"op": op, "fmt": fmt, "n_seq": _log_int(rng, 1, max(1, min(128, (1 << 27) // (longest * kv * dim)))), "kv": kv, "dim": dim,
                "page": page, "order": order, "min_len": rng.choice([0, 1, (longest + 1) // 2]), "max_len": longest,
                "lens": rng.randrange(1 << 30), "keep": keep, "first": rng.choice([0, 1, 4]), "recent": rng.choice([0, 1, keep // 4, keep // 2]),
                "moved": rng.random() < 0.5}
    heads, kv, dim = rng.choice([(32, 8, 128), (32, 8, 128), (32, 4, 128), (16, 16, 64), (32, 8, 64), (8, 1, 256), (16, 8, 256),
                                 (14, 2, 64), (40, 8, 128), (24, 2, 96), (32, 2, 128)])
    longest = _log_int(rng, 1, 65536)
    most = 1 << (27 if op == "scores" else 28)  # elements of K; scores are drawn over wider formats too
    n_seq = _log_int(rng, 1, max(1, min(256, most // (longest * kv * dim))))
    case = {"op": "weigh" if op == "weigh" else "attend", "fmt": "a4" if op == "attend" else fmt, "n_seq": n_seq, "heads": heads, "kv": kv,
            "dim": dim, **_SCORES, "page": page, "min_len": rng.choice([0, 1, (longest + 1) // 2]), "max_len": longest,
            "lens": rng.randrange(1 << 30), "order": order, "window": rng.choice([0, 0, 0, _log_int(rng, 1, longest)])}
    if op == "scores" or (op == "weigh" and rng.random() < 0.4):
        kind = rng.choice(["cap", "slopes", "starts", "all"])
        case.update(cap=rng.choice([15.0, 30.0, 50.0]) if kind in ("cap", "all") else 0.0, slopes=kind in ("slopes", "all"),
                    starts=kind in ("starts", "all"), moved=kind in ("slopes", "all") and rng.random() < 0.5)
    return case


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _lens(case):
    """The lengths that the case stands for; the first is the longest."""
    r = random.Random(case["lens"])
    lo, hi = case["min_len"], case["max_len"]
    return [hi] + [r.randint(lo, hi) for _ in range(case["n_seq"] - 1)]


def _starts(case):
    """First token of each sequence's last document: anywhere, and for a few behind the last token."""
    r = random.Random(case["lens"] + 1)
    return [n if r.random() < 0.1 else r.randint(0, max(0, n - 1)) if case["starts"] else 0 for n in _lens(case)]


def _pages(n, page):
    return (n + page - 1) // page


def _pool(case, n_pages, gen):
    """K and V pools [n_pages][page][kv][..] (order "head": stored head-major) and their scales: of Q8 a number, of the
    4-bit format the step and the least value of 32 elements, whose two values a byte are counted from there."""
    P, H, D = case["page"], case["kv"], case["dim"]

    def make(last, fill):
        shape = (n_pages, H, P, *last) if case["order"] == "head" else (n_pages, P, H, *last)
        t = fill(shape)
        return t.transpose(1, 2) if case["order"] == "head" else t

    def uniform(s):
        return torch.rand(s, generator=gen, device=_DEV)

    def nibbles(s):
        u = (torch.randn(s, generator=gen, device=_DEV) * 3 + 7.5).round_().clamp_(0, 15).to(torch.uint8)
        return u[..., 0::2] | (u[..., 1::2] << 4)

    def steps(s):
        d = 0.25 + 0.25 * uniform(s)
        return torch.stack([d, -7.5 * d + 0.2 * uniform(s)], -1).bfloat16()

    if case["fmt"] == "bf16":
        return [make([D], lambda s: torch.randn(s, generator=gen, device=_DEV, dtype=torch.bfloat16)) for _ in range(2)] + [None, None]
    if case["fmt"] == "a4":
        return [make([D], nibbles) for _ in range(2)] + [make([D // _BLOCK], steps) for _ in range(2)]
    q = [make([D], lambda s: (torch.randn(s, generator=gen, device=_DEV) * 40).round_().clamp_(-127, 127).to(torch.int8)) for _ in range(2)]
    return q + [make([D // _BLOCK], lambda s: 0.015 + 0.02 * uniform(s)) for _ in range(2)]


def prepare(case, seed):
    gen = torch.Generator(device=_DEV).manual_seed(seed)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=_DEV)  # noqa: E731
    P, H, D = case["page"], case["kv"], case["dim"]
    st = {"case": case}
    if case["op"] == "append":
        n = case["n"]
        n_pages = _pages(n, P) + 3
        st["pool"] = _pool(case, n_pages, gen)
        pages = torch.randperm(n_pages, generator=gen, device=_DEV)
        tok = torch.arange(n, device=_DEV)
        st["slots"] = (pages[tok // P] * P + tok % P).to(torch.int32)
        if case["fused"]:  # columns of one q/k/v result, q as wide as four times k
            x = torch.randn((n, 6, H, D), generator=gen, device=_DEV)
            st["k"], st["v"] = x[:, 4], x[:, 5]
        else:
            st["k"], st["v"] = (torch.randn((n, H, D), generator=gen, device=_DEV) for _ in range(2))
        st["k_read"], st["v_read"] = (torch.empty((n, H, D), device=_DEV) for _ in range(2))
    else:
        lens = _lens(case)
        n, width = len(lens), max(1, case["max_len"])
        held = [_pages(m, P) for m in lens]
        n_pages, cols = sum(held) + 2, max(1, max(held))
        st["pool"] = _pool(case, n_pages, gen)
        perm = torch.randperm(n_pages, generator=gen, device=_DEV).to(torch.int32)
        col = torch.arange(cols, device=_DEV)
        h = torch.tensor(held, device=_DEV)
        at = (torch.cumsum(h, 0) - h)[:, None] + col
        st["table"] = torch.where(col < h[:, None], perm[at.clamp(max=n_pages - 1)], 0).to(torch.int32).contiguous()
        st["lens"] = i32(lens)
        st["positions"] = None
        if case["moved"]:  # of tokens that earlier evictions have moved: in any order, the last one the newest
            st["positions"] = torch.rand((n, width), generator=gen, device=_DEV).argsort(-1).to(torch.int32)
            st["positions"].scatter_(1, (st["lens"].long() - 1).clamp(min=0)[:, None], width)
        if case["op"] != "attend":  # most tokens collect little, some much, some nothing yet
            u = torch.rand((n, width), generator=gen, device=_DEV)
            st["weights"] = torch.where(u < 0.05, 0.0, u ** -0.7 - 1)
            st["weights_out"] = st["weights"].clone()
        if case["op"] == "evict":
            st["positions_out"] = None if st["positions"] is None else st["positions"].clone()
            st["kept"] = torch.empty((n, case["keep"]), dtype=torch.int32, device=_DEV)
            st["drop"] = torch.empty(n, dtype=torch.int32, device=_DEV)
            if case["fmt"] != "bf16":  # the tokens that are left, to be read back as values
                left = torch.arange(case["keep"], device=_DEV)
                slot = st["table"][:, (left // P).clamp(max=cols - 1)] * P + left % P
                st["slots"] = torch.where(left < st["lens"][:, None], slot, -1).to(torch.int32).flatten()
                st["k_read"], st["v_read"] = (torch.empty((n * case["keep"], H, D), device=_DEV) for _ in range(2))
        else:
            heads = case["heads"]
            st["q"] = torch.randn((n, heads, D), generator=gen, device=_DEV)
            st["starts"] = i32(_starts(case)) if case["starts"] else None
            # the powers 2^(-8 h / heads) that such biases take
            st["slopes"] = torch.exp2(-8 * torch.arange(1, heads + 1, device=_DEV) / heads) if case["slopes"] else None
            if case["op"] == "attend":
                st["out"], st["lse"] = torch.empty_like(st["q"]), torch.empty((n, heads), device=_DEV)
            else:
                st["add"] = i32([1] * n)
                s = _plain_scores(st)
                m = s.amax(-1, keepdim=True)
                st["lse"] = (m + torch.log(torch.exp(s - torch.where(m == -math.inf, 0.0, m)).sum(-1, keepdim=True))).view(n, heads)
    if own:
        import shared_input_linear_gb300 as sil
        st["cache"] = sil.KVCache(*st["pool"])
    return st


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(st):
    case = st["case"]
    op = case["op"]
    if own:
        import shared_input_linear_gb300 as sil
        if op == "append":
            sil.kv_append(st["cache"], st["k"], st["v"], st["slots"])
            sil.kv_read(st["cache"], st["slots"], st["k_read"], st["v_read"])  # as the values they stand for
            return {"k": st["k_read"], "v": st["v_read"]}
        if op == "evict":
            sil.kv_evict(st["cache"], st["table"], st["lens"], st["weights"], st["kept"], st["drop"], first=case["first"],
                         recent=case["recent"], weights_out=st["weights_out"], positions=st["positions"], positions_out=st["positions_out"])
            if case["fmt"] != "bf16":
                sil.kv_read(st["cache"], st["slots"], st["k_read"], st["v_read"])
            return _evicted(st)
        scores = {"window": case["window"], "cap": case["cap"], "slopes": st["slopes"], "starts": st["starts"], "positions": st["positions"]}
        if op == "attend":
            sil.kv_attend(st["cache"], st["q"], st["table"], st["lens"], st["out"], lse=st["lse"], **scores)
            return {"out": st["out"], "lse": st["lse"]}
        sil.kv_weigh(st["cache"], st["q"], st["table"], st["lens"], st["lse"], st["weights"], weights_out=st["weights_out"],
                     add=st["add"], **scores)
        return {"weights": st["weights_out"]}
    return {"append": _plain_append, "attend": _plain_attend, "weigh": _plain_weigh, "evict": _plain_evict}[op](st)


def _plain_quantise(x, pool, steps, page, at, out):
    """Rows x [n][kv][dim] into a 4-bit pool, and what they read back as.  Of 32 values: the least one rounded down to
    bf16, a fifteenth of the range from there rounded up to bf16, and for each the nearest of 16 steps."""
    def toward(v, up):  # bf16 at or beyond a 32-bit float: the upper half of its bits, one more where that falls short
        bits = v.view(torch.int32)
        head = bits & -65536
        short = (bits != head) & ((bits >= 0) if up else (bits < 0))
        return (head + short.int() * 65536).view(torch.float32)

    b = x.reshape(*x.shape[:2], -1, _BLOCK)
    least = toward(b.amin(-1), False)
    fifteen = torch.full((), 15.0, device=x.device)  # a tensor: torch multiplies by the rounded reciprocal of a plain number
    d = toward((b.amax(-1) - least) / fifteen, True)
    u = torch.where(d[..., None] > 0, (b - least[..., None]) / d[..., None], 0.0).round().clamp(0, 15).to(torch.uint8).view(x.shape)
    pool[page, at] = u[..., 0::2] | (u[..., 1::2] << 4)
    steps[page, at] = torch.stack([d, least], -1).bfloat16()
    out.copy_(_values(pool[page, at], steps[page, at]))


def _plain_append(st):
    P = st["case"]["page"]
    page, at = st["slots"].long() // P, st["slots"].long() % P
    pk, pv, dk, dv = st["pool"]
    _plain_quantise(st["k"], pk, dk, page, at, st["k_read"])
    _plain_quantise(st["v"], pv, dv, page, at, st["v_read"])
    return {"k": st["k_read"], "v": st["v_read"]}


def _values(x, scale):
    """Cached rows [..][dim] of any format in 32 bits."""
    if scale is None:
        return x.float()
    if x.dtype == torch.int8:
        return (x.float().unflatten(-1, (-1, _BLOCK)) * scale[..., None]).flatten(-2)
    u = torch.stack([x & 15, x >> 4], -1).flatten(-2).float().unflatten(-1, (-1, _BLOCK))
    return (u * scale[..., :1].float() + scale[..., 1:].float()).flatten(-2)


def _rows(st, pool, scale):
    """K or V of every sequence [n][kv][T][dim]."""
    tok = torch.arange(st["case"]["max_len"], device=st["lens"].device)
    page, at = st["table"].long()[:, tok // st["case"]["page"]], (tok % st["case"]["page"]).expand(st["lens"].numel(), -1)
    return _values(pool[page, at], None if scale is None else scale[page, at]).transpose(1, 2)


def _plain_scores(st):
    """Logits [n][kv][heads / kv][T], -inf where a token is not seen."""
    case = st["case"]
    H, Hk, D = case["heads"], case["kv"], case["dim"]
    lens = st["lens"].long()[:, None]
    n, tok = lens.numel(), torch.arange(case["max_len"], device=lens.device)
    seen = tok < lens
    if case["window"]:
        seen = seen & (tok >= lens - case["window"])
    if st["starts"] is not None:
        seen = seen & (tok >= st["starts"].long()[:, None])
    q = st["q"].view(n, Hk, H // Hk, D) * (1.0 / math.sqrt(D))
    s = torch.matmul(q, _rows(st, st["pool"][0], st["pool"][2]).transpose(2, 3))
    if case["cap"]:
        s = torch.tanh_(s.div_(case["cap"])).mul_(case["cap"])
    if st["slopes"] is not None:  # times the distance from the last token, which is 0 or negative
        pos = tok.expand(n, -1) if st["positions"] is None else st["positions"].long()[:, : tok.numel()]
        far = (pos - pos.gather(1, (lens - 1).clamp(min=0))).float()
        s += st["slopes"].view(1, Hk, H // Hk, 1) * far[:, None, None]
    return s.masked_fill_(~seen[:, None, None], -math.inf)


def _plain_attend(st):
    case = st["case"]
    s = _plain_scores(st)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, 0.0, m))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, _rows(st, st["pool"][1], st["pool"][3])) / torch.where(total == 0, 1.0, total)
    st["out"].copy_(o.view(st["out"].shape))
    st["lse"].copy_((m + torch.log(total)).view(-1, case["heads"]))
    return {"out": st["out"], "lse": st["lse"]}


def _plain_weigh(st):
    s = _plain_scores(st)
    lse = st["lse"].view(*s.shape[:3], 1)
    p = torch.where(s == -math.inf, 0.0, torch.exp(s - lse)).sum((1, 2))  # over all query heads
    tok, lens = torch.arange(p.shape[1], device=p.device), st["lens"].long()[:, None]
    before = torch.where(tok >= lens - st["add"].long()[:, None], 0.0, st["weights"])
    st["weights_out"].copy_(torch.where(tok < lens, before + p, st["weights_out"]))
    return {"weights": st["weights_out"]}


def _plain_evict(st):
    case = st["case"]
    w, keep, P = st["weights"], case["keep"], case["page"]
    n, width = w.shape
    idx, lens = torch.arange(width, device=w.device), st["lens"].long()[:, None]
    live = idx < lens
    pos = idx.expand(n, -1) if st["positions"] is None else st["positions"].long()
    newest = pos.gather(1, (lens - 1).clamp(min=0))
    always = (pos < case["first"]) | (pos > newest - case["recent"])
    order = torch.sort(w, dim=1, descending=True, stable=True).indices
    rank = torch.where(live, 1 + always.long(), 0).gather(1, order)
    order = order.gather(1, torch.sort(rank, dim=1, descending=True, stable=True).indices)
    chosen = torch.zeros_like(live).scatter(1, order[:, :keep], True) & live
    left = lens.clamp(max=keep)
    hole, spare = ~chosen & (idx < left), chosen & (idx >= left)
    source = torch.sort(spare.int(), dim=1, descending=True, stable=True).indices  # tokens that move, the first first
    entry = torch.where(hole, source.gather(1, (hole.cumsum(1) - 1).clamp(min=0)), idx)
    entry = torch.where(idx < left, entry, -1)
    st["kept"].fill_(-1)
    st["kept"][:, : min(keep, width)] = entry[:, :keep]
    st["drop"].copy_((left - lens)[:, 0])
    old = entry.clamp(min=0)
    st["weights_out"].copy_(torch.where(entry >= 0, w.gather(1, old), st["weights_out"]))
    if st["positions"] is not None:
        st["positions_out"].copy_(torch.where(entry >= 0, st["positions"].gather(1, old), st["positions_out"]))
    r, i = hole.nonzero(as_tuple=True)
    j = entry[r, i]
    to, of = (st["table"].long()[r, i // P], i % P), (st["table"].long()[r, j // P], j % P)
    k, v, dk, dv = st["pool"]
    k[to], v[to] = k[of], v[of]
    if dk is not None:
        dk[to], dv[to] = dk[of], dv[of]
        slot = st["slots"].long()
        page, at = slot.clamp(min=0) // P, slot.clamp(min=0) % P
        there = (slot >= 0)[:, None, None]
        st["k_read"].copy_(torch.where(there, _values(k[page, at], dk[page, at]), 0.0))
        st["v_read"].copy_(torch.where(there, _values(v[page, at], dv[page, at]), 0.0))
    return _evicted(st)


def _evicted(st):
    found = {"kept": st["kept"], "drop": st["drop"], "weights": st["weights_out"], "positions": st["positions_out"]}
    bf16 = st["case"]["fmt"] == "bf16"
    return {**found, "k": st["pool"][0] if bf16 else st["k_read"], "v": st["pool"][1] if bf16 else st["v_read"]}


# ---------------------------------------------------------------------------
# What a pass cannot do without, and what it gives in 64 bits
# ---------------------------------------------------------------------------
def _row_bytes(case):
    """Bytes of K, or of V, of one token in the cache."""
    width = case["kv"] * case["dim"]
    return {"bf16": 2 * width, "q8": width + 4 * width // _BLOCK, "a4": width // 2 + 4 * width // _BLOCK}[case["fmt"]]


def work(case):
    row = _row_bytes(case)
    if case["op"] == "append":
        return {"bytes": case["n"] * (8 * case["kv"] * case["dim"] + row * 4 + 8 * case["kv"] * case["dim"] + 4), "flops": 0}
    lens, P = _lens(case), case["page"]
    if case["op"] == "evict":
        # every weight (and position) is read and every one that is kept written; the rows that move are taken to be those
        # of a choice without regard to the place, read and written once; a cache in 8 or 4 bits is read back
        scalar = 8 if case["moved"] else 4
        total = 0
        for n in lens:
            left = min(n, case["keep"])
            total += scalar * (n + left) + 4 * case["keep"] + 8
            total += 0 if n <= left else int(left * (n - left) / n) * 4 * row
            total += 0 if case["fmt"] == "bf16" else left * (2 * row + 8 * case["kv"] * case["dim"])
        return {"bytes": total, "flops": 0}
    first = _starts(case) if case["starts"] else [0] * len(lens)
    seen = [max(0, n - max(s, n - case["window"] if case["window"] else 0)) for n, s in zip(lens, first)]
    heads, D = case["heads"], case["dim"]
    pages = sum(_pages(m, P) for m in seen)
    side = 4 * (pages + len(lens)) + (4 * sum(seen) if case["moved"] else 0)
    if case["op"] == "weigh":
        return {"bytes": sum(seen) * row + 8 * sum(lens) + case["n_seq"] * heads * (4 * D + 4) + side, "flops": 2 * sum(seen) * heads * D}
    return {"bytes": 2 * sum(seen) * row + case["n_seq"] * heads * (8 * D + 4) + side, "flops": 4 * sum(seen) * heads * D}


def _single(x):
    """Rounded to a 32-bit float, as the definition of a format says at that place."""
    return x.float().double()


def _exact_rows(case, pool, scale, page, at):
    x = pool[page, at]
    if case["fmt"] == "bf16":
        return x.double()
    if case["fmt"] == "q8":
        return x.double() * scale[page, at].double().repeat_interleave(_BLOCK, -1)
    step, least = scale[page, at].double().unbind(-1)
    both = torch.empty((*x.shape[:-1], 2 * x.shape[-1]), dtype=torch.float64, device=x.device)
    both[..., 0::2], both[..., 1::2] = (x % 16).double(), (x // 16).double()
    return both * step.repeat_interleave(_BLOCK, -1) + least.repeat_interleave(_BLOCK, -1)


def _exact_append(x):
    def coarse(v, sign):  # the nearest number of 8 bits on that side
        unit = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=1e-30))) - 7)
        return torch.where(v == 0, v, sign * torch.floor(sign * v / unit) * unit)

    x = x.double().unflatten(-1, (-1, _BLOCK))
    least = coarse(x.min(-1, keepdim=True).values, 1)
    step = coarse(_single(_single(x.max(-1, keepdim=True).values - least) / 15), -1)
    u = torch.round(_single(_single(x - least) / step)).clamp(0, 15)
    return (u * step + least).flatten(-2)


def _exact_evict(case, st):
    P, keep = case["page"], case["keep"]
    weights = st["weights"].double()
    pools = [None if p is None else p.clone() for p in st["pool"]]
    k, v, dk, dv = pools
    for r, n in enumerate(_lens(case)):
        if n <= keep:
            continue
        pos = torch.arange(n, device=_DEV) if st["positions"] is None else st["positions"][r, :n].long()
        w = st["weights"][r, :n].double()
        w[(pos < case["first"]) | (pos > pos[-1] - case["recent"])] = math.inf
        best = sorted(zip((-w).tolist(), range(n)))[:keep]
        stay = {i for _, i in best}
        holes, movers = [i for i in range(keep) if i not in stay], sorted(i for i in stay if i >= keep)
        i, j = torch.tensor(holes, dtype=torch.long, device=_DEV), torch.tensor(movers, dtype=torch.long, device=_DEV)
        weights[r, i] = weights[r, j]
        row = st["table"][r].long()
        for p in pools:
            if p is not None:
                p[row[i // P], i % P] = p[row[j // P], j % P]
    if case["fmt"] == "bf16":
        k, v = k.double(), v.double()
    else:
        slot = st["slots"].long()
        page, at = slot.clamp(min=0) // P, slot.clamp(min=0) % P
        k, v = (_exact_rows(case, p, d, page, at) * (slot >= 0)[:, None, None] for p, d in ((k, dk), (v, dv)))
    return {"kept": None, "drop": None, "weights": weights, "positions": None, "k": k, "v": v}


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "append":
        return {"k": _exact_append(st["k"]), "v": _exact_append(st["v"])}
    if case["op"] == "evict":
        return _exact_evict(case, st)
    P, H, Hk, D = case["page"], case["heads"], case["kv"], case["dim"]
    out = torch.zeros((case["n_seq"], H, D), dtype=torch.float64, device=_DEV)
    lse = torch.full((case["n_seq"], H), -math.inf, dtype=torch.float64, device=_DEV)
    weights = st["weights"].double() if case["op"] == "weigh" else None
    starts = _starts(case) if case["starts"] else [0] * case["n_seq"]
    for r, n in enumerate(_lens(case)):
        if weights is not None and n > 0:
            weights[r, n - 1] = 0  # the token that has just come
        begin = max(starts[r], n - case["window"] if case["window"] else 0)
        if begin >= n:
            continue
        at = torch.arange(begin, n, device=_DEV)
        page = st["table"][r][at // P].long()
        k = _exact_rows(case, st["pool"][0], st["pool"][2], page, at % P)
        v = _exact_rows(case, st["pool"][1], st["pool"][3], page, at % P) if weights is None else None
        for h in range(Hk):
            heads = slice(h * (H // Hk), (h + 1) * (H // Hk))
            s = st["q"][r, heads].double() @ k[:, h].T / math.sqrt(D)
            if case["cap"]:
                s = case["cap"] * torch.tanh(s / case["cap"])
            if case["slopes"]:
                pos = at if st["positions"] is None else st["positions"][r, begin:n].long()
                s = s + st["slopes"][heads].double()[:, None] * (pos - pos[-1]).double()
            if weights is not None:
                weights[r, begin:n] += torch.exp(s - st["lse"][r, heads].double()[:, None]).sum(0)
                continue
            lse[r, heads] = torch.logsumexp(s, -1)
            out[r, heads] = torch.softmax(s, -1) @ v[:, h]
    return {"weights": weights} if weights is not None else {"out": out, "lse": lse}
