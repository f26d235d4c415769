"""Cases of the paged K/V cache operators: block tables and slot maps (``kv_extend``), rows written
into the cache (``kv_append``; ``kv_read`` brings them back as values) and the attention of one new
token per sequence over it (``kv_attend``).

``run`` computes an operator in elementary torch operations in 32 bits where ``own`` is false, and
through the package's entry points where it is true.  Head counts 32 / 8 of 128 are the q/k/v
projections 4096 -> 4096 / 1024 / 1024 that the benchmark runs; the others are generic.
"""
import math
import random

import torch

own = False

_DEV = "cuda" if torch.cuda.is_available() else "cpu"
_BLOCK = 32  # elements of one Q8 scale


def listed():
    return [
        # one decode step of a small batch: every sequence one token longer
        {"name": "extend_32_decode", "op": "extend", "n_seq": 32, "page": 16, "mix": "decode", "max_len": 4000, "lens": 1},
        # a scheduler step of a large server: decoding, chunks of prompts, rejected drafts, finished requests
        {"name": "extend_1024_mixed", "op": "extend", "n_seq": 1024, "page": 16, "mix": "mixed", "max_len": 6000, "lens": 2},
        # one token of one sequence: the smallest write
        {"name": "append_1_bf16", "op": "append", "fmt": "bf16", "n": 1, "kv": 8, "dim": 128, "page": 16, "order": "head", "fused": False},
        # a long prompt's K and V, as columns of one q/k/v result
        {"name": "append_16384_bf16", "op": "append", "fmt": "bf16", "n": 16384, "kv": 8, "dim": 128, "page": 16, "order": "head", "fused": True},
        # a decode step of 64 sequences into an 8-bit cache
        {"name": "append_64_q8", "op": "append", "fmt": "q8", "n": 64, "kv": 8, "dim": 128, "page": 64, "order": "token", "fused": False},
        # a prompt chunk of odd length into an 8-bit cache
        {"name": "append_4097_q8", "op": "append", "fmt": "q8", "n": 4097, "kv": 8, "dim": 128, "page": 16, "order": "head", "fused": True},
        # one short chat: latency
        {"name": "attend_1x512_bf16", "op": "attend", "fmt": "bf16", "n_seq": 1, "heads": 32, "kv": 8, "dim": 128, "page": 16,
         "order": "head", "min_len": 512, "max_len": 512, "lens": 3, "window": 0},
        # a batch of unlike lengths, some slots of it idle (length 0)
        {"name": "attend_32_ragged_bf16", "op": "attend", "fmt": "bf16", "n_seq": 32, "heads": 32, "kv": 8, "dim": 128, "page": 16,
         "order": "token", "min_len": 0, "max_len": 8192, "lens": 4, "window": 0},
        # a full server at an ordinary length: the largest
        {"name": "attend_128x4096_bf16", "op": "attend", "fmt": "bf16", "n_seq": 128, "heads": 32, "kv": 8, "dim": 128, "page": 64,
         "order": "head", "min_len": 4096, "max_len": 4096, "lens": 5, "window": 0},
        # one long document: the split over the length
        {"name": "attend_1x131071_q8", "op": "attend", "fmt": "q8", "n_seq": 1, "heads": 32, "kv": 8, "dim": 128, "page": 64,
         "order": "head", "min_len": 131071, "max_len": 131071, "lens": 6, "window": 0},
        # a batch of unlike lengths in an 8-bit cache
        {"name": "attend_64_ragged_q8", "op": "attend", "fmt": "q8", "n_seq": 64, "heads": 32, "kv": 8, "dim": 128, "page": 16,
         "order": "head", "min_len": 1, "max_len": 8192, "lens": 7, "window": 0},
        # one K/V head of 256 under a sliding window
        {"name": "attend_16_window_d256", "op": "attend", "fmt": "bf16", "n_seq": 16, "heads": 8, "kv": 1, "dim": 256, "page": 32,
         "order": "head", "min_len": 1000, "max_len": 16384, "lens": 8, "window": 4096},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["extend", "append", "append", "attend", "attend", "attend"])
    page = rng.choice([8, 16, 16, 24, 32, 64, 128])
    if op == "extend":
        return {"op": op, "n_seq": _log_int(rng, 1, 2048), "page": page, "mix": rng.choice(["decode", "mixed"]),
                "max_len": _log_int(rng, 16, 6000), "lens": rng.randrange(1 << 30)}
    fmt, order = rng.choice(["bf16", "q8"]), rng.choice(["head", "token"])
    if op == "append":
        kv, dim = rng.choice([(8, 128), (8, 64), (4, 128), (1, 256), (2, 96), (12, 64)])
        return {"op": op, "fmt": fmt, "n": _log_int(rng, 1, 16384), "kv": kv, "dim": dim, "page": page, "order": order,
                "fused": rng.random() < 0.5}
    heads, kv, dim = rng.choice([(32, 8, 128), (32, 8, 128), (32, 4, 128), (16, 16, 64), (32, 8, 64), (8, 1, 256), (16, 8, 256),
                                 (14, 2, 64), (40, 8, 128), (24, 2, 96), (32, 2, 128)])
    longest = _log_int(rng, 1, 65536)
    n_seq = _log_int(rng, 1, max(1, min(256, (1 << 28) // (longest * kv * dim))))
    return {"op": op, "fmt": fmt, "n_seq": n_seq, "heads": heads, "kv": kv, "dim": dim, "page": page, "order": order,
            "min_len": rng.choice([0, 1, (longest + 1) // 2]), "max_len": longest, "lens": rng.randrange(1 << 30),
            "window": rng.choice([0, 0, 0, _log_int(rng, 1, longest)])}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _lens(case):
    """The lengths that the case stands for; the first is the longest."""
    r = random.Random(case["lens"])
    lo, hi = case.get("min_len", 0), case["max_len"]
    return [hi] + [r.randint(lo, hi) for _ in range(case["n_seq"] - 1)]


def _adds(case, lens):
    """Changes of length of one scheduler step."""
    if case["mix"] == "decode":
        return [1] * len(lens)
    r = random.Random(case["lens"] + 1)
    got = []
    for n in lens:
        u = r.random()
        if u < 0.6:
            got.append(1)                        # decodes
        elif u < 0.8:
            got.append(r.randint(2, 512))        # a chunk of a prompt
        elif u < 0.9:
            got.append(-min(n, r.randint(1, 4)))  # rejected draft tokens
        elif u < 0.95:
            got.append(-n)                       # finished
        else:
            got.append(0)                        # waits
    return got


def _pages(n, page):
    return (n + page - 1) // page


def _pool(case, n_pages, gen):
    """K and V pools [n_pages][page][kv][dim] (order "head": stored head-major) and, for Q8, their scales."""
    P, H, D = case["page"], case["kv"], case["dim"]

    def make(last, fill):
        shape = (n_pages, H, P, last) if case["order"] == "head" else (n_pages, P, H, last)
        t = fill(shape)
        return t.transpose(1, 2) if case["order"] == "head" else t

    if case["fmt"] == "bf16":
        return [make(D, lambda s: torch.randn(s, generator=gen, device=_DEV, dtype=torch.bfloat16)) for _ in range(2)] + [None, None]
    q = [make(D, lambda s: (torch.randn(s, generator=gen, device=_DEV) * 40).round_().clamp_(-127, 127).to(torch.int8)) for _ in range(2)]
    d = [make(D // _BLOCK, lambda s: 0.015 + 0.02 * torch.rand(s, generator=gen, device=_DEV)) for _ in range(2)]
    return q + d


def prepare(case, seed):
    gen = torch.Generator(device=_DEV).manual_seed(seed)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=_DEV)  # noqa: E731
    st = {"case": case}
    if case["op"] == "extend":
        lens, P = _lens(case), case["page"]
        adds = _adds(case, lens)
        want = [max(0, n + a) for n, a in zip(lens, adds)]
        held = [_pages(n, P) for n in lens]
        spare = sum(max(0, _pages(w, P) - h) for w, h in zip(want, held)) + 7
        n_pages = sum(held) + spare
        perm = torch.randperm(n_pages, generator=gen, device=_DEV).to(torch.int32)
        width = max(max(_pages(w, P), h) for w, h in zip(want, held)) + 1
        col = torch.arange(width, device=_DEV)
        h = torch.tensor(held, device=_DEV)
        at = (torch.cumsum(h, 0) - h)[:, None] + col
        table = torch.where(col < h[:, None], perm[at.clamp(max=n_pages - 1)], -1).to(torch.int32).contiguous()
        head = int(torch.randint(0, 5 * n_pages, (1,), generator=gen, device=_DEV))
        ring = torch.full((n_pages,), -1, dtype=torch.int32, device=_DEV)
        ring[(head + torch.arange(spare, device=_DEV)) % n_pages] = perm[sum(held):]
        tokens = sum(max(0, a) for a in adds)
        most = tokens + 3
        st.update(page=P, lens=i32(lens), add=i32(adds), table=table, ring=ring,
                  cursor=torch.tensor([head, head + spare], dtype=torch.int64, device=_DEV),
                  lens_out=torch.empty(len(lens), dtype=torch.int32, device=_DEV),
                  cursor_out=torch.empty(2, dtype=torch.int64, device=_DEV),
                  slots=torch.empty(most, dtype=torch.int32, device=_DEV),
                  positions=torch.empty(most, dtype=torch.int32, device=_DEV),
                  first=torch.empty(len(lens) + 1, dtype=torch.int32, device=_DEV),
                  info=torch.empty(4, dtype=torch.int64, device=_DEV))
        return st
    if case["op"] == "append":
        n, H, D, P = case["n"], case["kv"], case["dim"], case["page"]
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
        if case["fmt"] == "q8":
            st["k_read"], st["v_read"] = (torch.empty((n, H, D), device=_DEV) for _ in range(2))
    else:
        lens, P, H = _lens(case), case["page"], case["heads"]
        held = [_pages(n, P) for n in lens]
        n_pages, width = sum(held) + 2, max(1, max(held))
        st["pool"] = _pool(case, n_pages, gen)
        perm = torch.randperm(n_pages, generator=gen, device=_DEV).to(torch.int32)
        col = torch.arange(width, device=_DEV)
        h = torch.tensor(held, device=_DEV)
        at = (torch.cumsum(h, 0) - h)[:, None] + col
        st["table"] = torch.where(col < h[:, None], perm[at.clamp(max=n_pages - 1)], 0).to(torch.int32).contiguous()
        st["lens"] = i32(lens)
        st["q"] = torch.randn((len(lens), H, case["dim"]), generator=gen, device=_DEV)
        st["out"] = torch.empty_like(st["q"])
        st["lse"] = torch.empty((len(lens), H), device=_DEV)
    if own:
        import shared_input_linear_gb300 as sil
        st["cache"] = sil.KVCache(*st["pool"])
    return st


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(st):
    op = st["case"]["op"]
    if own:
        import shared_input_linear_gb300 as sil
        if op == "extend":
            sil.kv_extend(st["lens"], st["add"], st["table"], st["ring"], st["cursor"], st["page"], st["slots"],
                          lens_out=st["lens_out"], cursor_out=st["cursor_out"], positions=st["positions"],
                          first=st["first"], info=st["info"])
            return {k: st[k] for k in ("lens_out", "table", "ring", "cursor_out", "slots", "positions", "first", "info")}
        if op == "append":
            sil.kv_append(st["cache"], st["k"], st["v"], st["slots"])
            if st["case"]["fmt"] == "bf16":
                return {"k": st["pool"][0], "v": st["pool"][1]}
            sil.kv_read(st["cache"], st["slots"], st["k_read"], st["v_read"])  # as the values they stand for
            return {"k": st["k_read"], "v": st["v_read"]}
        sil.kv_attend(st["cache"], st["q"], st["table"], st["lens"], st["out"], lse=st["lse"], window=st["case"]["window"])
        return {"out": st["out"], "lse": st["lse"]}
    return {"extend": _plain_extend, "append": _plain_append, "attend": _plain_attend}[op](st)


def _plain_extend(st):
    lens, add, table, ring, cursor, P = (st[k] for k in ("lens", "add", "table", "ring", "cursor", "page"))
    n_seq, width = table.shape
    size, most = ring.numel(), st["slots"].numel()
    lens, add, head, tail = lens.long(), add.long(), cursor[0], cursor[1]
    new = (lens + add).clamp(min=0)
    had, has = (lens + P - 1) // P, (new + P - 1) // P
    take, give, grow = (has - had).clamp(min=0), (had - has).clamp(min=0), add.clamp(min=0)
    take_end, give_end, grow_end = take.cumsum(0), give.cumsum(0), grow.cumsum(0)
    code = (take_end[-1] > tail - head) * 1 + (has.max() > width) * 2 + (grow_end[-1] > most) * 4
    ok = code == 0

    def owner(end, count):  # for item i of `count`: the sequence it belongs to, its rank in it, whether there is one
        i = torch.arange(count, device=end.device)
        s = torch.searchsorted(end, i, right=True).clamp(max=n_seq - 1)
        return i, s, (i < end[-1]) & ok

    # pages given back, from the table as it was, to the tail of the ring
    j, s, live = owner(give_end, size)
    page = table[s, (has[s] + j - (give_end - give)[s]).clamp(0, width - 1)]
    ring_new = torch.cat([ring, ring[:1]]).scatter(0, torch.where(live, (tail + j) % size, size), page)[:size]
    # pages taken from its head
    i, s, live = owner(take_end, most)
    col = torch.where(live, had[s] + i - (take_end - take)[s], width).clamp(max=width)
    wide = torch.cat([table, table[:, :1]], 1).flatten()
    table_new = wide.scatter(0, s * (width + 1) + col, ring[(head + i) % size]).view(n_seq, width + 1)[:, :width]
    # the new tokens' positions and slots
    i, s, live = owner(grow_end, most)
    pos = lens[s] + i - (grow_end - grow)[s]
    slot = table_new[s, (pos // P).clamp(0, width - 1)] * P + pos % P
    st["slots"].copy_(torch.where(live, slot, -1))
    st["positions"].copy_(torch.where(live, pos, -1))
    st["first"].copy_(torch.cat([grow_end.new_zeros(1), grow_end]) * ok)
    st["lens_out"].copy_(torch.where(ok, new, lens))
    st["cursor_out"].copy_(torch.stack([head + take_end[-1] * ok, tail + give_end[-1] * ok]))
    st["info"].copy_(torch.stack([code, grow_end[-1], take_end[-1], give_end[-1]]))
    st["table"].copy_(table_new)
    st["ring"].copy_(ring_new)
    return {k: st[k] for k in ("lens_out", "table", "ring", "cursor_out", "slots", "positions", "first", "info")}


def _plain_append(st):
    P = st["case"]["page"]
    page, at = st["slots"].long() // P, st["slots"].long() % P
    pk, pv, dk, dv = st["pool"]
    if dk is None:
        pk[page, at] = st["k"].to(pk.dtype)
        pv[page, at] = st["v"].to(pv.dtype)
        return {"k": pk, "v": pv}
    top = torch.full((), 127.0, device=pk.device)  # a tensor: torch multiplies by the rounded reciprocal of a plain number
    for x, pool, scales, out in ((st["k"], pk, dk, st["k_read"]), (st["v"], pv, dv, st["v_read"])):
        blocks = x.reshape(*x.shape[:2], -1, _BLOCK)
        d = blocks.abs().amax(-1) / top
        q = torch.where(d[..., None] > 0, blocks / d[..., None], 0.0).round().clamp(-127, 127)
        pool[page, at] = q.reshape(x.shape).to(torch.int8)
        scales[page, at] = d
        back = pool[page, at].float().view(blocks.shape) * scales[page, at][..., None]
        out.copy_(back.view(out.shape))
    return {"k": st["k_read"], "v": st["v_read"]}


def _plain_attend(st):
    case = st["case"]
    P, H, Hk, D = case["page"], case["heads"], case["kv"], case["dim"]
    lens, table = st["lens"].long(), st["table"].long()
    n, T = lens.numel(), case["max_len"]
    tok = torch.arange(T, device=lens.device)
    page, at = table[:, tok // P], (tok % P).expand(n, T)
    pk, pv, dk, dv = st["pool"]

    def rows(pool, scale):  # [n][Hk][T][D] in 32 bits
        x = pool[page, at].float()
        if scale is not None:
            x = (x.view(n, T, Hk, -1, _BLOCK) * scale[page, at][..., None]).view(n, T, Hk, D)
        return x.transpose(1, 2)

    live = (tok < lens[:, None]) & ((tok >= lens[:, None] - case["window"]) if case["window"] else True)
    live = live[:, None, None, :]
    q = st["q"].view(n, Hk, H // Hk, D) * (1.0 / math.sqrt(D))
    s = torch.matmul(q, rows(pk, dk).transpose(2, 3)).masked_fill_(~live, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, 0.0, m))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, rows(pv, dv)) / torch.where(total == 0, 1.0, total)
    st["out"].copy_(o.view(n, H, D))
    st["lse"].copy_((m + torch.log(total)).view(n, H))
    return {"out": st["out"], "lse": st["lse"]}


# ---------------------------------------------------------------------------
# What a pass cannot do without, and what it gives in 64 bits
# ---------------------------------------------------------------------------
def _token_bytes(case):
    """Bytes of K and V of one token in the cache."""
    width = case["kv"] * case["dim"]
    return 2 * (2 * width if case["fmt"] == "bf16" else width + 4 * width // _BLOCK)


def work(case):
    if case["op"] == "extend":
        lens, P = _lens(case), case["page"]
        adds = _adds(case, lens)
        tokens = sum(max(0, a) for a in adds)
        moved = sum(abs(_pages(max(0, n + a), P) - _pages(n, P)) for n, a in zip(lens, adds))
        return {"bytes": 16 * len(lens) + 8 * moved + 8 * tokens + 64, "flops": 0}
    if case["op"] == "append":
        n, width = case["n"], case["kv"] * case["dim"]
        back = 0 if case["fmt"] == "bf16" else _token_bytes(case) + 8 * width  # the values read back
        return {"bytes": n * (8 * width + _token_bytes(case) + back + 4), "flops": 0}
    tokens = sum(min(n, case["window"]) if case["window"] else n for n in _lens(case))
    qo = case["n_seq"] * case["heads"] * (8 * case["dim"] + 4)
    pages = sum(_pages(min(n, case["window"] or n), case["page"]) for n in _lens(case))
    return {"bytes": tokens * _token_bytes(case) + qo + 4 * (pages + case["n_seq"]),
            "flops": 4 * tokens * case["heads"] * case["dim"]}


def exact(case, seed):
    if case["op"] == "extend":
        return None  # whole numbers
    st = prepare(case, seed)
    P = case["page"]
    if case["op"] == "append":
        if case["fmt"] == "bf16":
            k, v = st["pool"][0].double(), st["pool"][1].double()
            for i, s in enumerate(st["slots"].tolist()):
                k[s // P, s % P] = st["k"][i].double()
                v[s // P, s % P] = st["v"][i].double()
            return {"k": k, "v": v}
        found = []
        for x in (st["k"], st["v"]):
            x = x.double()
            x = x.reshape(x.shape[0], x.shape[1], -1, _BLOCK)
            unit = x.abs().max(dim=-1, keepdim=True).values / 127
            found.append((torch.round(x / unit) * unit).reshape(x.shape[0], x.shape[1], -1))
        return {"k": found[0], "v": found[1]}
    H, Hk, D = case["heads"], case["kv"], case["dim"]
    out = torch.zeros((case["n_seq"], H, D), dtype=torch.float64, device=_DEV)
    lse = torch.full((case["n_seq"], H), -math.inf, dtype=torch.float64, device=_DEV)
    for r, n in enumerate(_lens(case)):
        begin = max(0, n - case["window"]) if case["window"] else 0
        if n == 0:
            continue
        at = torch.arange(begin, n, device=_DEV)
        page = st["table"][r][at // P].long()
        k, v = (p[page, at % P].double() for p in st["pool"][:2])
        if case["fmt"] == "q8":
            k, v = (x * d[page, at % P].double().repeat_interleave(_BLOCK, -1) for x, d in zip((k, v), st["pool"][2:]))
        for h in range(Hk):
            heads = slice(h * (H // Hk), (h + 1) * (H // Hk))
            s = st["q"][r, heads].double() @ k[:, h].T / math.sqrt(D)
            lse[r, heads] = torch.logsumexp(s, -1)
            out[r, heads] = torch.softmax(s, -1) @ v[:, h]
    return {"out": out, "lse": lse}
