"""Cases for a paged key-value cache held in 8 bits, with a scale for each block of tokens and key head.

The cache needs no calibration: a block's scale follows from what is written to it.  A layer of a decoder passes through

  append  rotary positions on q and k; k and v quantised as they are written to their slots; a block that a larger value
          joins later gets a larger scale, and what it holds already is rounded again
  read    tokens of the requests as rows of bf16 again, request behind request
  attend  attention of each request's newest tokens over its pages

`run` computes an operator either in elementary torch operations (`own` false) or through group_affine_bit_gb300.api.
"""
import math
import random

import numpy as np
import torch

own = False

KV = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
LEAST, MOST = 2.0 ** -48, 2.0 ** 48  # between which a scale lies


# ----------------------------------------------------------------------------- cases
def listed():
    return [
        # One request early in its answer: the shortest call, where latency is all there is.
        attend("attend_one_short", batch=1, longest=577, spread="full", heads=32, kv_heads=8, dim=256, page=16, block=16),
        # Ordinary serving: 32 requests of mixed lengths, heads as the 8192-deep output projection has them.
        attend("attend_ordinary", batch=32, longest=4096, spread="ragged", heads=32, kv_heads=8, dim=256, page=16, block=16),
        # One reader of a very long document: all the parallelism is in the cache's length.
        attend("attend_one_long", batch=1, longest=262143, spread="full", heads=32, kv_heads=8, dim=128, page=64, block=64, kv="e4m3"),
        # The largest: many long requests, bound by the cache's bytes.
        attend("attend_large", batch=64, longest=32768, spread="ragged", heads=32, kv_heads=8, dim=128, page=32, block=32),
        # Checking five drafted tokens a request, in a layer with a sliding window, over head-major pages.
        attend("attend_draft_window", batch=12, longest=6000, spread="ragged", heads=32, kv_heads=16, dim=256, page=16, block=16, kv="e4m3",
               tokens=5, window=1024, layout="head"),
        # Odd everything: seven query heads to a key head, 80 values a head, pages of 8, a scale for every token, requests of no token and of one.
        attend("attend_odd", batch=19, longest=1501, spread="empty", heads=28, kv_heads=4, dim=80, page=8, block=1),
        # A decode step's rows of 64 requests, most of them in the middle of a block.
        append("append_decode", batch=64, most=1, longest=8192, heads=32, kv_heads=8, dim=128, page=16, block=16, rotary=128, kv="e4m3"),
        # Prompt chunks of four requests that had some already.
        append("append_prompt", batch=4, most=2048, longest=32768, heads=32, kv_heads=8, dim=128, page=64, block=16, rotary=128, kv="e4m3"),
        # A decode step written and its blocks read again, as a check of the cache or a copy of it to somewhere else does.
        append("write_read_decode", batch=48, most=1, longest=16384, heads=32, kv_heads=8, dim=256, page=16, block=16, rotary=256, read=True),
        # Ragged chunks, part of the head turns, neighbouring values make the pairs, two axes, padded rows; read for a prompt's own attention.
        append("write_read_odd", batch=7, most=300, longest=131072, heads=28, kv_heads=4, dim=80, page=8, block=8, rotary=40, axes=2,
               pairs="neighbour", padded=True, read=True),
        # What 16 requests hold, for attention over whole prompts or a move to another pool.
        read("read_ordinary", batch=16, longest=8192, kv_heads=8, dim=128, page=32, block=32),
        # A few requests' tails behind a place of their own, a scale for every token.
        read("read_odd", batch=5, longest=701, kv_heads=4, dim=80, page=8, block=1, kv="e4m3", tail=True),
    ]


def draw(rng):
    """One more case of the same ranges."""
    kind = rng.choice(["attend", "attend", "attend", "append", "append", "read"])
    heads, kv_heads = rng.choice([(32, 8), (32, 16), (32, 4), (28, 4), (16, 16), (16, 1), (8, 2), (40, 8), (6, 2)])
    dim = rng.choice([64, 80, 96, 128, 128, 256, 256, 512])
    page = rng.choice([8, 16, 32, 64, 128])
    block = rng.choice([b for b in (1, 8, 16, 32, 64, 128) if b <= page])
    kv = rng.choice(["int8", "e4m3"])
    if kind == "attend":
        tokens = rng.choice([1, 1, 1, 2, 5, 8])
        batch = _log(rng, 1, 128)
        # what the largest listed case's cache can hold, shared out
        room = 64 * 32768 * 8 * 128 // (batch * kv_heads * dim)
        longest = _log(rng, 64, max(65, min(262144, room)))
        window = rng.choice([0, 0, 0, 512, 1024, 4096])
        spread = rng.choice(["full", "ragged", "ragged", "empty"])
        return attend("", batch, longest, spread, heads, kv_heads, dim, page, block, kv, tokens, window, rng.choice(["token", "head"]))
    if kind == "append":
        rows = _log(rng, 1, 8192 * 128 * 48 // (dim * (heads + 2 * kv_heads)))
        batch = _log(rng, 1, min(rows, 256))
        rotary = rng.choice([dim, dim, dim // 2])
        return append("", batch, max(1, rows // batch), _log(rng, 8192, 262144), heads, kv_heads, dim, page, block, rotary, rng.choice([1, 1, 2, 3]),
                      rng.choice(["half", "half", "neighbour"]), kv, rng.choice([False, True]), kv == "int8")
    batch = _log(rng, 1, 64)
    longest = _log(rng, 16, max(17, min(65536, 16 * 8192 * 8 * 128 // (batch * kv_heads * dim))))
    return read("", batch, longest, kv_heads, dim, page, block, kv, rng.choice([False, True]))


def _log(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def attend(name, batch, longest, spread, heads, kv_heads, dim, page, block, kv="int8", tokens=1, window=0, layout="token"):
    case = dict(op="attend", batch=batch, longest=longest, spread=spread, heads=heads, kv_heads=kv_heads, dim=dim, page=page, block=block, kv=kv,
                tokens=tokens, window=window, layout=layout)
    return {"name": name, **case} if name else case


def append(name, batch, most, longest, heads, kv_heads, dim, page, block, rotary, axes=1, pairs="half", kv="int8", padded=False, read=False):
    case = dict(op="append", batch=batch, most=most, longest=longest, heads=heads, kv_heads=kv_heads, dim=dim, page=page, block=block, rotary=rotary,
                axes=axes, pairs=pairs, kv=kv, padded=padded, read=read)
    return {"name": name, **case} if name else case


def read(name, batch, longest, kv_heads, dim, page, block, kv="int8", tail=False):
    case = dict(op="read", batch=batch, longest=longest, kv_heads=kv_heads, dim=dim, page=page, block=block, kv=kv, tail=tail)
    return {"name": name, **case} if name else case


def _of(case):
    """A generator that the case alone decides, for its requests' lengths."""
    return random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))


def _lengths(case):
    """attend: tokens in the cache of each request, the step's own included."""
    rng, n, most = _of(case), case["batch"], case["longest"]
    if case["spread"] == "full":
        return [most] * n
    lens = [rng.randint(min(case["tokens"], most), most) for _ in range(n)]
    lens[rng.randrange(n)] = most
    if case["spread"] == "empty" and n > 1:  # a slot without a request, a request of one token
        lens[0] = 0
        if n > 2:
            lens[1] = 1
    return lens


def _pieces(case):
    """append, read: (first token, tokens) of each request's piece."""
    rng, got = _of(case), []
    for i in range(case["batch"]):
        if case["op"] == "append":
            n = case["most"] if i == 0 else rng.randint((case["most"] + 1) // 2, case["most"])
            first = rng.randint(0, max(0, case["longest"] - n))
        else:
            end = case["longest"] if i == 0 else rng.randint(1, case["longest"])
            first = rng.randint(0, end - 1) if case["tail"] else 0
            n = end - first
        got.append((first, n))
    return got


def _blocks(case):
    """append with `read`: the pieces, from the beginnings of their first blocks on."""
    return [(first - first % case["block"], n + first % case["block"]) for first, n in _pieces(case)]


def _rows(case):
    """append: rows of the step, those behind the last token among them."""
    n = sum(n for _, n in _pieces(case))
    return -(-n // 64) * 64 + 64 if case["padded"] else n


# ----------------------------------------------------------------------------- what a program has in hand
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _need(top, kv):
    """The scale of a block whose largest magnitude is `top`."""
    if kv == "int8":
        return (top / 127).clamp(LEAST, MOST)
    m, e = torch.frexp((top / 448).clamp(LEAST, MOST))
    return torch.ldexp(torch.ones_like(top), e - (m == 0.5).int())


def _coded(x, kv):
    return x.round().clamp(-127, 127).nan_to_num(0).to(torch.int8) if kv == "int8" else x.clamp(-448, 448).to(torch.float8_e4m3fn)


def _pool(case, pages, g):
    """Codes [page, token, head, value], in either order in memory, and scales [page, block, head], of k and v that were normal."""
    page, block, heads, dim, kv = case["page"], case["block"], case["kv_heads"], case["dim"], case["kv"]
    out = []
    for _ in "kv":
        if case.get("layout") == "head":
            codes = torch.empty(pages, heads, page, dim, dtype=KV[kv], device="cuda").transpose(1, 2)
        else:
            codes = torch.empty(pages, page, heads, dim, dtype=KV[kv], device="cuda")
        scales = torch.empty(pages, page // block, heads, device="cuda")
        each = max(1, (1 << 26) // (page * heads * dim))
        for at in range(0, pages, each):
            n = min(each, pages - at)
            x = torch.empty(n, page // block, block, heads, dim, device="cuda").normal_(generator=g)
            scales[at: at + n] = _need(x.abs().amax((2, 4)), kv)
            codes[at: at + n] = _coded(x / scales[at: at + n, :, None, :, None], kv).view(n, page, heads, dim)
        out += [codes, scales]
    return out


def _tables(spans, page, wide, g):
    """Block tables [request, wide] with a page of a shuffled pool behind every page of the tokens in `spans`; the pool's pages."""
    used = [(f // page, -(-(f + n) // page)) for f, n in spans]
    pool = sum(b - a for a, b in used)
    pool += (pool >> 3) + 1
    order = torch.randperm(pool, device="cuda", generator=g).to(torch.int32)
    a, b = (torch.tensor(x, device="cuda", dtype=torch.int64) for x in zip(*used))
    column = torch.arange(wide, device="cuda")[None]
    at = (torch.cumsum(b - a, 0) - b)[:, None] + column
    held = (column >= a[:, None]) & (column < b[:, None])
    return torch.where(held, order[at.clamp(0, pool - 1)], -1).contiguous(), pool


def _starts(counts):
    return torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = _generator(seed)
    state = {"case": case}
    page, hk, D = case["page"], case["kv_heads"], case["dim"]
    ints = dict(dtype=torch.int32, device="cuda")
    if case["op"] == "attend":
        lens = _lengths(case)
        table, pool = _tables([(0, n) for n in lens], page, -(-case["longest"] // page), g)
        shape = (case["batch"], case["tokens"], case["heads"], D)
        state.update(table=table, lens=torch.tensor(lens, **ints), scale=D ** -0.5,
                     q=torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(generator=g),
                     out=torch.empty(shape, dtype=torch.bfloat16, device="cuda"), lse=torch.empty(shape[:3], device="cuda"))
    else:
        spans = _pieces(case)
        table, pool = _tables(spans, page, -(-case["longest"] // page), g)
        if case["op"] == "append":
            T, hq, axes, half = _rows(case), case["heads"], case["axes"], case["rotary"] // 2
            # the stacked projection's rows: channels of differing size
            gain = torch.exp(0.5 * torch.empty((hq + 2 * hk) * D, device="cuda").normal_(generator=g))
            qkv = (torch.empty(T, (hq + 2 * hk) * D, device="cuda").normal_(generator=g) * gain).to(torch.bfloat16)
            places = torch.cat([torch.arange(f, f + n, device="cuda") for f, n in spans])
            request = torch.cat([torch.full((n,), b, device="cuda") for b, (_, n) in enumerate(spans)])
            kept = places.numel()
            slots = torch.full((T,), -1, device="cuda")
            slots[:kept] = table[request, places // page].long() * page + places % page
            positions = torch.zeros(T, dtype=torch.int64, device="cuda")
            positions[:kept] = places
            side = 37  # an image's rows and columns beside its place in time
            grid = [positions, positions // side % side, positions % side][:axes]
            state.update(q=qkv[:, : hq * D].view(T, hq, D), k=qkv[:, hq * D: (hq + hk) * D].view(T, hk, D), v=qkv[:, (hq + hk) * D:].view(T, hk, D),
                         positions=torch.stack(grid).to(torch.int32).contiguous(), slots=slots.to(torch.int32),
                         turns=torch.from_numpy(_turns(case["rotary"]).view(np.int64)).cuda(), neighbour=case["pairs"] == "neighbour",
                         axis=torch.tensor([i * axes // half for i in range(half)], dtype=torch.uint8, device="cuda"),
                         out=torch.empty(T, hq, D, dtype=torch.bfloat16, device="cuda"))
            spans = _blocks(case)
        rows = sum(n for _, n in spans)
        capacity = rows + (9 if case.get("padded") else 0)
        state.update(table=table, starts=_starts([n for _, n in spans]), first=torch.tensor([f for f, _ in spans], **ints),
                     k_rows=torch.zeros(capacity, hk, D, dtype=torch.bfloat16, device="cuda"),
                     v_rows=torch.zeros(capacity, hk, D, dtype=torch.bfloat16, device="cuda"))
    state.update(zip(("k_codes", "k_scale", "v_codes", "v_scale"), _pool(case, pool, g)))
    return state


def _turns(rotary):
    """Turns that each pair makes a position, 10000^(-2i/rotary) / 2 pi, as 64-bit fractions of a turn."""
    f = 10000.0 ** (-2.0 * np.arange(rotary // 2) / rotary) / (2 * math.pi)
    return np.floor(f * 2.0 ** 64).astype(np.uint64)


# ----------------------------------------------------------------------------- one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return {"attend": _attend_own, "append": _append_own, "read": _read_own}[op](state)
    return {"attend": _attend_plain, "append": _append_plain, "read": _read_plain}[op](state)


def _handles(s):
    """What a program keeps beside its pool."""
    from group_affine_bit_gb300 import api
    if "cache" not in s:
        s["cache"] = api.BlockCache(s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"])
        if s["case"]["op"] == "append":
            s["rope"] = api.Rope(s["turns"], s["axis"], neighbour=s["neighbour"])
    return api


def _attend_own(s):
    api = _handles(s)
    out = api.paged_attention(s["q"], s["cache"], s["table"], s["lens"], scale=s["scale"], window=s["case"]["window"], out=s["out"], lse=s["lse"])
    return {"out": out, "lse": s["lse"]}


def _values(codes, scales, block):
    """codes [..., tokens, heads, dim] times the scales [..., blocks, heads] of their blocks, fp32."""
    return codes.float() * scales.repeat_interleave(block, -2)[..., None]


def _attend_plain(s):
    c = s["case"]
    B, Lq, H, D = s["q"].shape
    hk, page, block = c["kv_heads"], c["page"], c["block"]
    L = s["table"].shape[1] * page
    pages = s["table"].clamp(min=0).long()
    key = torch.arange(L, device="cuda")
    kept = key[None] < s["lens"][:, None]                                            # [B, L]
    last = s["lens"].long()[:, None] - Lq + torch.arange(Lq, device="cuda")[None]    # position of each query
    seen = kept[:, None] & (key[None, None] <= last[:, :, None])
    if c["window"]:
        seen &= key[None, None] > last[:, :, None] - c["window"]
    k = _values(s["k_codes"][pages], s["k_scale"][pages], block).reshape(B, L, hk, D)
    q = s["q"].float().view(B, Lq, hk, H // hk, D).permute(0, 2, 1, 3, 4).reshape(B, hk, -1, D)
    score = torch.matmul(q, k.permute(0, 2, 3, 1)).view(B, hk, Lq, H // hk, L) * s["scale"]
    del k
    score = score.masked_fill(~seen[:, None, :, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    v = _values(s["v_codes"][pages], s["v_scale"][pages], block).reshape(B, L, hk, D)
    v = torch.where(kept[:, :, None, None], v, 0.0).permute(0, 2, 1, 3)
    out = torch.matmul(p.view(B, hk, -1, L), v).view(B, hk, Lq, H // hk, D)
    out = torch.where(total > 0, out / total, 0.0)
    lse = torch.log(total) + top
    return {"out": out.permute(0, 2, 1, 3, 4).reshape(B, Lq, H, D).to(torch.bfloat16), "lse": lse[..., 0].permute(0, 2, 1, 3).reshape(B, Lq, H)}


def _append_own(s):
    api = _handles(s)
    q = api.rope_append(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["rope"], s["cache"], out=s["out"])
    return {"q": q, **_kept(s, _read_own)}


def _kept(s, read_rows):
    """What the cache holds after an append: read again, or its 8-bit floats, and the scales."""
    held = read_rows(s) if s["case"]["read"] else {"k_codes": s["k_codes"], "v_codes": s["v_codes"]}
    return {**held, "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _append_plain(s):
    c = s["case"]
    D, R, kv, block = c["dim"], c["rotary"], c["kv"], c["block"]
    phase = s["positions"].long()[s["axis"].long()].t() * s["turns"]                 # [T, R/2] fractions of a turn, times 2^64
    angle = (phase >> 32).double() * (2 * math.pi / 2 ** 32)
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]

    def turned(x):
        x = x.float()
        a, b = (x[..., 0:R:2], x[..., 1:R:2]) if s["neighbour"] else (x[..., : R // 2], x[..., R // 2: R])
        a, b = a * cos - b * sin, a * sin + b * cos
        both = torch.stack([a, b], -1).flatten(-2) if s["neighbour"] else torch.cat([a, b], -1)
        return torch.cat([both, x[..., R:]], -1)

    T, (pages, page) = s["q"].shape[0], s["k_codes"].shape[:2]
    blocks = pages * page // block
    slots = s["slots"].long()
    to = torch.where(slots >= 0, slots // block, blocks)                             # block of each row; one more for the rows that are not kept
    first = torch.zeros(blocks + 1, device="cuda").index_reduce_(0, to, (slots % block == 0).float(), "amax")[:-1] > 0
    joined = torch.zeros(blocks + 1, device="cuda").index_reduce_(0, to, torch.ones(T, device="cuda"), "amax")[:-1] > 0
    row = torch.full((pages * page + 1,), -1, device="cuda")                         # the row that each slot takes, if any
    row[torch.where(slots >= 0, slots, pages * page)] = torch.arange(T, device="cuda")
    row = row[:-1].view(pages, page)

    def written(codes, scales, x):
        heads = x.shape[1]
        top = torch.zeros(blocks + 1, heads, device="cuda").index_reduce_(0, to, x.abs().amax(-1), "amax")[:-1]
        before = scales.view(blocks, heads)
        old = torch.where(first[:, None], 0.0, before.clamp(LEAST, MOST))
        scale = torch.where(joined[:, None], torch.maximum(old, _need(top, kv)), before)
        grown = joined[:, None] & (old > 0) & (old < scale)
        each = lambda t: t.view(pages, page // block, heads).repeat_interleave(block, 1)[..., None]  # noqa: E731
        held = torch.where(each(grown), _coded(codes.float() * each(old / scale), kv).float(), codes.float())
        new = _coded(x[row.clamp(min=0)] / each(scale), kv).float()
        codes.copy_(torch.where((row >= 0)[:, :, None, None], new, held).to(codes.dtype))
        scales.copy_(scale.view(scales.shape))

    written(s["k_codes"], s["k_scale"], turned(s["k"]))
    written(s["v_codes"], s["v_scale"], s["v"].float())
    return {"q": turned(s["q"]).to(torch.bfloat16), **_kept(s, _read_plain)}


def _read_own(s):
    api = _handles(s)
    k, v = api.paged_read(s["cache"], s["table"], s["starts"], first=s["first"], k=s["k_rows"], v=s["v_rows"])
    return {"k": k, "v": v}


def _read_plain(s):
    c = s["case"]
    page, block = c["page"], c["block"]
    row = torch.arange(s["k_rows"].shape[0], device="cuda")
    starts = s["starts"].long()
    b = torch.searchsorted(starts[1:], row, right=True).clamp(max=c["batch"] - 1)
    inside = row < starts[-1]
    token = torch.where(inside, s["first"].long()[b] + row - starts[b], 0)
    at = s["table"][b, token // page].long().clamp(min=0)
    place = token % page
    out = []
    for codes, scales, rows in ((s["k_codes"], s["k_scale"], s["k_rows"]), (s["v_codes"], s["v_scale"], s["v_rows"])):
        x = codes[at, place].float() * scales[at, place // block][..., None]
        out.append(torch.where(inside[:, None, None], x.to(torch.bfloat16), rows))
    return {"k": out[0], "v": out[1]}


# ----------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    hk, D, page, block = case["kv_heads"], case["dim"], case["page"], case["block"]
    many = lambda spans, of: sum(-(-(f + n) // of) - f // of for f, n in spans if n)  # noqa: E731  (pages or blocks of some tokens)
    if case["op"] == "attend":
        H, Lq = case["heads"], case["tokens"]
        seen = [(max(0, n - Lq + 1 - case["window"]) if case["window"] else 0, n) for n in _lengths(case)]
        seen = [(a, n - a) for a, n in seen]
        rows = case["batch"] * Lq * H
        pairs = sum(_pairs(n, Lq, case["window"]) for n in _lengths(case))
        return {"bytes": sum(n for _, n in seen) * hk * D * 2 + many(seen, block) * hk * 8 + 4 * many(seen, page) + 4 * case["batch"] + rows * (4 * D + 4),
                "flops": 4 * pairs * H * D}
    back = 0
    if case["op"] == "read" or case["read"]:
        spans = _blocks(case) if case["op"] == "append" else _pieces(case)
        rows = sum(n for _, n in spans)
        back = rows * 4 * hk * D + 4 * many(spans, page) + 8 * case["batch"]
    if case["op"] == "read":
        return {"bytes": back + rows * 2 * hk * D + many(spans, block) * hk * 8, "flops": rows * 2 * hk * D}
    T, hq, kept = _rows(case), case["heads"], sum(n for _, n in _pieces(case))
    return {"bytes": 4 * T * hq * D + kept * 6 * hk * D + many(_pieces(case), block) * hk * 8 + 4 * T * (1 + case["axes"]) + back,
            "flops": 3 * case["rotary"] * (T * hq + kept * hk) + 4 * kept * hk * D}


def _pairs(n, Lq, window):
    """Query-key pairs of a request of n tokens whose last Lq ask."""
    ends = [n - Lq + j + 1 for j in range(Lq)]
    return sum(max(0, min(e, window) if window else e) for e in ends)


# ----------------------------------------------------------------------------- from the definition, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"attend": _attend_exact, "append": _append_exact, "read": _read_exact}[case["op"]](case, s)


def _tokens(s, case, which, b, begin, end, h):
    """Tokens begin .. end - 1 of request b at key head h, float64 [tokens, dim]."""
    page, block = case["page"], case["block"]
    pages = s["table"][b, begin // page: -(-end // page)].long()
    codes = s[which + "_codes"][pages][:, :, h].double()
    scale = s[which + "_scale"][pages][:, :, h].double()
    x = (codes.view(len(pages), page // block, block, -1) * scale[:, :, None, None]).reshape(len(pages) * page, -1)
    return x[begin % page: begin % page + end - begin]


def _attend_exact(case, s):
    B, Lq, H, D = s["q"].shape
    hk = case["kv_heads"]
    G = H // hk
    out = torch.zeros(B, Lq, H, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, Lq, H), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(_lengths(case)):
        if n == 0:
            continue
        for h in range(hk):
            k, v = (_tokens(s, case, x, b, 0, n, h) for x in "kv")
            for j in range(Lq):
                end = n - Lq + j + 1
                begin = max(0, end - case["window"]) if case["window"] else 0
                if end <= begin:
                    continue
                w = s["q"][b, j, h * G: (h + 1) * G].double() @ k[begin:end].t() * s["scale"]
                lse[b, j, h * G: (h + 1) * G] = torch.logsumexp(w, 1)
                out[b, j, h * G: (h + 1) * G] = torch.softmax(w, 1) @ v[begin:end]
    return {"out": out, "lse": lse}


def _append_exact(case, s):
    R, block, kv = case["rotary"], case["block"], case["kv"]
    frequency = 10000.0 ** (-2.0 * torch.arange(R // 2, dtype=torch.float64, device="cuda") / R)
    angle = torch.stack([s["positions"][int(a)].double() * f for a, f in zip(s["axis"].tolist(), frequency)], 1)

    def turned(x):
        x = x.double()
        z = x.clone()
        for i in range(R // 2):
            a, b = (2 * i, 2 * i + 1) if case["pairs"] == "neighbour" else (i, i + R // 2)
            c, d = torch.cos(angle[:, i, None]), torch.sin(angle[:, i, None])
            z[..., a] = x[..., a] * c - x[..., b] * d
            z[..., b] = x[..., b] * c + x[..., a] * d
        return z

    rows = {}
    for t, slot in enumerate(s["slots"].tolist()):
        if slot >= 0:
            rows.setdefault(slot // block, []).append((t, slot % block))
    each = case["page"] // block
    quantised = (lambda x: torch.round(x).clamp(-127, 127)) if kv == "int8" else (lambda x: x.clamp(-448, 448).to(torch.float8_e4m3fn).double())
    held = {}
    for which, x in (("k", turned(s["k"])), ("v", s["v"].double())):
        codes, scales = s[which + "_codes"].double(), s[which + "_scale"].double()
        for at, joined in rows.items():
            p, i = at // each, at % each
            here = codes[p, i * block: (i + 1) * block]
            t, place = (list(z) for z in zip(*joined))
            top = x[t].abs().amax((0, 2))
            need = top / 127
            if kv == "e4m3":
                need = torch.exp2(torch.ceil(torch.log2(top / 448)))
                need = torch.where(need / 2 * 448 >= top, need / 2, need)  # a logarithm just above a whole number
            need = need.clamp(LEAST, MOST)
            old = torch.zeros_like(need) if 0 in place else scales[p, i]
            scale = torch.maximum(old, need)
            if 0 not in place:
                here.copy_(torch.where((old < scale)[:, None], quantised(here * (old / scale)[:, None]), here))
            here[place] = quantised(x[t] / scale[:, None])
            scales[p, i] = scale
        held[which + "_codes"], held[which + "_scale"] = codes, scales
    out = {"q": turned(s["q"]), "k_scale": held["k_scale"], "v_scale": held["v_scale"]}
    return {**out, **(_read_exact(case, {**s, **held}) if case["read"] else {w: held[w] for w in ("k_codes", "v_codes")})}


def _read_exact(case, s):
    spans = _blocks(case) if case["op"] == "append" else _pieces(case)
    out = {}
    for which in "kv":
        rows = s[which + "_rows"].double()
        for b, ((f, n), at) in enumerate(zip(spans, s["starts"].tolist())):
            for h in range(case["kv_heads"]):
                rows[at: at + n, h] = _tokens(s, case, which, b, f, f + n, h)
        out[which] = rows
    return out
