"""Cases for the paged key-value cache's operators: planning a step, appending to the cache, attending over it.

A decode step of a served model passes, in each layer, from the stacked q/k/v projection to the o projection through

  plan    (once a step)  block tables, slot maps, positions and lengths of the step's tokens, from the requests' lengths
  append  rotary positions on q and k, k and v written to their slots of the paged cache
  attend  attention of each request's newest tokens over its pages

`run` computes an operator either in elementary torch operations (`own` false) or through group_affine_bit_gb300.api.
"""
import math
import random

import numpy as np
import torch

own = False

KV = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
LOG2_PAGES_SPARE = 3  # a pool holds 1/8 more pages than its requests use


# ----------------------------------------------------------------------------- cases
def listed():
    return [
        # One request early in its answer: the shortest call, where latency is all there is.
        attend("attend_one_short", batch=1, longest=577, spread="full", heads=32, kv_heads=8, dim=256, page=16),
        # Ordinary serving: 32 requests of mixed lengths, heads as the 8192-deep output projection has them.
        attend("attend_ordinary", batch=32, longest=4096, spread="ragged", heads=32, kv_heads=8, dim=256, page=16),
        # One reader of a very long document: all the parallelism is in the cache's length.
        attend("attend_one_long", batch=1, longest=262143, spread="full", heads=32, kv_heads=8, dim=128, page=64),
        # The largest: many long requests, bound by the cache's bytes.
        attend("attend_large", batch=64, longest=32768, spread="ragged", heads=32, kv_heads=8, dim=128, page=32),
        # The same kind of load over a cache of 8-bit floats with a scale for each head.
        attend("attend_bytes", batch=96, longest=8192, spread="ragged", heads=32, kv_heads=8, dim=128, page=32, kv="e4m3"),
        # Checking five drafted tokens a request, in a layer with a sliding window, over head-major pages.
        attend("attend_draft_window", batch=12, longest=6000, spread="ragged", heads=32, kv_heads=16, dim=256, page=16,
               tokens=5, window=1024, layout="head"),
        # Odd everything: seven query heads to a key head, 80 values a head, pages of 8, requests of no token and of one.
        attend("attend_odd", batch=19, longest=1501, spread="empty", heads=28, kv_heads=4, dim=80, page=8),
        # A decode step's rows of a few requests.
        append("append_decode", tokens=4, heads=32, kv_heads=8, dim=256, page=16, rotary=256, longest=262144),
        # A prompt with images: three axes (time, height, width) share the head's pairs.
        append("append_prompt", tokens=8192, heads=32, kv_heads=8, dim=128, page=64, rotary=128, axes=3, longest=32768),
        # Part of the head turns, neighbouring values make the pairs, 8-bit cache, padded rows.
        append("append_odd", tokens=1333, heads=28, kv_heads=4, dim=80, page=8, rotary=40, axes=2, pairs="neighbour",
               kv="e4m3", longest=131072, padded=True),
        # A decode step of 64 requests.
        plan("plan_decode", batch=64, longest=8192, most=1, page=16),
        # A server's mixed step: 2048 requests, some with prompts, some that have finished.
        plan("plan_mixed", batch=2048, longest=16384, most=512, page=32),
    ]


def draw(rng):
    """One more case of the same ranges."""
    kind = rng.choice(["attend", "attend", "attend", "append", "plan"])
    heads, kv_heads = rng.choice([(32, 8), (32, 16), (32, 4), (28, 4), (16, 16), (16, 1), (8, 2), (40, 8), (6, 2)])
    dim = rng.choice([64, 80, 96, 128, 128, 256, 256, 512])
    page = rng.choice([8, 16, 32, 64, 128])
    kv = rng.choice(["bf16", "bf16", "e4m3"])
    if kind == "attend":
        tokens = rng.choice([1, 1, 1, 2, 5, 8])
        batch = _log(rng, 1, 128)
        # what the largest listed case's cache can hold, shared out
        room = 64 * 32768 * 8 * 128 // (batch * kv_heads * dim)
        longest = _log(rng, 64, max(65, min(262144, room)))
        window = rng.choice([0, 0, 0, 512, 1024, 4096])
        spread = rng.choice(["full", "ragged", "ragged", "empty"])
        return attend("", batch, longest, spread, heads, kv_heads, dim, page, kv, tokens, window, rng.choice(["token", "head"]))
    if kind == "append":
        tokens = _log(rng, 1, 8192 * 128 * 48 // (dim * (heads + 2 * kv_heads)))
        rotary = rng.choice([dim, dim, dim // 2])
        return append("", tokens, heads, kv_heads, dim, page, rotary, rng.choice([1, 1, 2, 3]), rng.choice(["half", "half", "neighbour"]),
                      kv, _log(rng, 8192, 262144), rng.choice([False, True]))
    most = rng.choice([1, 1, 4, 64, 512])
    return plan("", _log(rng, 1, 2048), _log(rng, 512, 16384), most, page)


def _log(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def attend(name, batch, longest, spread, heads, kv_heads, dim, page, kv="bf16", tokens=1, window=0, layout="token"):
    case = dict(op="attend", batch=batch, longest=longest, spread=spread, heads=heads, kv_heads=kv_heads, dim=dim, page=page, kv=kv,
                tokens=tokens, window=window, layout=layout)
    return {"name": name, **case} if name else case


def append(name, tokens, heads, kv_heads, dim, page, rotary, axes=1, pairs="half", kv="bf16", longest=8192, padded=False):
    case = dict(op="append", tokens=tokens, heads=heads, kv_heads=kv_heads, dim=dim, page=page, rotary=rotary, axes=axes, pairs=pairs, kv=kv,
                longest=longest, padded=padded)
    return {"name": name, **case} if name else case


def plan(name, batch, longest, most, page):
    case = dict(op="plan", batch=batch, longest=longest, most=most, page=page)
    return {"name": name, **case} if name else case


def _of(case):
    """A generator that the case alone decides, for its requests' lengths."""
    return random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))


def _lengths(case):
    """Tokens in the cache of each request, the step's own included."""
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


def _steps(case):
    """plan: (cached tokens, new tokens, finished) of each request."""
    rng = _of(case)
    cached, new, done = [], [], []
    for i in range(case["batch"]):
        n = 1 if case["most"] == 1 or rng.random() < 0.7 else rng.randint(0, case["most"])
        cached.append(rng.randint(0, max(0, case["longest"] - n)))
        new.append(n)
        done.append(rng.random() < 0.03)
    return cached, new, done


# ----------------------------------------------------------------------------- what a program has in hand
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _cache(case, pages, g):
    """k and v [page, token, head, value] of the pool, in either order in memory, and their scales."""
    shape = (pages, case["page"], case["kv_heads"], case["dim"])
    if case.get("layout") == "head":
        shape = (shape[0], shape[2], shape[1], shape[3])
    out = []
    for _ in "kv":
        t = torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
        if case["kv"] == "e4m3":
            t = t.mul_(32).to(torch.float8_e4m3fn)
        out.append(t.transpose(1, 2) if case.get("layout") == "head" else t)
    scales = [None, None]
    if case["kv"] == "e4m3":
        scales = [(torch.rand(case["kv_heads"], device="cuda", generator=g) + 0.5) / 32 for _ in "kv"]
    return out[0], out[1], scales[0], scales[1]


def _tables(used, page, wide, pool, g):
    """Block tables [request, wide] of requests that use `used` pages each, taken from a shuffled pool; the pages left over."""
    order = torch.randperm(pool, device="cuda", generator=g).to(torch.int32)
    n = torch.tensor(used, device="cuda", dtype=torch.int64)
    at = (torch.cumsum(n, 0) - n)[:, None] + torch.arange(wide, device="cuda")[None]
    held = torch.arange(wide, device="cuda")[None] < n[:, None]
    return torch.where(held, order[at.clamp(max=pool - 1)], -1).contiguous(), order[int(sum(used)):]


def prepare(case, seed):
    g = _generator(seed)
    state = {"case": case}
    if case["op"] == "attend":
        lens = _lengths(case)
        used = [-(-n // case["page"]) for n in lens]
        pool = sum(used) + (sum(used) >> LOG2_PAGES_SPARE) + 1
        k, v, ks, vs = _cache(case, pool, g)
        wide = -(-case["longest"] // case["page"])
        table, _ = _tables(used, case["page"], wide, pool, g)
        shape = (case["batch"], case["tokens"], case["heads"], case["dim"])
        state.update(k=k, v=v, k_scale=ks, v_scale=vs, table=table, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                     q=torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(generator=g), scale=case["dim"] ** -0.5,
                     out=torch.empty(shape, dtype=torch.bfloat16, device="cuda"),
                     lse=torch.empty(shape[:3], dtype=torch.float32, device="cuda"))
    elif case["op"] == "append":
        T, hq, hk, D = case["tokens"], case["heads"], case["kv_heads"], case["dim"]
        pool = -(-T // case["page"]) + 3
        k, v, ks, vs = _cache(case, pool, g)
        qkv = torch.empty(T, (hq + 2 * hk) * D, dtype=torch.bfloat16, device="cuda").normal_(generator=g)  # the stacked projection's rows
        first = torch.randint(0, case["longest"], (1,), device="cuda", generator=g)
        positions = first + torch.arange(T, device="cuda") if T > 64 else torch.randint(0, case["longest"], (T,), device="cuda", generator=g)
        if case["axes"] > 1:  # an image's rows and columns behind its place in time
            side = 37
            grid = [positions // (side * side)] + [positions // side % side, positions % side][: case["axes"] - 1]
            positions = torch.stack([grid[0]] + [first + x for x in grid[1:]])
        else:
            positions = positions[None]
        slots = torch.randperm(pool * case["page"], device="cuda", generator=g)[:T]
        if case["padded"]:  # the last rows of a captured step's fixed capacity
            slots[T - T // 8:] = -1
        half = case["rotary"] // 2
        state.update(k_cache=k, v_cache=v, k_scale=ks, v_scale=vs, positions=positions.to(torch.int32).contiguous(), slots=slots.to(torch.int32),
                     q=qkv[:, : hq * D].view(T, hq, D), k=qkv[:, hq * D: (hq + hk) * D].view(T, hk, D), v=qkv[:, (hq + hk) * D:].view(T, hk, D),
                     turns=torch.from_numpy(_turns(case["rotary"]).view(np.int64)).cuda(), neighbour=case["pairs"] == "neighbour",
                     axis=torch.tensor([i * case["axes"] // half for i in range(half)], dtype=torch.uint8, device="cuda"),
                     out=torch.empty(T, hq, D, dtype=torch.bfloat16, device="cuda"))
    else:
        cached, new, done = _steps(case)
        page = case["page"]
        used = [-(-n // page) for n in cached]
        need = sum(-(-(c + n) // page) + 1 for c, n in zip(cached, new))
        wide = -(-case["longest"] // page)
        table, left = _tables(used, page, wide, need + 7, g)
        ring = torch.full((need + 7,), -1, dtype=torch.int32, device="cuda")
        head = seed % (need + 7)
        ring[(head + torch.arange(left.numel(), device="cuda")) % (need + 7)] = left
        total = sum(n for n, d in zip(new, done) if not d)
        state.update(table=table, ring=ring, ring_state=torch.tensor([head, left.numel()], dtype=torch.int32, device="cuda"),
                     lens=torch.tensor(cached, dtype=torch.int32, device="cuda"), new=torch.tensor(new, dtype=torch.int32, device="cuda"),
                     finished=torch.tensor(done, dtype=torch.bool, device="cuda"), page=page, capacity=-(-total // 64) * 64 + 64)
    return state


def _turns(rotary):
    """Turns that each pair makes a position, 10000^(-2i/rotary) / 2 pi, as 64-bit fractions of a turn."""
    f = 10000.0 ** (-2.0 * np.arange(rotary // 2) / rotary) / (2 * math.pi)
    return np.floor(f * 2.0 ** 64).astype(np.uint64)


# ----------------------------------------------------------------------------- one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return {"attend": _attend_own, "append": _append_own, "plan": _plan_own}[op](state)
    return {"attend": _attend_plain, "append": _append_plain, "plan": _plan_plain}[op](state)


def _attend_own(s):
    from group_affine_bit_gb300 import api
    if "cache" not in s:  # the handle that a program keeps beside its pool
        s["cache"] = api.KVCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
    out = api.paged_attention(s["q"], s["cache"], s["table"], s["lens"], scale=s["scale"], window=s["case"]["window"], out=s["out"], lse=s["lse"])
    return {"out": out, "lse": s["lse"]}


def _attend_plain(s):
    c = s["case"]
    B, Lq, H, D = s["q"].shape
    hk, page = c["kv_heads"], c["page"]
    L = s["table"].shape[1] * page
    pages = s["table"].clamp(min=0).long()
    key = torch.arange(L, device="cuda")
    kept = key[None] < s["lens"][:, None]                                            # [B, L]
    last = s["lens"].long()[:, None] - Lq + torch.arange(Lq, device="cuda")[None]    # position of each query
    seen = kept[:, None] & (key[None, None] <= last[:, :, None])
    if c["window"]:
        seen &= key[None, None] > last[:, :, None] - c["window"]
    k = s["k"][pages].reshape(B, L, hk, D).float()
    if s["k_scale"] is not None:
        k *= s["k_scale"][:, None]
    q = s["q"].float().view(B, Lq, hk, H // hk, D).permute(0, 2, 1, 3, 4).reshape(B, hk, -1, D)
    score = torch.matmul(q, k.permute(0, 2, 3, 1)).view(B, hk, Lq, H // hk, L) * s["scale"]
    del k
    score = score.masked_fill(~seen[:, None, :, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    v = s["v"][pages].reshape(B, L, hk, D).float()
    if s["v_scale"] is not None:
        v *= s["v_scale"][:, None]
    v = torch.where(kept[:, :, None, None], v, 0.0).permute(0, 2, 1, 3)
    out = torch.matmul(p.view(B, hk, -1, L), v).view(B, hk, Lq, H // hk, D)
    out = torch.where(total > 0, out / total, 0.0)
    lse = torch.log(total) + top
    return {"out": out.permute(0, 2, 1, 3, 4).reshape(B, Lq, H, D).to(torch.bfloat16), "lse": lse[..., 0].permute(0, 2, 1, 3).reshape(B, Lq, H)}


def _append_own(s):
    from group_affine_bit_gb300 import api
    if "cache" not in s:
        s["cache"] = api.KVCache(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
        s["rope"] = api.Rope(s["turns"], s["axis"], neighbour=s["neighbour"])
    out = api.rope_append(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["rope"], s["cache"], out=s["out"])
    return {"q": out, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _append_plain(s):
    D, R = s["q"].shape[2], 2 * s["turns"].numel()
    phase = s["positions"].long()[s["axis"].long()].t() * s["turns"]                 # [T, R/2] fractions of a turn, times 2^64
    angle = (phase >> 32).float() * (2 * math.pi / 2 ** 32)
    cos, sin = torch.cos(angle)[:, None], torch.sin(angle)[:, None]

    def turned(x):
        x = x.float()
        a, b = (x[..., 0:R:2], x[..., 1:R:2]) if s["neighbour"] else (x[..., : R // 2], x[..., R // 2: R])
        a, b = a * cos - b * sin, a * sin + b * cos
        both = torch.stack([a, b], -1).flatten(-2) if s["neighbour"] else torch.cat([a, b], -1)
        return torch.cat([both, x[..., R:]], -1)

    def written(cache, x, scale):
        x = (x if scale is None else (x / scale[:, None]).clamp(-448, 448)).to(cache.dtype).float()
        cache.copy_(torch.where(kept, x[row.clamp(min=0)], cache.float()).to(cache.dtype))

    T, (pages, page) = s["q"].shape[0], s["k_cache"].shape[:2]
    row = torch.full((pages * page + 1,), -1, device="cuda")                         # the row that each slot takes, if any
    row[torch.where(s["slots"] >= 0, s["slots"].long(), pages * page)] = torch.arange(T, device="cuda")
    row = row[:-1].view(pages, page)
    kept = (row >= 0)[:, :, None, None]
    written(s["k_cache"], turned(s["k"]), s["k_scale"])
    written(s["v_cache"], s["v"].float(), s["v_scale"])
    return {"q": turned(s["q"]).to(torch.bfloat16), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plan_own(s):
    from group_affine_bit_gb300 import api
    if "step" not in s:
        s["step"] = api.PagedStep.empty(s["lens"].numel(), s["capacity"], s["lens"].device)
    step = api.paged_plan(s["lens"], s["new"], s["finished"], s["table"], s["ring"], s["ring_state"], s["page"], out=s["step"])
    return {"starts": step.starts, "lens": step.lens, "slots": step.slots, "positions": step.positions, "requests": step.requests,
            "ring_state": step.ring_state, "status": step.status, "table": s["table"], "ring": s["ring"]}


def _plan_plain(s):
    page, cap, wide, pool = s["page"], s["capacity"], s["table"].shape[1], s["ring"].numel()
    head, free = s["ring_state"].long()
    lens, done = s["lens"].long(), s["finished"]
    new = torch.where(done, 0, s["new"].long())
    held, wanted = (lens + page - 1) // page, (lens + new + page - 1) // page
    ends = torch.cumsum(new, 0)
    fits = ~done & (lens + new <= wide * page) & (ends <= cap)
    need = torch.where(fits, wanted - held, 0)
    last = torch.cumsum(need, 0)
    served = fits & ((need == 0) | (last <= free))
    got = torch.where(served, need, 0)
    first = last - need
    back = torch.where(done, held, 0)
    back_first = torch.cumsum(back, 0) - back
    column = torch.arange(wide, device="cuda")[None]
    # a finished request's pages go behind the free ones, a served one's new pages come from the front
    at = (head + free + back_first[:, None] + column) % pool
    gives = done[:, None] & (column < held[:, None])
    ring = torch.cat([s["ring"], s["ring"][:1]])
    ring[torch.where(gives, at, pool)] = torch.where(gives, s["table"], 0)
    ring = ring[:pool]
    takes = served[:, None] & (column >= held[:, None]) & (column < wanted[:, None])
    table = torch.where(takes, s["ring"][(head + first[:, None] + column - held[:, None]) % pool], s["table"])
    token = torch.arange(cap, device="cuda")
    request = torch.searchsorted(ends, token, right=True)
    inside = request < lens.numel()
    request = request.clamp(max=lens.numel() - 1)
    place = lens[request] + token - (ends - new)[request]
    slot = table[request, (place // page).clamp(max=wide - 1)].long() * page + place % page
    slot = torch.where(inside & served[request], slot, -1)
    whole = lambda t: t.to(torch.int32)  # noqa: E731
    return {"starts": whole(torch.cat([ends[:1] * 0, ends])), "lens": whole(torch.where(done, 0, lens + torch.where(served, new, 0))), "slots": whole(slot),
            "positions": whole(torch.where(inside, place, 0)), "requests": whole(torch.where(inside, request, -1)),
            "ring_state": whole(torch.stack([(head + got.sum()) % pool, free - got.sum() + back.sum()])),
            "status": whole((fits & ~served).any().long() + 2 * (~done & (lens + new > wide * page)).any().long()
                            + 4 * (~done & (ends > cap)).any().long())[None],
            "table": table, "ring": ring}


# ----------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    if case["op"] == "attend":
        hk, D, H, Lq = case["kv_heads"], case["dim"], case["heads"], case["tokens"]
        size = 1 if case["kv"] == "e4m3" else 2
        seen = [n - max(0, n - Lq + 1 - case["window"]) if case["window"] else n for n in _lengths(case)]
        rows = case["batch"] * Lq * H
        pairs = sum(_pairs(n, Lq, case["window"]) for n in _lengths(case))
        return {"bytes": sum(seen) * hk * D * 2 * size + 4 * sum(-(-n // case["page"]) for n in seen) + 4 * case["batch"] + rows * (4 * D + 4),
                "flops": 4 * pairs * H * D}
    if case["op"] == "append":
        T, hq, hk, D = case["tokens"], case["heads"], case["kv_heads"], case["dim"]
        kept = T - T // 8 if case["padded"] else T
        size = 1 if case["kv"] == "e4m3" else 2
        return {"bytes": 4 * T * hq * D + kept * 2 * hk * D * (2 + size) + 4 * T * (1 + case["axes"]), "flops": 3 * case["rotary"] * (T * hq + kept * hk)}
    cached, new, done = _steps(case)
    page = case["page"]
    tokens = sum(n for n, d in zip(new, done) if not d)
    moved = sum(-(-c // page) if d else -(-(c + n) // page) - c // page for c, n, d in zip(cached, new, done))
    return {"bytes": 17 * case["batch"] + 12 * (tokens + 64) + 8 * moved, "flops": 8 * tokens + 16 * case["batch"]}


def _pairs(n, Lq, window):
    """Query-key pairs of a request of n tokens whose last Lq ask."""
    ends = [n - Lq + j + 1 for j in range(Lq)]
    return sum(max(0, min(e, window) if window else e) for e in ends)


# ----------------------------------------------------------------------------- from the definition, in 64 bits
def exact(case, seed):
    if case["op"] == "plan":
        return None  # whole numbers
    s = prepare(case, seed)
    return _attend_exact(case, s) if case["op"] == "attend" else _append_exact(case, s)


def _attend_exact(case, s):
    B, Lq, H, D = s["q"].shape
    hk = case["kv_heads"]
    G = H // hk
    out = torch.zeros(B, Lq, H, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, Lq, H), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(_lengths(case)):
        if n == 0:
            continue
        pages = s["table"][b, : -(-n // case["page"])].long()
        for h in range(hk):
            k = s["k"][pages][:, :, h].reshape(-1, D)[:n].double()
            v = s["v"][pages][:, :, h].reshape(-1, D)[:n].double()
            if s["k_scale"] is not None:
                k, v = k * s["k_scale"][h].double(), v * s["v_scale"][h].double()
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
    R = case["rotary"]
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

    caches = []
    for cache, x, scale in ((s["k_cache"], turned(s["k"]), s["k_scale"]), (s["v_cache"], s["v"].double(), s["v_scale"])):
        cache = cache.double()
        for t, slot in enumerate(s["slots"].tolist()):
            if slot >= 0:
                cache[slot // case["page"], slot % case["page"]] = x[t] if scale is None else (x[t] / scale[:, None].double()).clamp(-448, 448)
        caches.append(cache)
    return {"q": turned(s["q"]), "k_cache": caches[0], "v_cache": caches[1]}
