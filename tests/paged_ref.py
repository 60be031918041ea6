"""Plain 64-bit forms of the paged cache's operators, for the tests."""
from __future__ import annotations

import math

import numpy as np
import torch


def turns_of(rotary: int, base: float = 10000.0):
    """Frequencies of the usual rotary embedding, radians a position."""
    return [base ** (-2.0 * i / rotary) for i in range(rotary // 2)]


def attention(q, k, v, table, lens, scale, window=0, k_scale=None, v_scale=None):
    """q [B, n, H, D], k and v [pages, page, heads, D] on the CPU.  Returns out,
    lse, the probability-weighted |v| and the scores' rounding room, float64."""
    B, n, H, D = q.shape
    page, hk = k.shape[1], k.shape[2]
    G = H // hk
    out = torch.zeros(B, n, H, D, dtype=torch.float64)
    mag = torch.zeros(B, n, H, D, dtype=torch.float64)
    lse = torch.full((B, n, H), -math.inf, dtype=torch.float64)
    room = torch.zeros(B, n, H, dtype=torch.float64)
    for b in range(B):
        L = int(lens[b])
        if L == 0:
            continue
        pages = table[b, : -(-L // page)].long()
        for h in range(hk):
            kk = k[pages][:, :, h].reshape(-1, D)[:L].double() * (1.0 if k_scale is None else float(k_scale[h]))
            vv = v[pages][:, :, h].reshape(-1, D)[:L].double() * (1.0 if v_scale is None else float(v_scale[h]))
            for j in range(n):
                end = L - n + j + 1
                begin = max(0, end - window) if window else 0
                if end <= 0:
                    continue
                rows = slice(h * G, (h + 1) * G)
                qq = q[b, j, rows].double()
                s = qq @ kk[begin:end].T * scale
                p = torch.softmax(s, 1)
                out[b, j, rows] = p @ vv[begin:end]
                mag[b, j, rows] = p @ vv[begin:end].abs()
                lse[b, j, rows] = torch.logsumexp(s, 1)
                room[b, j, rows] = (qq.abs() @ kk[begin:end].abs().T * abs(scale)).amax(1)
    return out, lse, mag, room


def attention_bounds(out, lse, mag, room, dim, p_bits):
    """How far a right kernel may be.  Out: one rounding to bf16 (2^-9 of the
    value, doubled for values at a binade's edge); every probability rounded to
    p_bits significant bits (at most 2^-p_bits of the weighted |v|); 2^-11 of it
    for exponentials and scores, whose fp32 sums err by less than `room` (sum of
    |q k|) x dim x 2^-24.  lse: that error of the scores, and 2^-20 of 1 + |lse|
    for the exponentials, the sum and the logarithm."""
    score = room * (dim + 8) * 2.0 ** -24
    b_out = out.abs() * 2.0 ** -8 + mag * (2.0 ** -p_bits + 2.0 ** -11 + 2 * score[..., None])
    b_lse = score + 2.0 ** -20 * (1 + torch.where(torch.isfinite(lse), lse.abs(), 0.0))
    return b_out, b_lse


def rope(x, positions, freqs, axis, neighbour):
    """x [T, H, D] float64; positions [axes, T] ints; returns the turned x."""
    T, R = x.shape[0], 2 * len(freqs)
    pos = positions.long().numpy()
    angle = np.zeros((T, R // 2))
    for i, f in enumerate(freqs):
        # the phase in extended precision: whole turns leave before the float sees them
        turn = int(math.floor(f / (2 * math.pi) * 2.0 ** 64))
        for t in range(T):
            ph = int(pos[int(axis[i]), t]) * turn % (1 << 64)
            angle[t, i] = ph / 2.0 ** 64 * 2 * math.pi
    c, s = torch.from_numpy(np.cos(angle))[:, None], torch.from_numpy(np.sin(angle))[:, None]
    y = x.clone()
    if neighbour:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        y[..., 0:R:2], y[..., 1:R:2] = a * c - b * s, a * s + b * c
    else:
        a, b = x[..., : R // 2], x[..., R // 2: R]
        y[..., : R // 2], y[..., R // 2: R] = a * c - b * s, a * s + b * c
    return y


def plan(lens, fresh, finished, table, ring, ring_state, page, capacity):
    """One step of the page allocator, request by request.  table and ring
    (numpy) are copied; returns a dict of numpy arrays."""
    table, ring = table.copy(), ring.copy()
    before = ring.copy()
    B, wide = table.shape
    pool = ring.size
    head, free = (int(x) for x in ring_state)
    status = 0
    if not (0 <= head < pool and 0 <= free <= pool):
        head = free = 0
        status |= 8
    starts, new_lens = [0], []
    slots, positions, requests = [-1] * capacity, [0] * capacity, [-1] * capacity
    asked = back = taken = 0
    gives = []
    for i in range(B):
        L, n, done = int(lens[i]), int(fresh[i]), bool(finished[i])
        if L < 0 or L > wide * page or (not done and n < 0):
            status |= 8
            starts.append(starts[-1])
            new_lens.append(0 if done else L)
            continue
        if done:
            starts.append(starts[-1])
            new_lens.append(0)
            gives += [(back + j, table[i, j]) for j in range(-(-L // page))]
            back += -(-L // page)
            continue
        first = starts[-1]
        end = first + n
        starts.append(end)
        ok = True
        if L + n > wide * page:
            status |= 2
            ok = False
        if end > capacity:
            status |= 4
            ok = False
        held, want = -(-L // page), -(-(L + n) // page)
        if ok:
            asked += want - held
            if want > held and asked > free:
                status |= 1
                ok = False
        if ok:
            for j in range(held, want):
                table[i, j] = before[(head + asked - (want - held) + j - held) % pool]
            if want > held:
                taken = asked
        new_lens.append(L + n if ok else L)
        for j in range(n):
            t = first + j
            if t >= capacity:
                break
            positions[t], requests[t] = L + j, i
            if ok:
                slots[t] = int(table[i, (L + j) // page]) * page + (L + j) % page
    if free + back > pool:
        status |= 8
        back = 0
    else:
        for j, x in gives:
            ring[(head + free + j) % pool] = x
    arr = lambda x: np.asarray(x, dtype=np.int32)  # noqa: E731
    return {"starts": arr(starts), "lens": arr(new_lens), "slots": arr(slots), "positions": arr(positions),
            "requests": arr(requests), "ring_state": arr([(head + taken) % pool if pool else 0, free - taken + back]),
            "status": arr([status]), "table": table, "ring": ring}
