"""Plain 64-bit forms of the paged cache with a scale for each block of tokens and head, for the tests."""
from __future__ import annotations

import math

import torch

import paged_ref

LEAST, MOST = 2.0 ** -48, 2.0 ** 48


def values(codes, scales):
    """codes [pages, page, heads, dim] times scales [pages, blocks, heads], float64."""
    block = codes.shape[1] // scales.shape[1]
    return codes.double() * scales.double().repeat_interleave(block, 1)[..., None]


def need(top, kv):
    """The scale of a block whose largest finite magnitude is `top` (float64)."""
    if kv == "int8":
        return (top / 127).clamp(LEAST, MOST)
    m, e = torch.frexp((top / 448).clamp(LEAST, MOST))
    return torch.ldexp(torch.ones_like(top), e - (m == 0.5).int())


def quantise(x, kv):
    """A pool's worth of values [pages, blocks, block, heads, dim] as codes [pages, page, heads, dim] and scales."""
    scale = need(x.double().abs().amax((2, 4)), kv).float()
    y = x.double() / scale.double()[:, :, None, :, None]
    y = y.round().clamp(-127, 127).to(torch.int8) if kv == "int8" else y.clamp(-448, 448).float().to(torch.float8_e4m3fn)
    return y.flatten(1, 2), scale


def attention(q, k, v, ks, vs, table, lens, scale, window=0):
    """paged_ref.attention of the values, and how far a right kernel may be beyond paged_ref.attention_bounds:
    out, lse, mag, room, what the scales add to a score's error, and the products too small for 11 bits."""
    k64, v64, codes64 = values(k, ks), values(v, vs), v.double()
    out, lse, mag, room = paged_ref.attention(q, k64, v64, table, lens, scale, window)
    B, n, H, D = q.shape
    page, hk = k.shape[1], k.shape[2]
    block, G = page // ks.shape[1], H // hk
    more, small = torch.zeros(B, n, H, dtype=torch.float64), torch.zeros(B, n, H, D, dtype=torch.float64)
    for b in range(B):
        L = int(lens[b])
        if L <= 0:
            continue
        pages = table[b, : -(-L // page)].long()
        for h in range(hk):
            kk = k64[pages][:, :, h].reshape(-1, D)[:L]
            codes = codes64[pages][:, :, h].reshape(-1, D)[:L].abs()
            sv = vs[pages][:, :, h].double().repeat_interleave(block, 1).reshape(-1)[:L]
            for j in range(n):
                end = L - n + j + 1
                begin = max(0, end - window) if window else 0
                if end <= 0:
                    continue
                rows = slice(h * G, (h + 1) * G)
                s = q[b, j, rows].double() @ kk[begin:end].T * scale
                p = torch.softmax(s, 1) * sv[begin:end]
                more[b, j, rows] = (s.abs() * 1.45 + 2 * sv[begin:end].log2().abs()).amax(1)
                small[b, j, rows] = p.amax(1)[:, None] * codes[begin:end].sum(0)
    return out, lse, mag, room, more, small


def attention_bounds(out, lse, mag, room, more, small, dim):
    """paged_ref.attention_bounds with 12 bits (half a step of 11), and on top of it: 2^-38 of the largest product for
    each one; in the exponent, which is the score in log2 plus the scale's logarithm, 2^-24 of either's magnitude for
    each of two roundings and 2^-22 for the logarithm, twice that for its inverse and the exponential (all of them
    approximations to 2^-22)."""
    b_out, b_lse = paged_ref.attention_bounds(out, lse, mag, room, dim, 12)
    exponent = more * 2.0 ** -23 + 2.0 ** -20
    return b_out + small * 2.0 ** -38 + mag * 2 * exponent[..., None], b_lse + exponent


def largest(x):
    """The largest finite magnitude of x [rows, heads, dim] by head."""
    a = x.abs()
    return torch.where(torch.isfinite(a), a, 0.0).amax((0, 2))


class Checker:
    """One append to a cache, checked value by value against the arithmetic that include/affqmm.h states: what the
    cache held before and holds after, and the call's k (turned) and v in 64 bits with `slack`, how far fp32 may be
    from each of them."""

    def __init__(self, kv, block):
        self.kv, self.block = kv, block

    def check(self, before, after, x, slack, slots):
        (c0, s0), (c1, s1) = before, after
        page, kv, block = c0.shape[1], self.kv, self.block
        each = page // block
        c0, c1, s0, s1 = c0.double(), c1.double(), s0.double(), s1.double()
        rows: dict = {}
        for t, slot in enumerate(slots.tolist()):
            if 0 <= slot < c0.shape[0] * page:
                rows.setdefault(slot // block, []).append((t, slot % block))
        untouched = torch.ones(c0.shape[0], each, dtype=torch.bool)
        grown = 0
        for at, joined in rows.items():
            p, i = at // each, at % each
            untouched[p, i] = False
            t, place = (list(z) for z in zip(*joined))
            fresh = 0 in place
            top, off = largest(x[t]), slack[t].nan_to_num(0, 0, 0).amax((0, 2))
            old = torch.zeros_like(top) if fresh else s0[p, i].nan_to_num(LEAST).clamp(LEAST, MOST)
            least, most = (torch.maximum(old, need((top + e).clamp(min=0), kv)) for e in (-off, off))
            scale = s1[p, i]
            assert bool((scale >= least * (1 - 2.0 ** -22)).all()) and bool((scale <= most * (1 + 2.0 ** -22)).all())
            want = x[t] / scale[:, None]
            got = c1[p, i * block: (i + 1) * block]
            room = 2.0 ** -20 * want.abs() + slack[t] / scale[:, None]
            if kv == "int8":
                want = torch.where(torch.isnan(want), 0.0, want).clamp(-127, 127)
                room = torch.where(torch.isfinite(room), room, 0.0) + 0.5
            else:
                lost = torch.isnan(want)
                assert torch.equal(torch.isnan(got[place]), lost)
                want = want.clamp(-448, 448)
                room = torch.maximum(2.0 ** -4 * want.abs(), torch.tensor(2.0 ** -10, dtype=torch.float64)) + room.nan_to_num(0, 0, 0)
            off_by = (got[place] - want).abs()
            assert bool((off_by <= room)[~torch.isnan(off_by)].all())
            others = [j for j in range(block) if j not in place]
            if others:
                was, now = c0[p, i * block: (i + 1) * block][others], got[others]
                for h in range(scale.numel()):
                    if not fresh and old[h] < scale[h]:
                        grown += 1
                        y = was[:, h] * float(old[h] / scale[h])
                        room = torch.full_like(y, 0.5 + 2.0 ** -10) if kv == "int8" else torch.maximum(
                            2.0 ** -4 * y.abs(), torch.tensor(2.0 ** -10, dtype=torch.float64)) * (1 + 2.0 ** -10)
                        nan = torch.isnan(y)
                        assert torch.equal(torch.isnan(now[:, h]), nan) and bool(((now[:, h] - y).abs() <= room)[~nan].all())
                    else:
                        assert torch.equal(now[:, h].nan_to_num(1e9), was[:, h].nan_to_num(1e9))
        whole = untouched.repeat_interleave(block, 1)
        assert torch.equal(c1[whole].nan_to_num(1e9), c0[whole].nan_to_num(1e9))
        assert torch.equal(s1[untouched].nan_to_num(-1), s0[untouched].nan_to_num(-1))
        return grown
