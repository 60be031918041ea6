// block_append.cu -- rotary positions on a step's q and k, and k and v
// quantised as they are written to a cache with a scale for each block of
// tokens and key head (include/affqmm.h states the arithmetic):
//
//     top = max |x| of the call's tokens of the block, x = k turned, or v
//     scale = max(old, top / 127) or, e4m3, max(old, 2^ceil(log2(top / 448)))
//     code = round(x / scale), and the block's other codes times old / scale
//
// Every value of a block waits for the largest of them, so the rows that a call
// brings for a block are one team's work, for one key head and k or v: it reads
// them once, keeps them in registers as they are (two or four chunks of 16 values
// a thread), turns them for the maximum and once more for the codes.  A team is 1
// to 256 threads: as many as hold its rows, and more where a CTA's teams would
// leave threads without work (one token of 128 values: 8 threads or more; a block
// of 64 tokens: 128 or 256).  A row whose predecessor in the call lies in the same
// block belongs to that row's team, so no two CTAs write one block; every CTA
// finds from the slots which rows of its own begin one and how many follow.
//
// A block's scale only grows, and with it the codes that are there are rounded
// again, so a scale is as tight as its block's largest value.  e4m3 scales are
// powers of two: growth then only shifts exponents, and codes lose bits below the
// normal ones alone.
//
// One launch has CTAs for k and v, which come first, for q (up to four tokens, a
// chunk of each to a thread) and, with a status word, a few that look whether each
// block's tokens come one after another.  Sines are made once a CTA, from the
// nearest quarter of a turn.  Bound by memory and, nearly as much, by the way of a
// CTA from its slots to its codes (24 warps an SM; issue slots 61 % taken for a
// chunk of prompts; 44 to 56 bytes of spill beside 80 registers where values lie in
// runs or neighbours pair): measured (GB300, device time) 25.8 us for 5456 tokens
// of 32 + 2 x 8 heads of 128, e4m3, 123 MB, 71 % of the copy rate (68 us with a warp
// to a block and the rows as fp32; 33 with them as read; 30 with several tokens of q
// to a CTA); 29 us for 6210 tokens with a scale for each (81 with a warp to each);
// 3.3 to 3.5 us for a decode step of 64 tokens, 4.2 to 4.9 while its blocks grow.
// Two CTAs an SM instead of three are 15 to 20 % slower, four (64 registers) no
// faster; loads and stores that leave L2 first, packed fp32 arithmetic, and CTAs of
// k and v spread among those of q changed nothing.
#include <type_traits>

#include "affqmm_internal.h"
#include "affqmm_paged.h"
#include "rope_pieces.cuh"

namespace affqmm {
namespace {

constexpr int BA_THREADS = 256, BA_WARPS = BA_THREADS / 32;
constexpr int Q_TOKENS = 4;              // tokens of q to a CTA, at most
// Most shared memory for sines: 2176 / ceil(rotary / 16) tokens', where a block's and the CTA's rows before it are up to 128 + 15.
// Too few in long calls from rotary 242 on for blocks of 128 (136 of 143) and 434 on for blocks of 64 (68 of 79 at 512).
constexpr size_t BA_TABLE = 136 << 10;

// How a head's values pair: HALVES i with i + rotary / 2, where values lie in
// aligned runs of 8 (rotary a multiple of 16), 4 (of 8) or 1; NEIGHBOURS 2i
// with 2i + 1.
enum Pairs { NEIGHBOURS = 0, HALVES_1 = 1, HALVES_4 = 4, HALVES_8 = 8 };

// Eight pairs of a head: chunk c has the pairs 8c .. 8c + 7, where values that do not turn are pairs of neighbours
// (HALVES: of one run and the next).  Raw: as they are read.
struct Raw {
    uint4 a, b;
};
struct Chunk {
    float a[8], b[8];
};

// Where the two runs that begin with pair i begin (HALVES).
template <int RUN>
__device__ __forceinline__ void runs_of(int i, int half, int& d0, int& d1) {
    const bool turns = i < half;
    d0 = turns ? i : 2 * i;                         // 2 half + 2 (i - half)
    d1 = d0 + (turns ? half : RUN);
}

template <int PAIRS>
__device__ __forceinline__ Raw load_chunk(const uint16_t* src, int c, int half) {
    Raw x;
    if constexpr (PAIRS == NEIGHBOURS) {
        x.a = *reinterpret_cast<const uint4*>(src + 16 * c);
        x.b = *reinterpret_cast<const uint4*>(src + 16 * c + 8);
    } else if constexpr (PAIRS == HALVES_8) {
        int d0, d1;
        runs_of<8>(8 * c, half, d0, d1);
        x.a = *reinterpret_cast<const uint4*>(src + d0);
        x.b = *reinterpret_cast<const uint4*>(src + d1);
    } else if constexpr (PAIRS == HALVES_4) {
        int d0, d1;
        runs_of<4>(8 * c, half, d0, d1);
        const uint2 a = *reinterpret_cast<const uint2*>(src + d0), b = *reinterpret_cast<const uint2*>(src + d1);
        runs_of<4>(8 * c + 4, half, d0, d1);
        const uint2 e = *reinterpret_cast<const uint2*>(src + d0), f = *reinterpret_cast<const uint2*>(src + d1);
        x.a = make_uint4(a.x, a.y, e.x, e.y);
        x.b = make_uint4(b.x, b.y, f.x, f.y);
    } else {
        uint32_t a[8], b[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            int d0, d1;
            runs_of<1>(8 * c + e, half, d0, d1);
            a[e] = src[d0], b[e] = src[d1];
        }
        x.a = make_uint4(a[0] | a[1] << 16, a[2] | a[3] << 16, a[4] | a[5] << 16, a[6] | a[7] << 16);
        x.b = make_uint4(b[0] | b[1] << 16, b[2] | b[3] << 16, b[4] | b[5] << 16, b[6] | b[7] << 16);
    }
    return x;
}
template <int PAIRS>
__device__ __forceinline__ void unpack(const Raw& r, Chunk& x) {
    if constexpr (PAIRS == NEIGHBOURS) {
        const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) x.a[e] = bf_lo(w[e]), x.b[e] = bf_hi(w[e]);
    } else {
        unpack8(r.a, x.a);
        unpack8(r.b, x.b);
    }
}

// The sine and cosine by which pair i of token t turns, from an eighth of a turn at most: its 2^-32 of a turn then
// has 24 bits down to 2^-27 of one, so that a value seldom falls to the other side of a code's border.
__device__ __forceinline__ void near_turn_of(const RopeParams& p, int64_t t, int i, float* sine, float* cosine) {
    const int a = p.axis ? min((int)p.axis[i], p.axes - 1) : 0;
    const int64_t pos = p.positions[a * p.pos_stride + t];
    const uint32_t phase = (uint32_t)(((uint64_t)pos * (uint64_t)p.turns[i]) >> 32);   // of a turn, times 2^32
    const uint32_t quarter = (phase + 0x20000000u) >> 30;
    float s, c;
    sincospif((float)(int32_t)(phase - (quarter << 30)) * 0x1p-31f, &s, &c);
    if (quarter & 1u) {
        const float x = s;
        s = c, c = -x;
    }
    *sine = quarter & 2u ? -s : s;
    *cosine = quarter & 2u ? -c : c;
}

// A token's table of sines, of `groups` = ceil(rotary / 16) chunks: the cosines of a chunk's first four pairs, chunk behind
// chunk, then those of its last four, then the sines in the same way, so that neighbouring lanes read neighbouring words.
__device__ __forceinline__ int cosine_at(int pair, int groups) { return (pair >> 2 & 1) * 4 * groups + (pair >> 3) * 4 + (pair & 3); }
__device__ __forceinline__ void put_sines(const RopeParams& p, int64_t t, int pair, int groups, float* row) {
    float* at = row + cosine_at(pair, groups);
    near_turn_of(p, t, pair, at + 8 * groups, at);
}
// Chunk c turned by it.
template <int PAIRS>
__device__ __forceinline__ void turn_chunk(Chunk& x, int c, int half, int groups, const float* row) {
    if (8 * c >= half) return;
    float co[8], si[8];
#pragma unroll
    for (int e = 0; e < 8; e += 4) {                // pairs that do not turn: whatever is there
        const float4 u = *reinterpret_cast<const float4*>(row + (e + 0) * groups + 4 * c), w = *reinterpret_cast<const float4*>(row + (e + 8) * groups + 4 * c);
        co[e] = u.x, co[e + 1] = u.y, co[e + 2] = u.z, co[e + 3] = u.w;
        si[e] = w.x, si[e + 1] = w.y, si[e + 2] = w.z, si[e + 3] = w.w;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        if (PAIRS != HALVES_8 && 8 * c + e >= half) continue;
        const float a = x.a[e], b = x.b[e];
        x.a[e] = a * co[e] - b * si[e];
        x.b[e] = a * si[e] + b * co[e];
    }
}
__device__ __forceinline__ void turn_chunk_far(const RopeParams& p, Chunk& x, int64_t t, int c, int half) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        if (8 * c + e >= half) continue;
        float si, co;
        near_turn_of(p, t, 8 * c + e, &si, &co);
        const float a = x.a[e], b = x.b[e];
        x.a[e] = a * co - b * si;
        x.b[e] = a * si + b * co;
    }
}

// Four values times `by` as codes.
template <bool I8>
__device__ __forceinline__ uint32_t codes4(float x, float y, float z, float w, float by) {
    if constexpr (I8) {
        auto one = [&](float v) { return (uint32_t)max(-127, min(127, __float2int_rn(v * by))) & 0xffu; };   // NaN: 0
        return one(x) | one(y) << 8 | one(z) << 16 | one(w) << 24;
    } else {
        return e4m3x2(x * by, y * by) | e4m3x2(z * by, w * by) << 16;
    }
}
template <bool I8>
__device__ __forceinline__ void values4(uint32_t w, float (&x)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t c = w >> (8 * i) & 0xffu;
        if constexpr (I8) x[i] = (float)(int8_t)c;
        else x[i] = __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)c, __NV_E4M3)));
    }
}

template <int PAIRS, bool I8>
__device__ __forceinline__ void store_codes(uint8_t* dst, int c, int half, const Chunk& x, float by) {
    if constexpr (PAIRS == NEIGHBOURS) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = codes4<I8>(x.a[2 * i], x.b[2 * i], x.a[2 * i + 1], x.b[2 * i + 1], by);
        *reinterpret_cast<uint4*>(dst + 16 * c) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
        uint32_t a[2], b[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            a[i] = codes4<I8>(x.a[4 * i], x.a[4 * i + 1], x.a[4 * i + 2], x.a[4 * i + 3], by);
            b[i] = codes4<I8>(x.b[4 * i], x.b[4 * i + 1], x.b[4 * i + 2], x.b[4 * i + 3], by);
        }
#pragma unroll
        for (int i = 0; i < 8; i += PAIRS) {
            int d0, d1;
            runs_of<PAIRS>(8 * c + i, half, d0, d1);
            if constexpr (PAIRS == HALVES_8) {
                *reinterpret_cast<uint2*>(dst + d0) = make_uint2(a[0], a[1]);
                *reinterpret_cast<uint2*>(dst + d1) = make_uint2(b[0], b[1]);
            } else if constexpr (PAIRS == HALVES_4) {
                *reinterpret_cast<uint32_t*>(dst + d0) = a[i >> 2];
                *reinterpret_cast<uint32_t*>(dst + d1) = b[i >> 2];
            } else {
                dst[d0] = (uint8_t)(a[i >> 2] >> (8 * (i & 3)));
                dst[d1] = (uint8_t)(b[i >> 2] >> (8 * (i & 3)));
            }
        }
    }
}
template <int PAIRS>
__device__ __forceinline__ void store_bf16(uint16_t* dst, int c, int half, const Chunk& x) {
    if constexpr (PAIRS == NEIGHBOURS) {
        *reinterpret_cast<uint4*>(dst + 16 * c) = make_uint4(bf2(x.a[0], x.b[0]), bf2(x.a[1], x.b[1]), bf2(x.a[2], x.b[2]), bf2(x.a[3], x.b[3]));
        *reinterpret_cast<uint4*>(dst + 16 * c + 8) = make_uint4(bf2(x.a[4], x.b[4]), bf2(x.a[5], x.b[5]), bf2(x.a[6], x.b[6]), bf2(x.a[7], x.b[7]));
    } else {
        uint32_t a[4], b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = bf2(x.a[2 * i], x.a[2 * i + 1]), b[i] = bf2(x.b[2 * i], x.b[2 * i + 1]);
#pragma unroll
        for (int i = 0; i < 8; i += PAIRS) {
            int d0, d1;
            runs_of<PAIRS>(8 * c + i, half, d0, d1);
            if constexpr (PAIRS == HALVES_8) {
                *reinterpret_cast<uint4*>(dst + d0) = make_uint4(a[0], a[1], a[2], a[3]);
                *reinterpret_cast<uint4*>(dst + d1) = make_uint4(b[0], b[1], b[2], b[3]);
            } else if constexpr (PAIRS == HALVES_4) {
                *reinterpret_cast<uint2*>(dst + d0) = make_uint2(a[i >> 1], a[(i >> 1) + 1]);
                *reinterpret_cast<uint2*>(dst + d1) = make_uint2(b[i >> 1], b[(i >> 1) + 1]);
            } else {
                dst[d0] = (uint16_t)(a[i >> 1] >> (16 * (i & 1)));
                dst[d1] = (uint16_t)(b[i >> 1] >> (16 * (i & 1)));
            }
        }
    }
}

// The largest finite magnitude of a chunk.
__device__ __forceinline__ float top_of(const Chunk& x) {
    float m = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = fmaxf(m, fmaxf(fabsf(x.a[e]), fabsf(x.b[e])));   // NaN does not count
    if (m == __int_as_float(0x7f800000)) {
        m = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (fabsf(x.a[e]) < __int_as_float(0x7f800000)) m = fmaxf(m, fabsf(x.a[e]));
            if (fabsf(x.b[e]) < __int_as_float(0x7f800000)) m = fmaxf(m, fabsf(x.b[e]));
        }
    }
    return m;
}

// The scale that a block whose largest magnitude is `top` needs.
template <bool I8>
__device__ __forceinline__ float scale_for(float top) {
    float s;
    if constexpr (I8) {
        s = __fdiv_rn(top, 127.f);
    } else {
        // 448 = 1.75 x 2^8: the power of two at or above top / 1.75, over 2^8
        const uint32_t w = __float_as_uint(fmaxf(top, 0x1p-100f)) + 0x1fffffu;
        s = __uint_as_float((w & 0x7f800000u) - (8u << 23));
    }
    return fminf(fmaxf(s, kLeastScale), kMostScale);
}

struct Grid {
    int kv_ctas, rows;                   // of k and v: CTAs, rows of the call to a CTA
    int order_ctas, order_words;         // that look whether each block's tokens come one after another, and the words of their tables
    int parts, least_parts;              // CTAs that may share k's (v's) heads, and that do so in any case
    int q_tokens, q_parts;               // of q: tokens to a CTA, or (one token) CTAs that share its heads
    int table_rows;                      // rows whose sines shared memory holds
    int chunks;                          // of a head
    int groups;                          // chunks of a head that turn, the last perhaps in part
    uint32_t m_chunks, m_half, m_parts, m_q_parts;
};

// The threads that share a block's rows: `threads`, a power of two, the `index`-th of the CTA's teams.
struct Team {
    int threads, index;
    __device__ __forceinline__ int thread() const { return (int)threadIdx.x & (threads - 1); }
    __device__ __forceinline__ void sync() const {
        if (threads <= 32) __syncwarp();
        else asm volatile("barrier.cta.sync %0, %1;" ::"r"(1 + index), "r"(threads) : "memory");
    }
    // The largest of the team's; `tops`: a word for each warp, free again after the team's next sync().
    __device__ __forceinline__ float largest(float x, float* tops) const {
        if (threads >= 32) {
            x = __uint_as_float(__reduce_max_sync(~0u, __float_as_uint(x)));
            if (threads == 32) return x;
            if ((threadIdx.x & 31) == 0) tops[threadIdx.x >> 5] = x;
            sync();
            for (int w = 0; w < threads >> 5; ++w) x = fmaxf(x, tops[index * (threads >> 5) + w]);
            return x;
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
            const float y = __shfl_xor_sync(~0u, x, d);
            if (d < threads) x = fmaxf(x, y);
        }
        return x;
    }
};

// One block's rows of the call, of one key head: tokens t .. t + n - 1 (none: n = 0).
struct Rows {
    int64_t t;
    int n;
    bool fresh;                          // the block's first token is among them
    const uint16_t* src;                 // rows `ts` apart
    int64_t ts;
    uint8_t* codes;                      // of the block's first token
    float* scale;
    int table;                           // the first one's row in the table of sines
};

// HOLD: chunks of 16 values that a thread keeps between a block's maximum and its codes.
template <int PAIRS, int HOLD>
__device__ __forceinline__ void load_rows(const Grid& gr, const Rows& u, int first, int step, int half, Raw (&raw)[HOLD]) {
    const int all = u.n * gr.chunks;
#pragma unroll
    for (int j = 0; j < HOLD; ++j) {
        const int i = first + step * j;
        if (i < all) {
            const int r = over(i, gr.m_chunks, gr.chunks);
            raw[j] = load_chunk<PAIRS>(u.src + (int64_t)r * u.ts, i - r * gr.chunks, half);
        }
    }
}

// The codes and the scale of a block's rows; `raw`: their first chunks, loaded already, `held`: its scale.  Every thread of
// a warp calls it, whatever its team has to do.
template <int PAIRS, bool I8, bool FAR, int HOLD>
__device__ __forceinline__ void write_block(const BlockParams& p, const Grid& gr, const Rows& u, int half, const float* table,
                                            Raw (&raw)[HOLD], float held, const Team& team, float* tops) {
    const int own = team.thread(), step = team.threads, all = u.n * gr.chunks, bs = p.block_shift;
    const float old = u.fresh ? 0.f : fminf(fmaxf(held, kLeastScale), kMostScale);
    auto value = [&](int i, const Raw& w, Chunk& x, int& r, int& c) {
        r = over(i, gr.m_chunks, gr.chunks), c = i - r * gr.chunks;
        unpack<PAIRS>(w, x);
        const int row = u.table + r;
        if (!FAR || row < gr.table_rows) turn_chunk<PAIRS>(x, c, half, gr.groups, table + row * 16 * gr.groups);
        else turn_chunk_far(p.rope, x, u.t + r, c, half);
    };
    float top = 0.f;
#pragma unroll 1
    for (int first = own; first < all; first += step * HOLD) {
        if (first != own) load_rows<PAIRS, HOLD>(gr, u, first, step, half, raw);
#pragma unroll
        for (int j = 0; j < HOLD; ++j)
            if (first + step * j < all) {
                Chunk x;
                int r, c;
                value(first + step * j, raw[j], x, r, c);
                top = fmaxf(top, top_of(x));
            }
    }
    __syncwarp();
    top = team.largest(top, tops);
    const float scale = fmaxf(old, scale_for<I8>(top));
    if (own == 0 && all > 0) *u.scale = scale;
    const bool grows = all > 0 && old > 0.f && old < scale;
    if (grows) {
        // the block's codes to the new scale; those of this call's tokens are written after
        const float by = __fdiv_rn(old, scale);
        auto at = [&](int i) {
            const int r = over(i, gr.m_chunks, gr.chunks);
            return reinterpret_cast<uint4*>(u.codes + (int64_t)r * p.rope.token_bytes + 16 * (i - r * gr.chunks));
        };
#pragma unroll 1
        for (int first = own; first < gr.chunks << bs; first += HOLD * step) {
#pragma unroll
            for (int j = 0; j < HOLD; ++j)       // in flight together, in the rows' place
                if (first + j * step < gr.chunks << bs) raw[j].a = *at(first + j * step);
#pragma unroll
            for (int j = 0; j < HOLD; ++j)
                if (first + j * step < gr.chunks << bs) {
                    for (uint32_t* k : {&raw[j].a.x, &raw[j].a.y, &raw[j].a.z, &raw[j].a.w}) {
                        float x[4];
                        values4<I8>(*k, x);
                        *k = codes4<I8>(x[0], x[1], x[2], x[3], by);
                    }
                    *at(first + j * step) = raw[j].a;
                }
        }
    }
    team.sync();
    const float by = __frcp_rn(scale);
#pragma unroll 1
    for (int first = own; first < all; first += step * HOLD) {
        if (grows || all > step * HOLD) load_rows<PAIRS, HOLD>(gr, u, first, step, half, raw);
#pragma unroll
        for (int j = 0; j < HOLD; ++j)
            if (first + step * j < all) {
                Chunk x;
                int r, c;
                value(first + step * j, raw[j], x, r, c);
                const int place = p.rope.slots[u.t + r] & ((1 << bs) - 1);
                store_codes<PAIRS, I8>(u.codes + (int64_t)place * p.rope.token_bytes, c, half, x, by);
            }
    }
    __syncwarp();
}

// Whether the tokens of each block come one after another, and are no more than it has: the blocks that begin in a token
// are put into a table in shared memory of `words` (a power of two), at most half full, in which none may be found.  The
// `part`-th of `parts` CTAs has those whose hash falls to it.  Beside the others' work this shows little: 4096 single tokens
// 20.4 us with and without it, 5456 of prompts 25.4 -> 25.6, 46597 193 -> 194 (one slot after the other, and one table for
// 4096 single tokens: 40 us).
__device__ __forceinline__ void look_at_order(const RopeParams& r, int bs, uint32_t* table, int words, int part, int parts) {
    constexpr int AHEAD = 8;                 // tokens of a thread whose slots are under way at once
    constexpr uint32_t NONE = 0xffffffffu;
    for (int i = threadIdx.x; i < words; i += BA_THREADS) table[i] = NONE;
    __syncthreads();
    bool again = false;
#pragma unroll 1
    for (int64_t t0 = threadIdx.x; t0 < r.tokens; t0 += AHEAD * BA_THREADS) {
        int32_t slot[AHEAD], before[AHEAD], full[AHEAD];
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
            const int64_t t = t0 + j * BA_THREADS;
            slot[j] = t < r.tokens ? r.slots[t] : -1;
            before[j] = t < r.tokens && t > 0 ? r.slots[t - 1] : -1;
            full[j] = t < r.tokens && t >> bs ? r.slots[t - (1 << bs)] : -1;
        }
        uint32_t at[AHEAD], was[AHEAD];
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
            const uint32_t block = (uint32_t)(slot[j] >> bs);
            const bool there = slot[j] >= 0 && slot[j] >> r.page_shift < r.pages;
            again |= there && full[j] >= 0 && (uint32_t)(full[j] >> bs) == block;
            const bool begins = there && (before[j] < 0 || (uint32_t)(before[j] >> bs) != block);
            uint32_t h = block * 0x9e3779b1u;    // 2^32 over the golden ratio
            h = (h ^ h >> 15) * 0x9e3779b1u;
            at[j] = h ^ h >> 13;
            was[j] = begins && (int)__umulhi(at[j], (uint32_t)parts) == part ? atomicCAS(&table[at[j] & (words - 1)], NONE, block) : NONE;
        }
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
            const uint32_t block = (uint32_t)(slot[j] >> bs);
#pragma unroll 1
            for (int i = 1; was[j] != NONE && was[j] != block && i < words; ++i) was[j] = atomicCAS(&table[(at[j] + i) & (words - 1)], NONE, block);
            again |= was[j] == block && was[j] != NONE;
        }
    }
    if (again) atomicOr(r.status, 4u);
}

// FAR: blocks whose tokens' sines do not all fit the table.
template <int PAIRS, bool I8, bool FAR, int HOLD>
__global__ void __launch_bounds__(BA_THREADS, PAIRS != HALVES_1 && !FAR ? 3 : 2) block_append_kernel(const __grid_constant__ BlockParams p, const __grid_constant__ Grid gr) {
    extern __shared__ __align__(16) float table[];       // sines of a few tokens
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const RopeParams& r = p.rope;
    const int half = r.rotary >> 1, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if ((int)blockIdx.x >= gr.kv_ctas) {
        const int cta = (int)blockIdx.x - gr.order_ctas;
        if (cta < gr.kv_ctas) {
            look_at_order(r, p.block_shift, reinterpret_cast<uint32_t*>(table), gr.order_words, (int)blockIdx.x - gr.kv_ctas, gr.order_ctas);
            return;
        }
        // ================= q of a few tokens, or of a share of one's heads: a thread takes a chunk of each token
        const int at = cta - gr.kv_ctas, group = over(at, gr.m_q_parts, gr.q_parts);
        const int64_t t0 = (int64_t)group * gr.q_tokens;
        const int tokens = (int)min((int64_t)gr.q_tokens, r.tokens - t0), part = at - group * gr.q_parts;
        const int all = r.heads_q * gr.chunks, step = gr.q_parts * BA_THREADS;
        const uint16_t* q = r.q + t0 * r.q_ts;
        uint16_t* out = r.out + t0 * r.o_ts;
        Raw raw[Q_TOKENS];
        int h, c;
        auto load = [&](int i) {
            h = over(i, gr.m_chunks, gr.chunks), c = i - h * gr.chunks;
#pragma unroll
            for (int j = 0; j < Q_TOKENS; ++j)
                if (j < tokens) raw[j] = load_chunk<PAIRS>(q + j * r.q_ts + h * r.q_hs, c, half);
        };
        int i = part * BA_THREADS + tid;
        if (i < all) load(i);
        for (int k = tid; k < tokens * half; k += BA_THREADS) {
            const int token = over(k, gr.m_half, half);
            put_sines(r, t0 + token, k - token * half, gr.groups, table + token * 16 * gr.groups);
        }
        __syncthreads();
#pragma unroll 1
        while (i < all) {
#pragma unroll
            for (int j = 0; j < Q_TOKENS; ++j)
                if (j < tokens) {
                    Chunk x;
                    unpack<PAIRS>(raw[j], x);
                    turn_chunk<PAIRS>(x, c, half, gr.groups, table + j * 16 * gr.groups);
                    store_bf16<PAIRS>(out + j * r.o_ts + h * r.o_hs, c, half, x);
                }
            i += step;
            if (i < all) load(i);
        }
        return;
    }
    // ================= k, or v, of the blocks that begin, for this call, in these rows
    const int window = over((int)blockIdx.x, gr.m_parts, 2 * gr.parts), part = (int)blockIdx.x - window * 2 * gr.parts;
    const bool is_v = part >= gr.parts;
    const int64_t t0 = (int64_t)window * gr.rows;
    const int bs = p.block_shift;
    __shared__ float tops[BA_WARPS];
    __shared__ int8_t leader[BA_WARPS][32];
    // Lane l has the slot of token t0 - 1 + l.  A token of these whose predecessor lies in another block begins the rows of its
    // block, as many as follow in it.
    auto slot_at = [&](int64_t i) { return i >= 0 && i < r.tokens ? r.slots[i] : -1; };
    const int32_t own = slot_at(t0 - 1 + lane), before = __shfl_up_sync(~0u, own, 1);
    const bool there = own >= 0 && own >> r.page_shift < r.pages, mine = lane >= 1 && lane <= gr.rows;
    const bool follows = lane >= 1 && before >= 0 && before >> bs == own >> bs;
    if (mine && own != -1 && !there && r.status && part == 0 && warp == 0) atomicOr(r.status, 2u);
    const uint32_t leaders = __ballot_sync(~0u, mine && there && !follows);
    if (leaders == 0) return;
    const uint32_t following = __ballot_sync(~0u, follows), begins = __ballot_sync(~0u, (own & ((1 << bs) - 1)) == 0);
    const uint32_t stop = lane < 31 ? ~following >> (lane + 1) : 0u;     // the first token behind that does not follow
    int n = stop && lane + __ffs(stop) < 32 ? __ffs(stop) : 32 - lane;
    bool fresh = (begins >> lane & (n == 32 ? ~0u : (1u << n) - 1u)) != 0;
    const int last = 31 - __clz(leaders);
    if (last + __shfl_sync(~0u, n, last) == 32 && 32 - last < 1 << bs) {
        // the last block's rows may go on behind lane 31
        const int block = __shfl_sync(~0u, own, last) >> bs;
        int more = 0;
        bool any = false;
        for (;;) {
            const int32_t s = slot_at(t0 + 31 + more + lane);
            const uint32_t other = ~__ballot_sync(~0u, s >= 0 && s >> bs == block), first = __ballot_sync(~0u, (s & ((1 << bs) - 1)) == 0);
            const int run = other ? __ffs(other) - 1 : 32;
            any |= (first & (run == 32 ? ~0u : (1u << run) - 1u)) != 0;
            more += run;
            if (run < 32 || more >= 1 << bs) break;
        }
        if (lane == last) n += more, fresh |= any;
    }
    n = min(n, 1 << bs);                     // more would name a slot twice
    if (leaders >> lane & 1u) leader[warp][__popc(leaders & ((1u << lane) - 1u))] = (int8_t)lane;
    __syncwarp();
    const int most = __reduce_max_sync(~0u, leaders >> lane & 1u ? n : 0), first_lane = __ffs(leaders) - 1;
    // As many CTAs share the heads as make two rounds of them, or what there are; the others have nothing to do.
    int parts = gr.least_parts;
    while (parts < gr.parts && most * gr.chunks * r.heads_kv > 2 * HOLD * BA_THREADS * parts) parts = min(2 * parts, gr.parts);
    const int mine_of = is_v ? part - gr.parts : part;
    if (mine_of >= parts) return;
    const int h0 = mine_of * r.heads_kv / parts, heads = (mine_of + 1) * r.heads_kv / parts - h0, total = __popc(leaders) * heads;
    // As many threads to a block's rows as keep them in registers, or find something to do when each has a team: with the
    // rows, or with what the block holds already, should its scale grow.
    const bool joins = __any_sync(~0u, (leaders >> lane & 1u) && !fresh);
    const int work = max(most, joins ? 1 << bs : 0) * gr.chunks;
    Team team = {1, 0};
    while (team.threads < BA_THREADS && (most * gr.chunks > HOLD * team.threads || (work > team.threads && 2 * team.threads * total <= BA_THREADS)))
        team.threads *= 2;
    team.index = tid / team.threads;
    const int teams = BA_THREADS / team.threads;
    const int turns = is_v ? 0 : half;
    Raw raw[HOLD];
    float held = 0.f;
    Rows x;
    auto load = [&](int i) {                 // the team's i-th block and head
        const int which = i < total ? i / heads : 0, h = h0 + i - which * heads, l = leader[warp][which];
        const int32_t slot = __shfl_sync(~0u, own, l);
        x.n = __shfl_sync(~0u, n, l);
        x.fresh = __shfl_sync(~0u, (int)fresh, l) != 0;
        if (i >= total) {
            x.n = 0;
            return;
        }
        const int64_t page = slot >> r.page_shift;
        const int in_page = (slot >> bs << bs) & ((1 << r.page_shift) - 1);
        x.t = t0 - 1 + l;
        x.table = l - first_lane;
        x.ts = is_v ? r.v_ts : r.k_ts;
        x.src = (is_v ? r.v : r.k) + x.t * x.ts + h * (is_v ? r.v_hs : r.k_hs);
        x.codes = (is_v ? r.vc : r.kc) + page * r.page_bytes + in_page * r.token_bytes + h * r.head_bytes;
        x.scale = (is_v ? p.v_scales : p.k_scales) + page * p.s_ps + (int64_t)(in_page >> bs) * p.s_bs + h * p.s_hs;
        held = *x.scale;
        if (PAIRS != HALVES_1 || !is_v) load_rows<PAIRS, HOLD>(gr, x, team.thread(), team.threads, turns, raw);
        else load_rows<HALVES_8, HOLD>(gr, x, team.thread(), team.threads, 0, raw);
    };
    int i = team.index;
    load(i);
    if (!is_v) {
        const int rows = last + __shfl_sync(~0u, n, last) - first_lane, many = min(rows, gr.table_rows) * half;
#pragma unroll 4
        for (int k = tid; k < many; k += BA_THREADS) {
            const int row = over(k, gr.m_half, half);
            put_sines(r, min(t0 - 1 + first_lane + row, r.tokens - 1), k - row * half, gr.groups, table + row * 16 * gr.groups);
        }
        __syncthreads();
    }
#pragma unroll 1
    for (int round = 0; round < total; round += teams) {
        if (PAIRS != HALVES_1 || !is_v) write_block<PAIRS, I8, FAR, HOLD>(p, gr, x, turns, table, raw, held, team, tops);
        else write_block<HALVES_8, I8, false, HOLD>(p, gr, x, 0, table, raw, held, team, tops);
        i += teams;
        if (round + teams < total) load(i);
        if (team.threads > 32) team.sync();  // `tops` serves the next
    }
}

}  // namespace

cudaError_t launch_block_append(const BlockParams& p, int sms, cudaStream_t st) {
    const RopeParams& r = p.rope;
    const int pairs = r.neighbour ? NEIGHBOURS : r.rotary % 16 == 0 ? HALVES_8 : r.rotary % 8 == 0 ? HALVES_4 : HALVES_1;
    const int half = r.rotary / 2, block = 1 << p.block_shift;
    auto reciprocal = [](int d) { return d > 1 ? (uint32_t)((((uint64_t)1 << 32) + d - 1) / d) : 0u; };
    Grid g = {};
    g.chunks = r.dim / 16;
    // k and v: some rows to a CTA, so that a CTA of short blocks has several and one in which none begins is soon done; and
    // parts that share the heads, where there are few CTAs even if a block begins in each row (a decode step of 64 tokens:
    // 3.3 us; with a part for each of 8 heads 8.4), or so many rows that they are prompts' and most blocks are whole.  Of a few
    // tokens nobody knows here how many come to a block: parts for whole ones are there, and those that have nothing to do
    // end (237 tokens in blocks of 64: 19.4 -> 9.7 us; 256 single tokens of such blocks 15.2 -> 18.6)
    g.rows = r.tokens >= 32 * sms ? 16 : r.tokens >= 8 * sms ? 8 : r.tokens >= 2 * sms ? 2 : 1;
    const int64_t whole = (r.tokens + block - 1) / block;
    const int64_t want = r.tokens >= 8 * sms ? (sms + whole - 1) / whole : 3 * sms * g.rows / (4 * r.tokens);
    g.least_parts = (int)(want < 1 ? 1 : want < r.heads_kv ? want : r.heads_kv);
    const int large = (block * g.chunks + 127) / 128;    // parts for a block that is brought whole, should one be
    g.parts = r.tokens >= 8 * sms || large <= g.least_parts ? g.least_parts : large < r.heads_kv ? large : r.heads_kv;
    g.kv_ctas = (int)((r.tokens + g.rows - 1) / g.rows) * 2 * g.parts;
    g.groups = (half + 7) / 8;
    g.table_rows = half ? (int)(BA_TABLE / (64 * g.groups)) : block;
    if (g.table_rows > block + g.rows - 1) g.table_rows = block + g.rows - 1;
    // q: several tokens to a CTA, or with few of them as many CTAs a token as fill the SMs and find a chunk for each thread
    const int64_t split = (2 * sms + r.tokens - 1) / r.tokens;
    const int wide = (r.heads_q * g.chunks + BA_THREADS - 1) / BA_THREADS;
    g.q_tokens = r.tokens >= 16 * sms ? Q_TOKENS : r.tokens >= 8 * sms ? 2 : 1;
    g.q_parts = g.q_tokens > 1 ? 1 : (int)(split < wide ? split : wide);
    g.m_chunks = reciprocal(g.chunks), g.m_half = reciprocal(half), g.m_parts = reciprocal(2 * g.parts), g.m_q_parts = reciprocal(g.q_parts);
    const int64_t q_ctas = (r.tokens + g.q_tokens - 1) / g.q_tokens * g.q_parts;
    size_t smem = (size_t)(g.table_rows > g.q_tokens ? g.table_rows : g.q_tokens) * 64 * g.groups;
    if (r.status && r.tokens <= AFFQMM_BLOCK_ORDER) {
        // a block begins in each token at most, and the tables are half full then, 32 KB at most, with which an SM still holds
        // three CTAs; eight CTAs share more than a few such tokens, more only where the tables ask for it, as each reads every slot
        const int64_t room = 2 * r.tokens, tables = (room + 8191) / 8192, shared = (r.tokens + 511) / 512;
        g.order_words = 256;
        while (g.order_words < 8192 && g.order_words < room) g.order_words *= 2;
        g.order_ctas = (int)(tables > 8 ? tables : shared < 8 ? shared : 8);
        if (smem < (size_t)g.order_words * 4) smem = (size_t)g.order_words * 4;
    }
    // Two chunks to a thread where there are few tokens: a call's time is then the kernel's way through its code, cold (64
    // tokens of a decode step: 3.8 us with four, 3.3 with two; 7646 rows of prompts: 34.5 with four, 36.0 with two).
    auto pick = [&](auto i8, auto far, auto hold) {
        constexpr bool I8 = decltype(i8)::value, FAR = decltype(far)::value;
        constexpr int HOLD = decltype(hold)::value;
        return pairs == HALVES_8   ? block_append_kernel<HALVES_8, I8, FAR, HOLD>
               : pairs == HALVES_4 ? block_append_kernel<HALVES_4, I8, FAR, HOLD>
               : pairs == HALVES_1 ? block_append_kernel<HALVES_1, I8, FAR, HOLD>
                                   : block_append_kernel<NEIGHBOURS, I8, FAR, HOLD>;
    };
    using Four = std::integral_constant<int, 4>;
    const bool far = half && g.table_rows < block + g.rows - 1, few = r.tokens < 16 * sms;
    auto typed = [&](auto i8) {
        return far   ? pick(i8, std::true_type{}, Four{})
               : few ? pick(i8, std::false_type{}, std::integral_constant<int, 2>{})
                     : pick(i8, std::false_type{}, Four{});
    };
    auto* kernel = r.e4m3 ? typed(std::false_type{}) : typed(std::true_type{});
    if (smem > 40 << 10) {                   // the kernel has some of its own beside it
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)BA_TABLE);
        if (e != cudaSuccess) return e;
    }
    return launch_pdl(kernel, dim3((unsigned)(g.kv_ctas + g.order_ctas + q_ctas)), BA_THREADS, smem, st, p, g);
}

}  // namespace affqmm
