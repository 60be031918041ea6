// block_append.cu -- rotary positions on a step's q and k, and k and v
// quantised as they are written to a cache with a scale for each block of
// tokens and key head (include/affqmm.h states the arithmetic):
//
//     top = max |x| of the call's tokens of the block, x = k turned, or v
//     scale = max(old, top / 127) or, e4m3, max(old, 2^ceil(log2(top / 448)))
//     code = round(x / scale), and the block's other codes times old / scale
//
// Every value of a block waits for the largest of them, so a block's rows are
// one warp's work, for one key head and k or v: it turns them, reduces the
// maximum and writes the codes.  One launch has two kinds of CTAs: those of q
// take a token each (the sines once for all heads), those of k and v a few
// rows of the call and a share of the heads.  A row whose predecessor lies in
// the same block belongs to that row's warp; the first one's warp finds how
// many follow.
#include <type_traits>

#include "affqmm_internal.h"
#include "affqmm_paged.h"
#include "rope_pieces.cuh"

namespace affqmm {
namespace {

constexpr int BA_THREADS = 256, BA_WARPS = BA_THREADS / 32;
constexpr int HOLD = 4;                  // chunks of 16 values that a lane has in flight, and keeps while a block's maximum is found
constexpr size_t BA_TABLE = 136 << 10;   // most shared memory for sines: all but those of 128 tokens at rotary 512

// How a head's values pair: HALVES i with i + rotary / 2, in whole chunks of
// 8 pairs (rotary a multiple of 16); NEIGHBOURS 2i with 2i + 1; ODD_HALVES as
// HALVES, at any even rotary.
enum Pairs { HALVES, NEIGHBOURS, ODD_HALVES };

// Eight pairs of a head: chunk c has the pairs 8c .. 8c + 7, where values that do not turn are pairs of neighbours
// (HALVES: of one run of eight and the next).  Raw: as they are read, two runs of eight.
struct Raw {
    uint4 a, b;
};
struct Chunk {
    float a[8], b[8];
};

// Where chunk c's two runs of eight values begin (HALVES).
__device__ __forceinline__ void runs_of(int c, int half, int& d0, int& d1) {
    const bool turns = 8 * c < half;
    d0 = turns ? 8 * c : 16 * c;                    // 2 half + 16 (c - half / 8)
    d1 = d0 + (turns ? half : 8);
}

template <int PAIRS>
__device__ __forceinline__ Raw load_chunk(const uint16_t* src, int c, int half) {
    Raw x;
    if constexpr (PAIRS == HALVES) {
        int d0, d1;
        runs_of(c, half, d0, d1);
        x.a = *reinterpret_cast<const uint4*>(src + d0);
        x.b = *reinterpret_cast<const uint4*>(src + d1);
    } else if constexpr (PAIRS == NEIGHBOURS) {
        x.a = *reinterpret_cast<const uint4*>(src + 16 * c);
        x.b = *reinterpret_cast<const uint4*>(src + 16 * c + 8);
    } else {
        uint32_t a[8], b[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int i = 8 * c + e;
            a[e] = src[i < half ? i : 2 * i], b[e] = src[i < half ? i + half : 2 * i + 1];
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

// Chunk c turned, by a token's table of sines or, where that has no room for it, by sines made here (token t).
template <int PAIRS>
__device__ __forceinline__ void turn_chunk(Chunk& x, int c, int half, const float* cosines, const float* sines) {
    if (8 * c >= half) return;
    float co[8], si[8];
    if constexpr (PAIRS == HALVES) {
#pragma unroll
        for (int e = 0; e < 8; e += 4) {
            const float4 u = *reinterpret_cast<const float4*>(cosines + 8 * c + e), w = *reinterpret_cast<const float4*>(sines + 8 * c + e);
            co[e] = u.x, co[e + 1] = u.y, co[e + 2] = u.z, co[e + 3] = u.w;
            si[e] = w.x, si[e + 1] = w.y, si[e + 2] = w.z, si[e + 3] = w.w;
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (8 * c + e < half) co[e] = cosines[8 * c + e], si[e] = sines[8 * c + e];
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        if (PAIRS != HALVES && 8 * c + e >= half) continue;
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
    if constexpr (PAIRS == HALVES) {
        int d0, d1;
        runs_of(c, half, d0, d1);
        *reinterpret_cast<uint2*>(dst + d0) = make_uint2(codes4<I8>(x.a[0], x.a[1], x.a[2], x.a[3], by), codes4<I8>(x.a[4], x.a[5], x.a[6], x.a[7], by));
        *reinterpret_cast<uint2*>(dst + d1) = make_uint2(codes4<I8>(x.b[0], x.b[1], x.b[2], x.b[3], by), codes4<I8>(x.b[4], x.b[5], x.b[6], x.b[7], by));
    } else if constexpr (PAIRS == NEIGHBOURS) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = codes4<I8>(x.a[2 * i], x.b[2 * i], x.a[2 * i + 1], x.b[2 * i + 1], by);
        *reinterpret_cast<uint4*>(dst + 16 * c) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int i = 8 * c + e, d0 = i < half ? i : 2 * i, d1 = i < half ? i + half : 2 * i + 1;
            const uint32_t w = codes4<I8>(x.a[e], x.b[e], 0.f, 0.f, by);
            dst[d0] = (uint8_t)w, dst[d1] = (uint8_t)(w >> 8);
        }
    }
}
template <int PAIRS>
__device__ __forceinline__ void store_bf16(uint16_t* dst, int c, int half, const Chunk& x) {
    if constexpr (PAIRS == HALVES) {
        int d0, d1;
        runs_of(c, half, d0, d1);
        *reinterpret_cast<uint4*>(dst + d0) = make_uint4(bf2(x.a[0], x.a[1]), bf2(x.a[2], x.a[3]), bf2(x.a[4], x.a[5]), bf2(x.a[6], x.a[7]));
        *reinterpret_cast<uint4*>(dst + d1) = make_uint4(bf2(x.b[0], x.b[1]), bf2(x.b[2], x.b[3]), bf2(x.b[4], x.b[5]), bf2(x.b[6], x.b[7]));
    } else if constexpr (PAIRS == NEIGHBOURS) {
        *reinterpret_cast<uint4*>(dst + 16 * c) = make_uint4(bf2(x.a[0], x.b[0]), bf2(x.a[1], x.b[1]), bf2(x.a[2], x.b[2]), bf2(x.a[3], x.b[3]));
        *reinterpret_cast<uint4*>(dst + 16 * c + 8) = make_uint4(bf2(x.a[4], x.b[4]), bf2(x.a[5], x.b[5]), bf2(x.a[6], x.b[6]), bf2(x.a[7], x.b[7]));
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int i = 8 * c + e, d0 = i < half ? i : 2 * i, d1 = i < half ? i + half : 2 * i + 1;
            const uint32_t w = bf2(x.a[e], x.b[e]);
            dst[d0] = (uint16_t)w, dst[d1] = (uint16_t)(w >> 16);
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
    int kv_ctas, rows, parts;            // of k and v: CTAs, rows of the call to a CTA, CTAs that share the heads
    int q_tokens, q_parts;               // of q: tokens to a CTA, or (one token) CTAs that share its heads
    int table_rows;                      // rows whose sines shared memory holds
    int chunks;                          // of a head
    uint32_t m_chunks, m_half, m_parts, m_q_parts, m_heads_q;
};

// One block's rows t .. t + n - 1 of the call, of one key head.
struct Rows {
    const uint16_t* src;                 // rows `ts` apart
    int64_t ts;
    uint8_t* codes;                      // of the block's first token
    float* scale;
};

// The warps that share a block's rows: `warps` of them, the `index`-th of the CTA's teams.
struct Team {
    int warps, index;
    __device__ __forceinline__ int threads() const { return 32 * warps; }
    __device__ __forceinline__ int thread() const { return (int)threadIdx.x & (threads() - 1); }
    __device__ __forceinline__ void sync() const {
        if (warps == 1) __syncwarp();
        else asm volatile("barrier.cta.sync %0, %1;" ::"r"(1 + index), "r"(threads()) : "memory");
    }
};

template <int PAIRS>
__device__ __forceinline__ void load_rows(const Grid& gr, const Rows& u, int n, int first, int step, int half, Raw (&raw)[HOLD]) {
    const int all = n * gr.chunks;
#pragma unroll
    for (int j = 0; j < HOLD; ++j) {
        const int i = first + step * j;
        if (i < all) {
            const int r = over(i, gr.m_chunks, gr.chunks);
            raw[j] = load_chunk<PAIRS>(u.src + (int64_t)r * u.ts, i - r * gr.chunks, half);
        }
    }
}

// The codes and the scale of a block's rows; `raw`: their first chunks, loaded already, `held`: its scale, `tops`: of the
// CTA's warps.
template <int PAIRS, bool I8, bool FAR>
__device__ __forceinline__ void write_block(const BlockParams& p, const Grid& gr, int64_t t, int n, bool fresh, const Rows& u, int half,
                                            const float* cosines, const float* sines, Raw (&raw)[HOLD], float held, const Team& team, float* tops) {
    const int own = team.thread(), step = team.threads(), all = n * gr.chunks, bs = p.block_shift;
    const float old = fresh ? 0.f : fminf(fmaxf(held, kLeastScale), kMostScale);
    auto value = [&](int i, const Raw& w, Chunk& x, int& r, int& c) {
        r = over(i, gr.m_chunks, gr.chunks), c = i - r * gr.chunks;
        unpack<PAIRS>(w, x);
        if (!FAR || r < gr.table_rows) turn_chunk<PAIRS>(x, c, half, cosines + r * half, sines + r * half);
        else turn_chunk_far(p.rope, x, t + r, c, half);
    };
    float top = 0.f;
#pragma unroll 1
    for (int first = own; first < all; first += step * HOLD) {
        if (first != own) load_rows<PAIRS>(gr, u, n, first, step, half, raw);
#pragma unroll
        for (int j = 0; j < HOLD; ++j)
            if (first + step * j < all) {
                Chunk x;
                int r, c;
                value(first + step * j, raw[j], x, r, c);
                top = fmaxf(top, top_of(x));
            }
    }
    top = __uint_as_float(__reduce_max_sync(~0u, __float_as_uint(top)));
    if (team.warps > 1) {
        const int warp = threadIdx.x >> 5;
        if ((threadIdx.x & 31) == 0) tops[warp] = top;
        team.sync();
        for (int w = 0; w < team.warps; ++w) top = fmaxf(top, tops[team.index * team.warps + w]);
    }
    const float scale = fmaxf(old, scale_for<I8>(top));
    if (own == 0) *u.scale = scale;
    if (old > 0.f && old < scale) {
        // the block's codes to the new scale; those of this call's tokens are written after
        const float by = __fdiv_rn(old, scale);
#pragma unroll 1
        for (int i = own; i < gr.chunks << bs; i += step) {
            const int r = over(i, gr.m_chunks, gr.chunks), c = i - r * gr.chunks;
            uint4* at = reinterpret_cast<uint4*>(u.codes + (int64_t)r * p.rope.token_bytes + 16 * c);
            uint4 w = *at;
            for (uint32_t* k : {&w.x, &w.y, &w.z, &w.w}) {
                float x[4];
                values4<I8>(*k, x);
                *k = codes4<I8>(x[0], x[1], x[2], x[3], by);
            }
            *at = w;
        }
        team.sync();
    }
    const float by = __frcp_rn(scale);
#pragma unroll 1
    for (int first = own; first < all; first += step * HOLD) {
        if (all > step * HOLD) load_rows<PAIRS>(gr, u, n, first, step, half, raw);
#pragma unroll
        for (int j = 0; j < HOLD; ++j)
            if (first + step * j < all) {
                Chunk x;
                int r, c;
                value(first + step * j, raw[j], x, r, c);
                const int place = p.rope.slots[t + r] & ((1 << bs) - 1);
                store_codes<PAIRS, I8>(u.codes + (int64_t)place * p.rope.token_bytes, c, half, x, by);
            }
    }
}

// FAR: blocks whose tokens' sines do not all fit the table.
template <int PAIRS, bool I8, bool FAR>
__global__ void __launch_bounds__(BA_THREADS, PAIRS == HALVES && !FAR ? 3 : 2) block_append_kernel(const __grid_constant__ BlockParams p, const __grid_constant__ Grid gr) {
    extern __shared__ __align__(16) float table[];       // cosines, sines: [row][rotary / 2]
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const RopeParams& r = p.rope;
    const int half = r.rotary >> 1, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    float* cosines = table;
    if ((int)blockIdx.x >= gr.kv_ctas) {
        // ================= q of a few tokens, or of a share of one's heads
        const int at = (int)blockIdx.x - gr.kv_ctas, group = over(at, gr.m_q_parts, gr.q_parts);
        const int64_t t0 = (int64_t)group * gr.q_tokens;
        const int tokens = (int)min((int64_t)gr.q_tokens, r.tokens - t0), part = at - group * gr.q_parts;
        const int all = tokens * r.heads_q * gr.chunks, step = gr.q_parts * BA_THREADS;
        float* sines = table + gr.q_tokens * half;
        auto place = [&](int i, int& token, int& h, int& c) {
            const int row = over(i, gr.m_chunks, gr.chunks);
            c = i - row * gr.chunks, token = over(row, gr.m_heads_q, r.heads_q), h = row - token * r.heads_q;
        };
        Raw raw[HOLD];
        auto load = [&](int first) {
#pragma unroll
            for (int j = 0; j < HOLD; ++j)
                if (first + j * step < all) {
                    int token, h, c;
                    place(first + j * step, token, h, c);
                    raw[j] = load_chunk<PAIRS>(r.q + (t0 + token) * r.q_ts + h * r.q_hs, c, half);
                }
        };
        int i = part * BA_THREADS + tid;
        load(i);
        for (int k = tid; k < tokens * half; k += BA_THREADS) {
            const int token = over(k, gr.m_half, half);
            near_turn_of(r, t0 + token, k - token * half, sines + k, cosines + k);
        }
        __syncthreads();
#pragma unroll 1
        for (; i < all; i += HOLD * step, load(i)) {
#pragma unroll
            for (int j = 0; j < HOLD; ++j)
                if (i + j * step < all) {
                    int token, h, c;
                    place(i + j * step, token, h, c);
                    Chunk x;
                    unpack<PAIRS>(raw[j], x);
                    turn_chunk<PAIRS>(x, c, half, cosines + token * half, sines + token * half);
                    store_bf16<PAIRS>(r.out + (t0 + token) * r.o_ts + h * r.o_hs, c, half, x);
                }
        }
        return;
    }
    // ================= k and v of the blocks that begin, for this call, in these rows
    const int chunk_of_rows = over((int)blockIdx.x, gr.m_parts, gr.parts), part = (int)blockIdx.x - chunk_of_rows * gr.parts;
    const int64_t t0 = (int64_t)chunk_of_rows * gr.rows;
    const int units = 2 * r.heads_kv, u0 = part * units / gr.parts, u1 = (part + 1) * units / gr.parts;   // k's heads, then v's
    const int bs = p.block_shift;
    float* sines = table + gr.table_rows * half;
    __shared__ float tops[BA_WARPS];
    // lane l has the slot of token t0 - 1 + l; the tokens that begin a block's rows
    auto slot_at = [&](int64_t i) { return i >= 0 && i < r.tokens ? r.slots[i] : -1; };
    const int32_t own = slot_at(t0 - 1 + lane), before = __shfl_up_sync(~0u, own, 1);
    const bool there = own >= 0 && own >> r.page_shift < r.pages, mine = lane >= 1 && lane <= gr.rows;
    uint32_t leaders = __ballot_sync(~0u, mine && there && !(before >= 0 && before >> bs == own >> bs));
    if (mine && own != -1 && !there && r.status && part == 0 && warp == 0) atomicOr(r.status, 2u);
#pragma unroll 1
    for (; leaders; leaders &= leaders - 1u) {
        const int l = __ffs(leaders) - 1;
        const int64_t t = t0 - 1 + l;
        const int32_t slot = __shfl_sync(~0u, own, l);
        const int64_t page = slot >> r.page_shift;
        const int block = slot >> bs;
        // how many of the tokens from t on lie in the block, and whether its first one is among them
        int n = 0;
        bool fresh = false;
        int32_t s = own;
        for (int from = l;; from = 0) {
            const uint32_t behind = ~0u << from, same = __ballot_sync(~0u, s >= 0 && s >> bs == block), first = __ballot_sync(~0u, (s & ((1 << bs) - 1)) == 0);
            const uint32_t other = ~same & behind, run = other ? (1u << (__ffs(other) - 1)) - 1u : ~0u;   // lanes before the first other one
            fresh |= (first & run & behind) != 0;
            n += __popc(run & behind);
            if (other || n >= 1 << bs) break;
            s = slot_at(t + n + lane);
        }
        n = min(n, 1 << bs);                 // more would name a slot twice
        // as many warps to a block's rows as keep them in registers
        Team team = {1, 0};
        while (team.warps < BA_WARPS && n * gr.chunks > 32 * HOLD * team.warps) team.warps *= 2;
        team.index = warp / team.warps;
        const int teams = BA_WARPS / team.warps;
        const int first_of_block = (block << bs) & ((1 << r.page_shift) - 1);
        const int64_t at = page * r.page_bytes + first_of_block * r.token_bytes, scale_at = page * p.s_ps + (int64_t)(first_of_block >> bs) * p.s_bs;
        auto rows_of = [&](int u) {
            const bool is_v = u >= r.heads_kv;
            const int h = is_v ? u - r.heads_kv : u;
            return is_v ? Rows{r.v + t * r.v_ts + h * r.v_hs, r.v_ts, r.vc + at + h * r.head_bytes, p.v_scales + scale_at + h * p.s_hs}
                        : Rows{r.k + t * r.k_ts + h * r.k_hs, r.k_ts, r.kc + at + h * r.head_bytes, p.k_scales + scale_at + h * p.s_hs};
        };
        Raw raw[HOLD];
        float held = 0.f;
        Rows x = {};
        auto load = [&](int u) {
            x = rows_of(u);
            held = *x.scale;
            const int turns = u < r.heads_kv ? half : 0;
            if (PAIRS == HALVES || u < r.heads_kv) load_rows<PAIRS>(gr, x, n, team.thread(), team.threads(), turns, raw);
            else load_rows<HALVES>(gr, x, n, team.thread(), team.threads(), 0, raw);
        };
        int u = u0 + team.index;
        if (u < u1) load(u);
        if (u0 < u1 && u0 < r.heads_kv) {
            const int many = min(n, gr.table_rows) * half;
            for (int i = tid; i < many; i += BA_THREADS) {
                const int row = over(i, gr.m_half, half);
                near_turn_of(r, t + row, i - row * half, sines + i, cosines + i);
            }
            __syncthreads();
        }
#pragma unroll 1
        while (u < u1) {
            const int turns = u < r.heads_kv ? half : 0;
            if (PAIRS == HALVES || u < r.heads_kv) write_block<PAIRS, I8, FAR>(p, gr, t, n, fresh, x, turns, cosines, sines, raw, held, team, tops);
            else write_block<HALVES, I8, false>(p, gr, t, n, fresh, x, 0, cosines, sines, raw, held, team, tops);
            u += teams;
            if (u < u1) load(u);
            if (team.warps > 1) team.sync();   // `tops` serves the next
        }
        __syncthreads();
    }
}

}  // namespace

cudaError_t launch_block_append(const BlockParams& p, int sms, cudaStream_t st) {
    const RopeParams& r = p.rope;
    const int pairs = r.neighbour ? NEIGHBOURS : r.rotary % 16 == 0 ? HALVES : ODD_HALVES;
    const int half = r.rotary / 2, block = 1 << p.block_shift;
    auto reciprocal = [](int d) { return d > 1 ? (uint32_t)((((uint64_t)1 << 32) + d - 1) / d) : 0u; };
    Grid g = {};
    g.chunks = r.dim / 16;
    // k and v: parts enough that each SM has four CTAs with a block to write, but no more than give every team of a CTA
    // (block_append_kernel) one key head; and several rows to a CTA where that still leaves CTAs enough to find the blocks
    const int units = 2 * r.heads_kv, chunks = block * g.chunks;
    int team = 1;
    while (team < BA_WARPS && chunks > 32 * HOLD * team) team *= 2;
    const int64_t want = ((int64_t)4 * sms * block + r.tokens - 1) / r.tokens;
    const int most = (units * team + BA_WARPS - 1) / BA_WARPS;
    g.parts = (int)(want < 2 ? 2 : want < most ? want : most);
    g.rows = r.tokens * g.parts > 16 * sms ? 8 : 1;
    g.kv_ctas = (int)((r.tokens + g.rows - 1) / g.rows) * g.parts;
    g.table_rows = half ? (int)(BA_TABLE / (8 * half)) : block;
    if (g.table_rows > block) g.table_rows = block;
    // q: several tokens to a CTA, or with few of them as many CTAs a token as fill the SMs and find a chunk for each thread
    const int64_t split = (2 * sms + r.tokens - 1) / r.tokens;
    const int wide = (r.heads_q * g.chunks + BA_THREADS - 1) / BA_THREADS;
    g.q_tokens = r.tokens >= 16 * sms ? 4 : r.tokens >= 8 * sms ? 2 : 1;
    g.q_parts = g.q_tokens > 1 ? 1 : (int)(split < wide ? split : wide);
    g.m_chunks = reciprocal(g.chunks), g.m_half = reciprocal(half), g.m_parts = reciprocal(g.parts), g.m_q_parts = reciprocal(g.q_parts);
    g.m_heads_q = reciprocal(r.heads_q);
    const int64_t q_ctas = (r.tokens + g.q_tokens - 1) / g.q_tokens * g.q_parts;
    const size_t smem = (size_t)(g.table_rows > g.q_tokens ? g.table_rows : g.q_tokens) * 8 * half;
    auto pick = [&](auto i8, auto far) {
        constexpr bool I8 = decltype(i8)::value, FAR = decltype(far)::value;
        return pairs == HALVES ? block_append_kernel<HALVES, I8, FAR> : pairs == NEIGHBOURS ? block_append_kernel<NEIGHBOURS, I8, FAR>
                                                                                            : block_append_kernel<ODD_HALVES, I8, FAR>;
    };
    const bool far = g.table_rows < block;
    auto* kernel = r.e4m3 ? (far ? pick(std::false_type{}, std::true_type{}) : pick(std::false_type{}, std::false_type{}))
                          : (far ? pick(std::true_type{}, std::true_type{}) : pick(std::true_type{}, std::false_type{}));
    if (smem > 40 << 10) {                   // the kernel has some of its own beside it
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)BA_TABLE);
        if (e != cudaSuccess) return e;
    }
    return launch_pdl(kernel, dim3((unsigned)(g.kv_ctas + q_ctas)), BA_THREADS, smem, st, p, g);
}

}  // namespace affqmm
