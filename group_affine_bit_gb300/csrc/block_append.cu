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

constexpr int BA_THREADS = 128, BA_WARPS = BA_THREADS / 32;
constexpr int HOLD = 4;                  // chunks of 16 values that a lane keeps between the maximum and the codes
constexpr size_t BA_TABLE = 96 << 10;    // most shared memory for sines

// How a head's values pair: HALVES i with i + rotary / 2, in whole chunks of
// 8 pairs (rotary a multiple of 16); NEIGHBOURS 2i with 2i + 1; ODD_HALVES as
// HALVES, at any even rotary.
enum Pairs { HALVES, NEIGHBOURS, ODD_HALVES };

// Eight pairs of a head: chunk c has the pairs 8c .. 8c + 7, where values that do not turn are pairs of neighbours
// (HALVES: of one run of eight and the next).
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
__device__ __forceinline__ void load_chunk(const uint16_t* src, int c, int half, Chunk& x) {
    if constexpr (PAIRS == HALVES) {
        int d0, d1;
        runs_of(c, half, d0, d1);
        unpack8(*reinterpret_cast<const uint4*>(src + d0), x.a);
        unpack8(*reinterpret_cast<const uint4*>(src + d1), x.b);
    } else if constexpr (PAIRS == NEIGHBOURS) {
        float lo[8], hi[8];
        unpack8(*reinterpret_cast<const uint4*>(src + 16 * c), lo);
        unpack8(*reinterpret_cast<const uint4*>(src + 16 * c + 8), hi);
#pragma unroll
        for (int e = 0; e < 4; ++e) x.a[e] = lo[2 * e], x.b[e] = lo[2 * e + 1], x.a[e + 4] = hi[2 * e], x.b[e + 4] = hi[2 * e + 1];
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int i = 8 * c + e, d0 = i < half ? i : 2 * i, d1 = i < half ? i + half : 2 * i + 1;
            x.a[e] = __uint_as_float((uint32_t)src[d0] << 16);
            x.b[e] = __uint_as_float((uint32_t)src[d1] << 16);
        }
    }
}

// The sines of chunk c's pairs, of a token's table.
template <int PAIRS>
__device__ __forceinline__ void sines_of(int c, int half, const float* cosines, const float* sines, float (&co)[8], float (&si)[8]) {
    if constexpr (PAIRS == HALVES) {
        if (8 * c >= half) return;
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
}
template <int PAIRS>
__device__ __forceinline__ void turn_chunk(Chunk& x, int c, int half, const float (&co)[8], const float (&si)[8]) {
    if (8 * c >= half) return;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        if (PAIRS != HALVES && 8 * c + e >= half) continue;
        const float a = x.a[e], b = x.b[e];
        x.a[e] = a * co[e] - b * si[e];
        x.b[e] = a * si[e] + b * co[e];
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
    int q_parts;                         // CTAs to a token of q
    int table_rows;                      // rows whose sines shared memory holds
    int chunks;                          // of a head
    uint32_t m_chunks, m_half, m_parts, m_q_parts;
};

// One block's rows t .. t + n - 1 of the call, of one key head: x at `src` (rows src_ts apart), codes at `codes`.
template <int PAIRS, bool I8>
__device__ __forceinline__ void write_block(const BlockParams& p, const Grid& gr, int64_t t, int n, bool fresh, const uint16_t* src, int64_t src_ts,
                                            uint8_t* codes, float* scale_at, int half, const float* cosines, const float* sines) {
    const int lane = threadIdx.x & 31, all = n * gr.chunks;
    const int32_t* slots = p.rope.slots + t;
    const int bs = p.block_shift;
    const float old = fresh ? 0.f : fminf(fmaxf(*scale_at, kLeastScale), kMostScale);
    auto chunk = [&](int i, Chunk& x) {
        const int r = over(i, gr.m_chunks, gr.chunks), c = i - r * gr.chunks;
        load_chunk<PAIRS>(src + (int64_t)r * src_ts, c, half, x);
        float co[8], si[8];
        if (r < gr.table_rows) {
            sines_of<PAIRS>(c, half, cosines + r * half, sines + r * half, co, si);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (8 * c + e < half) turn_of(p.rope, t + r, 8 * c + e, si + e, co + e);
        }
        turn_chunk<PAIRS>(x, c, half, co, si);
    };
    auto write = [&](int i, const Chunk& x, float by) {
        const int r = over(i, gr.m_chunks, gr.chunks), c = i - r * gr.chunks;
        store_codes<PAIRS, I8>(codes + (int64_t)(slots[r] & ((1 << bs) - 1)) * p.rope.token_bytes, c, half, x, by);
    };
    Chunk held[HOLD];
    float top = 0.f;
    const bool keep = all <= 32 * HOLD;
    if (keep) {
#pragma unroll
        for (int j = 0; j < HOLD; ++j)
            if (lane + 32 * j < all) {
                chunk(lane + 32 * j, held[j]);
                top = fmaxf(top, top_of(held[j]));
            }
    } else {
#pragma unroll 1
        for (int i = lane; i < all; i += 32) {
            chunk(i, held[0]);
            top = fmaxf(top, top_of(held[0]));
        }
    }
    top = __uint_as_float(__reduce_max_sync(~0u, __float_as_uint(top)));
    const float scale = fmaxf(old, scale_for<I8>(top));
    if (lane == 0) *scale_at = scale;
    if (old > 0.f && old < scale) {
        // the block's codes to the new scale; those of this call's tokens are written after
        const float by = __fdiv_rn(old, scale);
        const int pieces = p.rope.dim >> 4;
#pragma unroll 1
        for (int i = lane; i < pieces << bs; i += 32) {
            const int r = over(i, gr.m_chunks, gr.chunks), c = i - r * pieces;
            uint4* at = reinterpret_cast<uint4*>(codes + (int64_t)r * p.rope.token_bytes + 16 * c);
            uint4 w = *at;
            for (uint32_t* u : {&w.x, &w.y, &w.z, &w.w}) {
                float x[4];
                values4<I8>(*u, x);
                *u = codes4<I8>(x[0], x[1], x[2], x[3], by);
            }
            *at = w;
        }
        __syncwarp();
    }
    const float by = __frcp_rn(scale);
    if (keep) {
#pragma unroll
        for (int j = 0; j < HOLD; ++j)
            if (lane + 32 * j < all) write(lane + 32 * j, held[j], by);
    } else {
#pragma unroll 1
        for (int i = lane; i < all; i += 32) {
            chunk(i, held[0]);
            write(i, held[0], by);
        }
    }
}

template <int PAIRS, bool I8>
__global__ void __launch_bounds__(BA_THREADS) block_append_kernel(const __grid_constant__ BlockParams p, const __grid_constant__ Grid gr) {
    extern __shared__ __align__(16) float table[];       // cosines, sines: [row][rotary / 2]
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const RopeParams& r = p.rope;
    const int half = r.rotary >> 1, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    float* cosines = table;
    if ((int)blockIdx.x >= gr.kv_ctas) {
        // ================= q of one token
        const int at = (int)blockIdx.x - gr.kv_ctas;
        const int64_t t = over(at, gr.m_q_parts, gr.q_parts);
        const int part = at - (int)t * gr.q_parts;
        float* sines = table + half;
        for (int i = tid; i < half; i += BA_THREADS) turn_of(r, t, i, sines + i, cosines + i);
        __syncthreads();
        for (int i = part * BA_THREADS + tid; i < r.heads_q * gr.chunks; i += gr.q_parts * BA_THREADS) {
            const int h = over(i, gr.m_chunks, gr.chunks), c = i - h * gr.chunks;
            Chunk x;
            load_chunk<PAIRS>(r.q + t * r.q_ts + h * r.q_hs, c, half, x);
            float co[8], si[8];
            sines_of<PAIRS>(c, half, cosines, sines, co, si);
            turn_chunk<PAIRS>(x, c, half, co, si);
            store_bf16<PAIRS>(r.out + t * r.o_ts + h * r.o_hs, c, half, x);
        }
        return;
    }
    // ================= k and v of the blocks that begin, for this call, in these rows
    const int64_t t0 = (int64_t)over((int)blockIdx.x, gr.m_parts, gr.parts) * gr.rows;
    const int part = (int)blockIdx.x - (int)(t0 / gr.rows) * gr.parts;
    const int units = 2 * r.heads_kv, u0 = part * units / gr.parts, u1 = (part + 1) * units / gr.parts;   // k's heads, then v's
    const int bs = p.block_shift;
    float* sines = table + gr.table_rows * half;
#pragma unroll 1
    for (int64_t t = t0; t < min(t0 + gr.rows, r.tokens); ++t) {
        const int32_t slot = r.slots[t];
        const int64_t page = slot >> r.page_shift;
        if (slot < 0 || page >= r.pages) {
            if (slot != -1 && r.status && part == 0 && tid == 0) atomicOr(r.status, 2u);
            continue;
        }
        const int block = slot >> bs;
        if (t > 0 && r.slots[t - 1] >= 0 && r.slots[t - 1] >> bs == block) continue;
        int n = 0;
        bool fresh = false;
        for (;;) {
            const int64_t next = t + n + lane;
            const int32_t s = next < r.tokens ? r.slots[next] : -1;
            const uint32_t same = __ballot_sync(~0u, s >= 0 && s >> bs == block), first = __ballot_sync(~0u, (s & ((1 << bs) - 1)) == 0);
            const int run = same == ~0u ? 32 : __ffs(~same) - 1;
            fresh |= (first & (run == 32 ? ~0u : (1u << run) - 1u)) != 0;
            n += run;
            if (run < 32 || n >= 1 << bs) break;
        }
        n = min(n, 1 << bs);                 // more would name a slot twice
        if (u0 < r.heads_kv) {
            const int many = min(n, gr.table_rows) * half;
            for (int i = tid; i < many; i += BA_THREADS) {
                const int row = over(i, gr.m_half, half);
                turn_of(r, t + row, i - row * half, sines + i, cosines + i);
            }
            __syncthreads();
        }
        const int first_of_block = (block << bs) & ((1 << r.page_shift) - 1);
        const int64_t at = page * r.page_bytes + first_of_block * r.token_bytes, scale_at = page * p.s_ps + (int64_t)(first_of_block >> bs) * p.s_bs;
        for (int u = u0 + warp; u < u1; u += BA_WARPS) {
            if (u < r.heads_kv)
                write_block<PAIRS, I8>(p, gr, t, n, fresh, r.k + t * r.k_ts + u * r.k_hs, r.k_ts, r.kc + at + u * r.head_bytes,
                                       p.k_scales + scale_at + u * p.s_hs, half, cosines, sines);
            else {
                const int h = u - r.heads_kv;
                write_block<HALVES, I8>(p, gr, t, n, fresh, r.v + t * r.v_ts + h * r.v_hs, r.v_ts, r.vc + at + h * r.head_bytes,
                                        p.v_scales + scale_at + h * p.s_hs, 0, cosines, sines);
            }
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
    // k and v: CTAs enough that every SM has several, a warp to a unit at most, and then rows to each of them
    const int units = 2 * r.heads_kv, most = (units + BA_WARPS - 1) / BA_WARPS;
    int64_t parts = (4 * sms + r.tokens - 1) / r.tokens;
    if (parts < 2) parts = 2;
    g.parts = (int)(parts < most ? parts : most);
    g.rows = r.tokens * g.parts > 16 * sms ? 8 : 1;
    g.kv_ctas = (int)((r.tokens + g.rows - 1) / g.rows) * g.parts;
    g.table_rows = half ? (int)(BA_TABLE / (8 * half)) : block;
    if (g.table_rows > block) g.table_rows = block;
    // q: as many CTAs a token as fill the SMs and find a chunk for each thread
    int64_t split = (2 * sms + r.tokens - 1) / r.tokens;
    const int wide = (r.heads_q * g.chunks + BA_THREADS - 1) / BA_THREADS;
    g.q_parts = (int)(split < wide ? split : wide);
    g.m_chunks = reciprocal(g.chunks), g.m_half = reciprocal(half), g.m_parts = reciprocal(g.parts), g.m_q_parts = reciprocal(g.q_parts);
    const size_t smem = (size_t)(g.table_rows > 1 ? g.table_rows : 1) * 8 * half;
    auto pick = [&](auto i8) {
        constexpr bool I8 = decltype(i8)::value;
        return pairs == HALVES ? block_append_kernel<HALVES, I8> : pairs == NEIGHBOURS ? block_append_kernel<NEIGHBOURS, I8>
                                                                                       : block_append_kernel<ODD_HALVES, I8>;
    };
    auto* kernel = r.e4m3 ? pick(std::false_type{}) : pick(std::true_type{});
    if (smem > 48 << 10) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)BA_TABLE);
        if (e != cudaSuccess) return e;
    }
    return launch_pdl(kernel, dim3((unsigned)(g.kv_ctas + r.tokens * g.q_parts)), BA_THREADS, smem, st, p, g);
}

}  // namespace affqmm
