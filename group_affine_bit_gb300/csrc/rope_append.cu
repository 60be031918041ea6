// rope_append.cu -- rotary positions on a step's q and k, and k and v written
// to their slots of the paged cache:
//
//     phi_i = 2 pi frac(pos[axis_i] * turns_i / 2^64)
//     (a, b) -> (a cos phi_i - b sin phi_i, a sin phi_i + b cos phi_i)
//
// for the pairs i < rotary / 2 of every q and k head -- values (i, i + rotary
// / 2), or (2i, 2i + 1) where neighbours pair -- the other values as they are.
// Each pair turns by the position on its own axis (time, height, width).
//
// The frequency is a 64-bit fraction of a turn, so pos * turns modulo 2^64 is
// the phase exactly, at any position: the whole turns fall off the top of the
// integer product.  (A product in fp32 is off by up to 2^-24 of the angle,
// 0.02 rad at position 262144.)  Its upper 32 bits go to sincospi in fp32,
// which leaves 2^-25 of a turn; the rotation is done in fp32 and rounded once,
// to bf16 or to the cache's e4m3.
//
// Bound by memory: each value is read once and written once, 16 bytes a
// thread.  One CTA takes one token, so that the token's sines are made once
// and serve every head from shared memory; with few tokens several CTAs share
// a token's heads.  The instructions beside the bytes are kept few: v and what
// does not turn is copied as it is (bf16), and a piece's head comes from one
// multiplication.  A call whose output is more than half of L2 (126 MB) loads
// and stores what leaves L2 first: 8192 tokens, 201 MB, in 32.6 us instead of
// 35.1; a smaller one leaves its output there for the attention that reads it.
#include "affqmm_internal.h"
#include "affqmm_paged.h"
#include "rope_pieces.cuh"

namespace affqmm {
namespace {

constexpr int RA_THREADS = 128;

// Where a value goes: q's output rows (bf16), or a row of the cache in its type.
struct Row {
    uint8_t* p;
    float scale;   // e4m3: values are divided by it
    bool bytes;    // e4m3
};

// STREAM: loads and stores that leave L2 first.
template <bool STREAM>
__device__ __forceinline__ uint4 load16(const uint16_t* src) {
    const uint4* from = reinterpret_cast<const uint4*>(src);
    if constexpr (STREAM) return __ldcs(from);
    else return *from;
}
template <bool STREAM>
__device__ __forceinline__ void store16(const Row& r, int d, const uint4& w) {
    if constexpr (STREAM) __stcs(reinterpret_cast<uint4*>(r.p + 2 * d), w);
    else *reinterpret_cast<uint4*>(r.p + 2 * d) = w;
}

template <bool STREAM>
__device__ __forceinline__ void put8(const Row& r, int d, const float (&x)[8]) {
    if (r.bytes) {
        const float s = r.scale;
        const uint32_t lo = e4m3x2(x[0] / s, x[1] / s) | (e4m3x2(x[2] / s, x[3] / s) << 16);
        const uint32_t hi = e4m3x2(x[4] / s, x[5] / s) | (e4m3x2(x[6] / s, x[7] / s) << 16);
        *reinterpret_cast<uint2*>(r.p + d) = make_uint2(lo, hi);
    } else {
        store16<STREAM>(r, d, make_uint4(bf2(x[0], x[1]), bf2(x[2], x[3]), bf2(x[4], x[5]), bf2(x[6], x[7])));
    }
}

__device__ __forceinline__ void put1(const Row& r, int d, float x) {
    if (r.bytes) r.p[d] = (uint8_t)e4m3x2(x / r.scale, 0.f);
    else *reinterpret_cast<__nv_bfloat16*>(r.p + 2 * d) = __float2bfloat16_rn(x);
}

template <bool STREAM>
__device__ __forceinline__ void copy8(const Row& r, int d, const uint16_t* src) {
    const uint4 w = load16<STREAM>(src + d);
    if (r.bytes) {
        float x[8];
        unpack8(w, x);
        put8<STREAM>(r, d, x);
    } else {
        store16<STREAM>(r, d, w);
    }
}

// WIDE: eight neighbouring values (half pairs: twice eight) to a thread, where
// rotary / 2 (half pairs) or rotary / 8 allows it; otherwise a pair or a
// single value to a thread.  The pieces of a head: `spun` that turn, `still`
// that do not, and `per_v` of v; m_*: their reciprocals.
template <bool NEIGHBOUR, bool WIDE, bool STREAM>
__global__ void __launch_bounds__(RA_THREADS) rope_append_kernel(RopeParams p, int spun, int still, int per_v, uint32_t m_spun,
                                                                 uint32_t m_still, uint32_t m_v) {
    __shared__ __align__(16) float cosines[256], sines[256];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t t = blockIdx.x;
    const int half = p.rotary >> 1, step = gridDim.y * RA_THREADS, idx0 = blockIdx.y * RA_THREADS + threadIdx.x;
    const int32_t slot = p.slots[t];
    for (int i = threadIdx.x; i < half; i += RA_THREADS) {
        turn_of(p, t, i, &sines[i], &cosines[i]);
    }
    const int64_t page = slot >> p.page_shift;
    const bool kept = slot >= 0 && page < p.pages;
    if (slot < -1 || (slot >= 0 && !kept))
        if (p.status && threadIdx.x == 0 && blockIdx.y == 0) atomicOr(p.status, 2u);
    const int64_t at = page * p.page_bytes + (int64_t)(slot & ((1 << p.page_shift) - 1)) * p.token_bytes;
    const uint16_t *q = p.q + t * p.q_ts, *k = p.k + t * p.k_ts, *v = p.v + t * p.v_ts;
    uint16_t* out = p.out + t * p.o_ts;
    // the source and the target of head h of q and k
    auto ends = [&](int h, const uint16_t*& src, Row& dst) {
        const int hk = h - p.heads_q;
        if (hk < 0) {
            src = q + h * p.q_hs;
            dst.p = reinterpret_cast<uint8_t*>(out + h * p.o_hs);
            dst.bytes = false;
        } else {
            src = k + hk * p.k_hs;
            dst.p = p.kc + at + hk * p.head_bytes;
            dst.bytes = p.e4m3;
            dst.scale = p.k_scale ? p.k_scale[hk] : 1.f;
        }
    };
    const int heads = p.heads_q + (kept ? p.heads_kv : 0);
    if (kept)
#pragma unroll 2
        for (int i = idx0; i < p.heads_kv * per_v; i += step) {
            const int h = over(i, m_v, per_v), d = i - h * per_v;
            const Row dst = {p.vc + at + h * p.head_bytes, p.v_scale ? p.v_scale[h] : 1.f, (bool)p.e4m3};
            if (WIDE) copy8<STREAM>(dst, 8 * d, v + h * p.v_hs);
            else put1(dst, d, __uint_as_float((uint32_t)v[h * p.v_hs + d] << 16));
        }
    for (int i = idx0; i < heads * still; i += step) {
        const int h = over(i, m_still, still), d = i - h * still;
        const uint16_t* src;
        Row dst;
        ends(h, src, dst);
        if (WIDE) copy8<STREAM>(dst, p.rotary + 8 * d, src);
        else put1(dst, p.rotary + d, __uint_as_float((uint32_t)src[p.rotary + d] << 16));
    }
    __syncthreads();
#pragma unroll 2
    for (int i = idx0; i < heads * spun; i += step) {
        const int h = over(i, m_spun, spun), piece = i - h * spun;
        const uint16_t* src;
        Row dst;
        ends(h, src, dst);
        if constexpr (!WIDE) {
            const int da = NEIGHBOUR ? 2 * piece : piece, db = NEIGHBOUR ? 2 * piece + 1 : piece + half;
            const float a = __uint_as_float((uint32_t)src[da] << 16), b = __uint_as_float((uint32_t)src[db] << 16);
            put1(dst, da, a * cosines[piece] - b * sines[piece]);
            put1(dst, db, a * sines[piece] + b * cosines[piece]);
        } else if constexpr (NEIGHBOUR) {
            float x[8], y[8];
            unpack8(load16<STREAM>(src + 8 * piece), x);
            const float4 c = *reinterpret_cast<const float4*>(cosines + 4 * piece), s = *reinterpret_cast<const float4*>(sines + 4 * piece);
            y[0] = x[0] * c.x - x[1] * s.x, y[1] = x[0] * s.x + x[1] * c.x;
            y[2] = x[2] * c.y - x[3] * s.y, y[3] = x[2] * s.y + x[3] * c.y;
            y[4] = x[4] * c.z - x[5] * s.z, y[5] = x[4] * s.z + x[5] * c.z;
            y[6] = x[6] * c.w - x[7] * s.w, y[7] = x[6] * s.w + x[7] * c.w;
            put8<STREAM>(dst, 8 * piece, y);
        } else {
            const uint4 wa = load16<STREAM>(src + 8 * piece), wb = load16<STREAM>(src + half + 8 * piece);
            float a[8], b[8], ya[8], yb[8];
            unpack8(wa, a);
            unpack8(wb, b);
#pragma unroll
            for (int e = 0; e < 8; e += 4) {
                const float4 c = *reinterpret_cast<const float4*>(cosines + 8 * piece + e), s = *reinterpret_cast<const float4*>(sines + 8 * piece + e);
                ya[e] = a[e] * c.x - b[e] * s.x, yb[e] = a[e] * s.x + b[e] * c.x;
                ya[e + 1] = a[e + 1] * c.y - b[e + 1] * s.y, yb[e + 1] = a[e + 1] * s.y + b[e + 1] * c.y;
                ya[e + 2] = a[e + 2] * c.z - b[e + 2] * s.z, yb[e + 2] = a[e + 2] * s.z + b[e + 2] * c.z;
                ya[e + 3] = a[e + 3] * c.w - b[e + 3] * s.w, yb[e + 3] = a[e + 3] * s.w + b[e + 3] * c.w;
            }
            put8<STREAM>(dst, 8 * piece, ya);
            put8<STREAM>(dst, half + 8 * piece, yb);
        }
    }
}

}  // namespace

cudaError_t launch_rope_append(const RopeParams& p, int sms, cudaStream_t st) {
    const bool wide = p.neighbour ? p.rotary % 8 == 0 : p.rotary % 16 == 0;
    const int spun = wide ? (p.neighbour ? p.rotary / 8 : p.rotary / 16) : p.rotary / 2;
    const int still = wide ? (p.dim - p.rotary) / 8 : p.dim - p.rotary, per_v = wide ? p.dim / 8 : p.dim;
    auto reciprocal = [](int d) { return d > 1 ? (uint32_t)((((uint64_t)1 << 32) + d - 1) / d) : 0u; };
    // with few tokens, as many CTAs a token as fill the SMs and find a piece for each thread
    int64_t split = (2 * sms + p.tokens - 1) / p.tokens;
    const int most = ((p.heads_q + p.heads_kv) * (spun > still ? spun : still) + RA_THREADS - 1) / RA_THREADS;
    if (split > most) split = most;
    if (split < 1) split = 1;
    const dim3 grid((unsigned)p.tokens, (unsigned)split);
    auto* kernel = p.neighbour ? (wide ? p.stream ? rope_append_kernel<true, true, true> : rope_append_kernel<true, true, false>
                                       : rope_append_kernel<true, false, false>)
                               : (wide ? p.stream ? rope_append_kernel<false, true, true> : rope_append_kernel<false, true, false>
                                       : rope_append_kernel<false, false, false>);
    return launch_pdl(kernel, grid, RA_THREADS, 0, st, p, spun, still, per_v, reciprocal(spun), reciprocal(still), reciprocal(per_v));
}

}  // namespace affqmm
