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
// a token's heads.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "affqmm_internal.h"
#include "affqmm_paged.h"

namespace affqmm {
namespace {

constexpr int RA_THREADS = 256;

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[8]) {
    x[0] = bf_lo(w.x), x[1] = bf_hi(w.x), x[2] = bf_lo(w.y), x[3] = bf_hi(w.y);
    x[4] = bf_lo(w.z), x[5] = bf_hi(w.z), x[6] = bf_lo(w.w), x[7] = bf_hi(w.w);
}

__device__ __forceinline__ uint32_t bf2(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}

// Where a value goes: q's output rows (bf16), or a row of the cache in its type.
struct Row {
    uint8_t* p;
    float scale;   // e4m3: values are divided by it
    bool bytes;    // e4m3
};

__device__ __forceinline__ void put8(const Row& r, int d, const float (&x)[8]) {
    if (r.bytes) {
        const float s = r.scale;
        const uint32_t lo = e4m3x2(x[0] / s, x[1] / s) | (e4m3x2(x[2] / s, x[3] / s) << 16);
        const uint32_t hi = e4m3x2(x[4] / s, x[5] / s) | (e4m3x2(x[6] / s, x[7] / s) << 16);
        *reinterpret_cast<uint2*>(r.p + d) = make_uint2(lo, hi);
    } else {
        *reinterpret_cast<uint4*>(r.p + 2 * d) =
            make_uint4(bf2(x[0], x[1]), bf2(x[2], x[3]), bf2(x[4], x[5]), bf2(x[6], x[7]));
    }
}

__device__ __forceinline__ void put1(const Row& r, int d, float x) {
    if (r.bytes) r.p[d] = (uint8_t)e4m3x2(x / r.scale, 0.f);
    else *reinterpret_cast<__nv_bfloat16*>(r.p + 2 * d) = __float2bfloat16_rn(x);
}

// WIDE: eight neighbouring values (half pairs: twice eight) to a thread, where
// rotary / 2 (half pairs) or rotary / 8 allows it; otherwise a pair or a
// single value to a thread.
template <bool NEIGHBOUR, bool WIDE>
__global__ void __launch_bounds__(RA_THREADS) rope_append_kernel(RopeParams p) {
    __shared__ __align__(16) float2 turn[256];   // (cos, sin) of the token's pairs
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t t = blockIdx.x;
    const int half = p.rotary >> 1, D = p.dim;
    for (int i = threadIdx.x; i < half; i += RA_THREADS) {
        const int a = p.axis ? min((int)p.axis[i], p.axes - 1) : 0;
        const int64_t pos = p.positions[a * p.pos_stride + t];
        const int64_t phase = (int64_t)((uint64_t)pos * (uint64_t)p.turns[i]);   // modulo a whole turn
        float s, c;
        sincospif((float)(int32_t)(phase >> 32) * 0x1p-31f, &s, &c);
        turn[i] = make_float2(c, s);
    }
    const int32_t slot = p.slots[t];
    const int64_t page = slot >> p.page_shift;
    const bool kept = slot >= 0 && page < p.pages;
    if (slot < -1 || (slot >= 0 && !kept))
        if (p.status && threadIdx.x == 0 && blockIdx.y == 0) atomicOr(p.status, 2u);
    const int64_t at = page * p.page_bytes + (int64_t)(slot & ((1 << p.page_shift) - 1)) * p.token_bytes;
    __syncthreads();

    const int spun = WIDE ? (NEIGHBOUR ? p.rotary >> 3 : p.rotary >> 4) : half;   // work items that turn, of a head
    const int per = spun + (WIDE ? (D - p.rotary) >> 3 : D - p.rotary);
    const int per_v = WIDE ? D >> 3 : D;
    const int turned = (p.heads_q + p.heads_kv) * per, items = turned + p.heads_kv * per_v;
    for (int idx = blockIdx.y * RA_THREADS + threadIdx.x; idx < items; idx += gridDim.y * RA_THREADS) {
        const uint16_t* src;
        Row dst;
        int it;
        bool value = false;
        if (idx < turned) {
            const int h = idx / per;
            it = idx - h * per;
            if (h < p.heads_q) {
                src = p.q + t * p.q_ts + h * p.q_hs;
                dst.p = reinterpret_cast<uint8_t*>(p.out + t * p.o_ts + h * p.o_hs);
                dst.bytes = false;
            } else {
                if (!kept) continue;
                const int hk = h - p.heads_q;
                src = p.k + t * p.k_ts + hk * p.k_hs;
                dst.p = p.kc + at + hk * p.head_bytes;
                dst.bytes = p.e4m3;
                dst.scale = p.k_scale ? p.k_scale[hk] : 1.f;
            }
        } else {
            if (!kept) continue;
            const int hk = (idx - turned) / per_v;
            it = idx - turned - hk * per_v;
            src = p.v + t * p.v_ts + hk * p.v_hs;
            dst.p = p.vc + at + hk * p.head_bytes;
            dst.bytes = p.e4m3;
            dst.scale = p.v_scale ? p.v_scale[hk] : 1.f;
            value = true;
        }
        if constexpr (WIDE) {
            if (value || it >= spun) {   // as it is
                const int d = value ? 8 * it : p.rotary + 8 * (it - spun);
                float x[8];
                unpack8(*reinterpret_cast<const uint4*>(src + d), x);
                put8(dst, d, x);
            } else if constexpr (NEIGHBOUR) {
                float x[8], y[8];
                unpack8(*reinterpret_cast<const uint4*>(src + 8 * it), x);
                const float4* cs = reinterpret_cast<const float4*>(turn + 4 * it);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float4 w = cs[e];
                    y[4 * e] = x[4 * e] * w.x - x[4 * e + 1] * w.y;
                    y[4 * e + 1] = x[4 * e] * w.y + x[4 * e + 1] * w.x;
                    y[4 * e + 2] = x[4 * e + 2] * w.z - x[4 * e + 3] * w.w;
                    y[4 * e + 3] = x[4 * e + 2] * w.w + x[4 * e + 3] * w.z;
                }
                put8(dst, 8 * it, y);
            } else {
                float a[8], b[8], ya[8], yb[8];
                unpack8(*reinterpret_cast<const uint4*>(src + 8 * it), a);
                unpack8(*reinterpret_cast<const uint4*>(src + half + 8 * it), b);
                const float4* cs = reinterpret_cast<const float4*>(turn + 8 * it);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float4 w = cs[e];
                    ya[2 * e] = a[2 * e] * w.x - b[2 * e] * w.y;
                    yb[2 * e] = a[2 * e] * w.y + b[2 * e] * w.x;
                    ya[2 * e + 1] = a[2 * e + 1] * w.z - b[2 * e + 1] * w.w;
                    yb[2 * e + 1] = a[2 * e + 1] * w.w + b[2 * e + 1] * w.z;
                }
                put8(dst, 8 * it, ya);
                put8(dst, half + 8 * it, yb);
            }
        } else {
            if (value || it >= spun) {
                const int d = value ? it : p.rotary + it - spun;
                put1(dst, d, __uint_as_float((uint32_t)src[d] << 16));
            } else {
                const int da = NEIGHBOUR ? 2 * it : it, db = NEIGHBOUR ? 2 * it + 1 : it + half;
                const float a = __uint_as_float((uint32_t)src[da] << 16), b = __uint_as_float((uint32_t)src[db] << 16);
                const float2 w = turn[it];
                put1(dst, da, a * w.x - b * w.y);
                put1(dst, db, a * w.y + b * w.x);
            }
        }
    }
}

}  // namespace

cudaError_t launch_rope_append(const RopeParams& p, int sms, cudaStream_t st) {
    const bool wide = p.neighbour ? p.rotary % 8 == 0 : p.rotary % 16 == 0;
    const int per = wide ? (p.neighbour ? p.dim / 8 : p.rotary / 16 + (p.dim - p.rotary) / 8) : p.dim - p.rotary / 2;
    const int items = (p.heads_q + p.heads_kv) * per + p.heads_kv * (wide ? p.dim / 8 : p.dim);
    // with few tokens, as many CTAs a token as fill the SMs and find an item for each thread
    int64_t split = (sms + p.tokens - 1) / p.tokens;
    const int most = (items + RA_THREADS - 1) / RA_THREADS;
    if (split > most) split = most;
    if (split < 1) split = 1;
    const dim3 grid((unsigned)p.tokens, (unsigned)split);
    if (p.neighbour)
        return wide ? launch_pdl(rope_append_kernel<true, true>, grid, RA_THREADS, 0, st, p)
                    : launch_pdl(rope_append_kernel<true, false>, grid, RA_THREADS, 0, st, p);
    return wide ? launch_pdl(rope_append_kernel<false, true>, grid, RA_THREADS, 0, st, p)
                : launch_pdl(rope_append_kernel<false, false>, grid, RA_THREADS, 0, st, p);
}

}  // namespace affqmm
