// rope_pieces.cuh -- what the two appends to a paged cache share: bf16 and
// e4m3 conversions, and the sine and cosine of a pair's turn.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "affqmm_paged.h"

namespace affqmm {

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

// n / d by m = ceil(2^32 / d), exact for n < 2^32 / d (heads <= 8192, pieces <= 512)
__device__ __forceinline__ int over(int n, uint32_t m, int d) { return d == 1 ? n : (int)__umulhi((uint32_t)n, m); }

// The sine and cosine by which pair i of token t turns.
__device__ __forceinline__ void turn_of(const RopeParams& p, int64_t t, int i, float* sine, float* cosine) {
    const int a = p.axis ? min((int)p.axis[i], p.axes - 1) : 0;
    const int64_t pos = p.positions[a * p.pos_stride + t];
    const int64_t phase = (int64_t)((uint64_t)pos * (uint64_t)p.turns[i]);   // modulo a whole turn
    sincospif((float)(int32_t)(phase >> 32) * 0x1p-31f, sine, cosine);
}

}  // namespace affqmm
