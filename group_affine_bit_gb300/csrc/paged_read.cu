// paged_read.cu -- tokens of the requests of a paged cache as rows of bf16:
// row starts[b] + j is token first[b] + j of request b, its stored values or
// its codes times their scale, rounded once.
//
// Bound by memory: a value is read once (two bytes, or one) and written once
// (two).  A CTA takes a few rows, whose requests, pages and places its first
// threads find (the request by bisection of `starts`, which are brought to
// shared memory first), and all heads of k and v; a thread takes eight
// neighbouring values, 16 bytes to write.
#include "affqmm_internal.h"
#include "affqmm_paged.h"
#include "rope_pieces.cuh"

namespace affqmm {
namespace {

constexpr int PR_THREADS = 256, PR_ROWS = 32;   // most rows of a CTA
constexpr int PR_STARTS = 2048;                 // most requests whose starts shared memory holds

// n / d by m = ceil(2^32 / d) where that is exact (m not 0)
__device__ __forceinline__ int part_of(int n, uint32_t m, int d) { return m ? (int)__umulhi((uint32_t)n, m) : n / d; }

template <int KIND>
__device__ __forceinline__ uint4 eight(const uint8_t* from, float scale) {
    if constexpr (KIND == READ_BF16) {
        return __ldcs(reinterpret_cast<const uint4*>(from));
    } else {
        const uint2 w = __ldcs(reinterpret_cast<const uint2*>(from));
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t c = (i < 4 ? w.x : w.y) >> (8 * (i & 3)) & 0xffu;
            if constexpr (KIND == READ_I8_BLOCKS) x[i] = (float)(int8_t)c * scale;
            else x[i] = __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)c, __NV_E4M3))) * scale;
        }
        return make_uint4(bf2(x[0], x[1]), bf2(x[2], x[3]), bf2(x[4], x[5]), bf2(x[6], x[7]));
    }
}

template <int KIND>
__global__ void __launch_bounds__(PR_THREADS) paged_read_kernel(const __grid_constant__ ReadParams p, int rows, int pieces, uint32_t m_pieces,
                                                                int per_row, uint32_t m_row) {
    constexpr bool BLOCKS = KIND == READ_E4M3_BLOCKS || KIND == READ_I8_BLOCKS;
    __shared__ int64_t at[PR_ROWS], scale_at[PR_ROWS];   // of the row's token in the cache (-1: none), and of its block's scales
    __shared__ int32_t kept[PR_STARTS];
    __shared__ int rows_here;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t row0 = (int64_t)blockIdx.x * rows;
    const int tid = threadIdx.x;
    const int32_t* ends = p.starts + 1;                  // of the requests
    if (p.batch <= PR_STARTS) {
        for (int i = tid; i < p.batch; i += PR_THREADS) kept[i] = ends[i];
        ends = kept;
        __syncthreads();
    }
    if (tid < rows) {
        const int64_t row = row0 + tid, end = min((int64_t)ends[p.batch - 1], p.rows);
        if (tid == 0) rows_here = (int)max((int64_t)0, min((int64_t)rows, end - row0));
        if (p.status && row == 0 && ends[p.batch - 1] > p.rows) atomicOr(p.status, 2u);
        if (row < end) {
            int lo = 0, hi = p.batch - 1;                // the first request that ends behind the row
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (ends[mid] > row) hi = mid;
                else lo = mid + 1;
            }
            const int64_t token = (p.first ? (int64_t)p.first[lo] : 0) + row - (lo > 0 ? ends[lo - 1] : p.starts[0]);
            int page = -1;
            if (token >= 0 && token < (int64_t)p.wide << p.page_shift) page = p.table[lo * p.table_stride + (token >> p.page_shift)];
            const bool there = page >= 0 && page < p.pages;
            const int place = (int)(token & ((1 << p.page_shift) - 1));
            at[tid] = there ? page * p.page_bytes + place * p.token_bytes : -1;
            if (BLOCKS) scale_at[tid] = page * p.s_ps + (int64_t)(place >> p.block_shift) * p.s_bs;
            if (!there && p.status) atomicOr(p.status, 2u);
        }
    }
    __syncthreads();
    const int all = rows_here * per_row;                 // a row's pieces of k, then of v
#pragma unroll 4
    for (int i = tid; i < all; i += PR_THREADS) {
        const int r = part_of(i, m_row, per_row), x = i - r * per_row;
        const bool is_v = x >= per_row >> 1;
        const int y = is_v ? x - (per_row >> 1) : x, h = part_of(y, m_pieces, pieces), d = 8 * (y - h * pieces);
        const int64_t row = row0 + r;
        uint16_t* to = is_v ? p.v + row * p.v_ts + h * p.v_hs + d : p.k + row * p.k_ts + h * p.k_hs + d;
        uint4 w = make_uint4(0, 0, 0, 0);
        if (at[r] >= 0) {
            const float* scales = is_v ? p.v_scale : p.k_scale;
            float scale = 1.f;
            if (BLOCKS) scale = scales[scale_at[r] + h * p.s_hs];
            else if (KIND == READ_E4M3 && scales) scale = scales[h];
            w = eight<KIND>((is_v ? p.vc : p.kc) + at[r] + h * p.head_bytes + (KIND == READ_BF16 ? 2 * d : d), scale);
        }
        __stcs(reinterpret_cast<uint4*>(to), w);
    }
}

}  // namespace

cudaError_t launch_paged_read(const ReadParams& p, int kind, int sms, cudaStream_t st) {
    // a CTA's first threads find its rows while nothing is read: many rows to each, where there are enough of them
    const int rows = p.rows >= 16 * PR_ROWS * (int64_t)sms ? PR_ROWS : p.rows >= 64 * (int64_t)sms ? 8 : 1;
    const int pieces = p.dim / 8, per_row = 2 * p.heads * pieces;
    auto reciprocal = [](int64_t most, int d) {          // of numbers below `most`
        return d > 1 && most * d < (int64_t)1 << 32 ? (uint32_t)((((uint64_t)1 << 32) + d - 1) / d) : 0u;
    };
    auto* kernel = kind == READ_BF16 ? paged_read_kernel<READ_BF16> : kind == READ_E4M3 ? paged_read_kernel<READ_E4M3>
                   : kind == READ_E4M3_BLOCKS ? paged_read_kernel<READ_E4M3_BLOCKS> : paged_read_kernel<READ_I8_BLOCKS>;
    return launch_pdl(kernel, dim3((unsigned)((p.rows + rows - 1) / rows)), PR_THREADS, 0, st, p, rows, pieces, reciprocal(per_row, pieces), per_row,
                      reciprocal((int64_t)PR_ROWS * per_row, per_row));
}

}  // namespace affqmm
