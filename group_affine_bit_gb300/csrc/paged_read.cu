// paged_read.cu -- tokens of the requests of a paged cache as rows of bf16:
// row starts[b] + j is token first[b] + j of request b, its stored values or
// its codes times their scale, rounded once.
//
// Bound by memory: a value is read once (two bytes, or one) and written once
// (two).  A CTA takes a few rows, whose requests, pages and places its first
// threads find (the request by bisection of `starts`, which are brought to shared
// memory first), and all heads of k and v; a thread has four pieces of k and of v
// in flight, of eight neighbouring values each, 16 bytes to write.  Measured
// (GB300, device time): 16 requests of up to 8192 tokens, int8, 372 MB, in 59.7
// us, 93 % of the copy rate (72 with one piece after the other: the loads'
// latency); 32,606 tokens of one head of 128 in 7.2 us (14.4 with 32 rows to every
// CTA, whose threads then had little to do).
#include <type_traits>

#include "affqmm_internal.h"
#include "affqmm_paged.h"
#include "rope_pieces.cuh"

namespace affqmm {
namespace {

constexpr int PR_THREADS = 256, PR_ROWS = 128;   // most rows of a CTA
constexpr int PR_BATCH = 4;                     // pieces of k and of v that a thread has in flight
constexpr int PR_STARTS = 2048;                 // most requests whose starts shared memory holds

// n / d by m = ceil(2^32 / d) where that is exact (m not 0)
__device__ __forceinline__ int part_of(int n, uint32_t m, int d) { return m ? (int)__umulhi((uint32_t)n, m) : n / d; }

// Eight stored values as they are read, and as bf16.
template <int KIND>
using Stored = std::conditional_t<KIND == READ_BF16, uint4, uint2>;

template <int KIND>
__device__ __forceinline__ uint4 eight(const Stored<KIND>& w, float scale) {
    if constexpr (KIND == READ_BF16) {
        return w;
    } else {
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
__global__ void __launch_bounds__(PR_THREADS, 4) paged_read_kernel(const __grid_constant__ ReadParams p, int rows, int pieces, uint32_t m_pieces,
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
    const int all = rows_here * per_row;                 // pieces of k, and of v
#pragma unroll 1
    for (int first = tid; first < all; first += PR_BATCH * PR_THREADS) {
        Stored<KIND> k[PR_BATCH], v[PR_BATCH];
        float ks[PR_BATCH], vs[PR_BATCH];
        auto place = [&](int j, int& r, int& h, int& d) {
            const int i = first + j * PR_THREADS;
            r = part_of(i, m_row, per_row);
            const int x = i - r * per_row;
            h = part_of(x, m_pieces, pieces), d = 8 * (x - h * pieces);
            return i < all;
        };
#pragma unroll
        for (int j = 0; j < PR_BATCH; ++j) {
            int r, h, d;
            const bool there = place(j, r, h, d) && at[r] >= 0;
            k[j] = v[j] = {};
            ks[j] = vs[j] = 1.f;
            if (there) {
                const int64_t from = at[r] + h * p.head_bytes + (KIND == READ_BF16 ? 2 * d : d);
                k[j] = __ldcs(reinterpret_cast<const Stored<KIND>*>(p.kc + from));
                v[j] = __ldcs(reinterpret_cast<const Stored<KIND>*>(p.vc + from));
                if (BLOCKS) {
                    const int64_t of = scale_at[r] + h * p.s_hs;
                    ks[j] = p.k_scale[of], vs[j] = p.v_scale[of];
                } else if (KIND == READ_E4M3) {
                    if (p.k_scale) ks[j] = p.k_scale[h];
                    if (p.v_scale) vs[j] = p.v_scale[h];
                }
            }
        }
#pragma unroll
        for (int j = 0; j < PR_BATCH; ++j) {
            int r, h, d;
            if (!place(j, r, h, d)) continue;
            __stcs(reinterpret_cast<uint4*>(p.k + (row0 + r) * p.k_ts + h * p.k_hs + d), eight<KIND>(k[j], ks[j]));
            __stcs(reinterpret_cast<uint4*>(p.v + (row0 + r) * p.v_ts + h * p.v_hs + d), eight<KIND>(v[j], vs[j]));
        }
    }
}

}  // namespace

cudaError_t launch_paged_read(const ReadParams& p, int kind, int sms, cudaStream_t st) {
    // rows to a CTA: two rounds of its threads, as finding the rows takes a while; fewer where that would leave SMs without
    // work, but not so few that threads are left without
    const int pieces = p.dim / 8, per_row = p.heads * pieces;
    const int64_t most = 2 * PR_BATCH * PR_THREADS / per_row, fair = p.rows / (4 * sms), least = PR_THREADS / per_row;
    const int64_t want = fair < least ? least : fair < most ? fair : most;
    const int rows = (int)(want < 1 ? 1 : want < PR_ROWS ? want : PR_ROWS);
    auto reciprocal = [](int64_t most, int d) {          // of numbers below `most`
        return d > 1 && most * d < (int64_t)1 << 32 ? (uint32_t)((((uint64_t)1 << 32) + d - 1) / d) : 0u;
    };
    auto* kernel = kind == READ_BF16 ? paged_read_kernel<READ_BF16> : kind == READ_E4M3 ? paged_read_kernel<READ_E4M3>
                   : kind == READ_E4M3_BLOCKS ? paged_read_kernel<READ_E4M3_BLOCKS> : paged_read_kernel<READ_I8_BLOCKS>;
    const int64_t ctas = p.rows > 0 ? (p.rows + rows - 1) / rows : 1;
    return launch_pdl(kernel, dim3((unsigned)ctas), PR_THREADS, 0, st, p, rows, pieces, reciprocal(per_row, pieces), per_row,
                      reciprocal((int64_t)PR_ROWS * per_row, per_row));
}

}  // namespace affqmm
