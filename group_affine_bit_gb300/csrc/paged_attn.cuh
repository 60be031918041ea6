// paged_attn.cuh -- attention of a request's newest tokens over its paged
// key-value cache:
//
//     s[r, key] = scale * q[r] . k[key],   key visible to token j of n when
//                 len - n + j - window < key <= len - n + j
//     out[r] = sum_key exp(s - lse) v[key],   lse = log sum_key exp(s)
//
// in one pass over the cache.  Bound by HBM: each visible key and value is
// read once, and the matrix work beside it is small (rows that share a key
// head: query heads of the group x tokens, 1 .. 64 to a tile).
//
// Roles.  A CTA has four consumer warps, one producer warp for K, one for V
// and one for q.  A tile is 64 keys.  The producers gather its rows through
// the block table (the next tile's entries are fetched ahead) with 16-byte
// asynchronous copies into a ring that K and V tiles share in turn; rows that
// no query may see, or whose table entry is out of range, are filled with
// zeros and not read.  They run ahead of the consumers across the borders of
// requests, so the memory pipeline does not drain there.
//
// Arithmetic.  Keys are the M side of the matrix instruction (m16n8k16) and
// query rows its N side, so that one to eight rows cost one instruction per 16
// x 16 keys x dims: S^T = K Q^T, a warp to 16 keys; then O^T = V^T P^T, a warp
// to a quarter of the dims, P^T through shared memory.  The running maximum is
// shared by the CTA and lazy: a tile is rescaled only if a score exceeds it by
// more than 2^8 (an OR over the barrier that P^T needs anyway), so most tiles
// cost one barrier and no shuffles.  Scores, maxima, sums and outputs are
// fp32.  P meets V in the matrix type.  Beside a bf16 cache it is the sum of two
// bf16 numbers, what the first leaves being in the second, each with its own
// matrix instruction: 16 bits of P instead of 8, so that the output's own
// rounding is what is left of the error (2-norm against 64 bits 0.0017; with
// one bf16 number 0.0023), for instructions that a memory-bound kernel has to
// spare.  Beside an e4m3 one it is one f16 (11 bits); f16 holds the cache's
// values exactly, and q is brought to f16 with a power of two per row, so that
// it keeps its eight bits.  The sum of P is taken before these roundings.
//
// Split.  All tiles of all (request, key head, row tile) units, in order, are
// cut into equal runs, one per CTA, so a batch of ragged lengths loads every
// SM alike; each CTA finds its run by a prefix sum over the lengths.  A unit
// that several runs share is joined by the CTA that finishes last, in run
// order: the same inputs give the same bits.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "affqmm_async.cuh"
#include "affqmm_internal.h"
#include "affqmm_paged.h"

namespace affqmm {
namespace attn {

constexpr int W = 4;                       // consumer warps
constexpr int CONSUMERS = 32 * W;
constexpr int THREADS = 32 * (W + 3);
constexpr int KEYS = kAttnKeys;
constexpr float LAZY = 8.f;                // log2 of how far a score may exceed the running maximum
constexpr size_t SM_SMEM = 233472;         // shared memory of an SM, 1 KB of it taken by each CTA
constexpr size_t CTA_SMEM = 232448;        // and what one CTA may have of it
constexpr size_t STATIC_SMEM = 512;        // above the kernel's few static variables
constexpr int MAX_SLOTS = 16;

template <int DP, int NT, bool E4M3>
struct Cfg {
    static constexpr int ES = E4M3 ? 1 : 2;
    static constexpr int ROWS = 8 * NT;
    static constexpr int PITCH = DP * ES;              // bytes of a cache row in shared memory
    static constexpr int CH = PITCH / 16;              // its 16-byte chunks
    static constexpr int TILE = KEYS * PITCH;
    static constexpr int QBYTES = ROWS * DP * 2;
    static constexpr int QBUF = (DP == 512 && NT > 1) ? 1 : 2;
    static constexpr int PN = E4M3 ? 1 : 2;            // numbers that make one P
    static constexpr int PBYTES = PN * NT * KEYS * 16; // [PN][NT][64 keys][8 rows] of 16 bits
    static constexpr int LOW = NT * KEYS * 16;         // from the first numbers to the second
    static constexpr int MT = DP / (16 * W);           // 16-dim tiles of a consumer warp
    static constexpr size_t FIXED = (size_t)QBUF * QBYTES + 2 * PBYTES + 2 * W * ROWS * 4 + QBUF * ROWS * 4 + 1024;
    static constexpr bool LIGHT = MT * NT * 4 + NT * 8 <= 64;   // registers allow two CTAs an SM
    static constexpr size_t HALF = SM_SMEM / 2 - 1024 - STATIC_SMEM;
    static constexpr int CPS = (LIGHT && FIXED + 4 * TILE <= HALF) ? 2 : 1;
    static constexpr size_t ROOM = (CPS == 2 ? HALF : CTA_SMEM - STATIC_SMEM) - FIXED;
    static constexpr int NS = ROOM / TILE > MAX_SLOTS ? MAX_SLOTS : (int)(ROOM / TILE);
    static constexpr size_t SMEM = FIXED + (size_t)NS * TILE;
    static constexpr size_t SLOT_FLOATS = (size_t)W * MT * NT * 32 * 4 + 2 * ROWS;
    static_assert(NS >= 3, "ring too short");
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
template <bool F16>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (F16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// two e4m3 values (the low 16 bits, the first in the low byte) -> f16x2, exact
__device__ __forceinline__ uint32_t e4m3_f16x2(uint32_t w) {
    uint32_t d;
    asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %1;\n cvt.rn.f16x2.e4m3x2 %0, lo;\n}\n" : "=r"(d) : "r"(w));
    return d;
}
__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
template <bool F16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    if constexpr (F16) {
        const __half2 v = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&v);
    } else {
        const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&v);
    }
}
__device__ __forceinline__ void st_shared(uint32_t addr, uint32_t v) {
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool real) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16u : 0u) : "memory");
}
// arrive on `bar` when this thread's copies so far have landed (counted in the barrier's own count)
__device__ __forceinline__ void cp_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void consumer_sync() { asm volatile("barrier.cta.sync 1, 128;" ::: "memory"); }
__device__ __forceinline__ bool consumer_any(bool v) {
    uint32_t r;
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred q, 1, 128, p;\n selp.u32 %0, 1, 0, q;\n}\n"
        : "=r"(r) : "r"((uint32_t)v) : "memory");
    return r != 0;
}
// 16-byte chunk `c` of row `row` of a tile whose rows have CH chunks: the
// eight rows that one ldmatrix phase reads fall into eight bank groups.
template <int CH>
__device__ __forceinline__ uint32_t chunk_at(int row, int c) {
    if constexpr (CH >= 8) return (uint32_t)(row * CH + (c ^ (row & 7))) * 16u;
    else return (uint32_t)(row * CH + (c ^ ((row >> 1) & (CH - 1)))) * 16u;
}

// What a request's tiles cover: keys lo .. hi - 1, tiles counted from `base`.
struct Span {
    int len, lo, hi, base, tiles;
};
__device__ __forceinline__ Span span_of(const AttnParams& p, int b) {
    Span s;
    const int64_t most = (int64_t)p.wide << p.page_shift;
    int len = p.lens[b];
    if (len > most) len = (int)most;
    s.len = max(len, 0);
    s.hi = s.len;
    s.lo = p.window > 0 ? max(0, s.len - p.tokens + 1 - p.window) : 0;
    s.base = s.lo & ~15;
    s.tiles = max(1, (s.hi - s.base + KEYS - 1) / KEYS);
    return s;
}

// The CTA's run, segment by segment: unit (request b, u = key head * row tiles + row tile), tiles t0 .. t1 - 1.
struct Walk {
    int b, u, t, t0, t1;
    int64_t left;      // tiles of the run not yet handed out
    int64_t unit0;     // number of the unit's first tile
    Span s;
    __device__ __forceinline__ bool next(const AttnParams& p, int units) {
        if (left <= 0) return false;
        if (t >= s.tiles) {
            unit0 += s.tiles;
            t = 0;
            if (++u == units) {
                u = 0;
                ++b;
                s = span_of(p, b);
            }
        }
        t0 = t;
        t1 = (int)min((int64_t)s.tiles, t0 + left);
        left -= t1 - t0;
        t = t1;
        return true;
    }
};

template <int DP, int NT, bool E4M3>
__global__ void __launch_bounds__(THREADS, Cfg<DP, NT, E4M3>::CPS) paged_attn_kernel(const __grid_constant__ AttnParams p) {
    using C = Cfg<DP, NT, E4M3>;
    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t* ring = smem;
    uint8_t* qbuf = ring + (size_t)C::NS * C::TILE;
    uint8_t* pbuf = qbuf + C::QBUF * C::QBYTES;
    float* red = reinterpret_cast<float*>(pbuf + 2 * C::PBYTES);      // [W][ROWS] maxima
    float* lred = red + W * C::ROWS;                                  // [W][ROWS] sums
    float* qscale = lred + W * C::ROWS;                               // [QBUF][ROWS] e4m3: what undoes q's power of two
    uint64_t* bars = reinterpret_cast<uint64_t*>(qscale + C::QBUF * C::ROWS);
    const uint32_t bar0 = smem_u32(bars);
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto empty = [&](int s) { return bar0 + 8u * (MAX_SLOTS + s); };
    auto qfull = [&](int s) { return bar0 + 8u * (2 * MAX_SLOTS + s); };
    auto qempty = [&](int s) { return bar0 + 8u * (2 * MAX_SLOTS + 2 + s); };
    __shared__ int64_t sums[THREADS / 32];
    __shared__ int64_t run_tiles, run_unit0, run_total, run_at;
    __shared__ int run_b;
    __shared__ uint32_t last_flag;

    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    if (tid == 0) {
        for (int s = 0; s < C::NS; ++s) {
            mbar_init(full(s), 32);
            mbar_init(empty(s), W);
        }
        for (int s = 0; s < C::QBUF; ++s) {
            mbar_init(qfull(s), 32);
            mbar_init(qempty(s), W);
        }
        fence_mbar_init();
    }
    // columns beyond the head's dim stay zero: nothing is copied there
    if (p.dim < DP) {
        uint4* z = reinterpret_cast<uint4*>(ring);
        for (int i = tid; i < C::NS * C::TILE / 16; i += THREADS) z[i] = make_uint4(0, 0, 0, 0);
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // ---- this CTA's run of tiles: a prefix sum over the requests' tiles
    const int units = p.heads_kv * p.row_tiles;
    {
        const int each = (p.batch + THREADS - 1) / THREADS;
        const int b0 = min(tid * each, p.batch), b1 = min(b0 + each, p.batch);
        int64_t mine = 0;
        for (int b = b0; b < b1; ++b) {
            if (blockIdx.x == 0 && p.user_status && (p.lens[b] < 0 || p.lens[b] > ((int64_t)p.wide << p.page_shift)))
                atomicOr(p.user_status, 2u);
            mine += (int64_t)span_of(p, b).tiles * units;
        }
        int64_t x = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t y = __shfl_up_sync(~0u, x, d);
            if (lane >= d) x += y;
        }
        if (lane == 31) sums[wid] = x;
        __syncthreads();
        int64_t before = 0, total = 0;
#pragma unroll
        for (int w = 0; w < THREADS / 32; ++w) {
            if (w < wid) before += sums[w];
            total += sums[w];
        }
        before += x - mine;
        // no run is empty: with fewer tiles than CTAs, the first `total` CTAs take one each
        const int64_t ctas = min((int64_t)gridDim.x, total), c = min((int64_t)blockIdx.x, ctas);
        const int64_t r0 = total * c / ctas, r1 = c < ctas ? total * (c + 1) / ctas : r0;
        if (tid == 0) run_tiles = r1 - r0, run_total = total;
        if (r1 > r0 && before <= r0 && r0 < before + mine) {
            int64_t at = before;
            int b = b0;
            for (;; ++b) {
                const int64_t n = (int64_t)span_of(p, b).tiles * units;
                if (r0 < at + n) break;
                at += n;
            }
            run_b = b;
            run_at = r0 - at;
            run_unit0 = at;
        }
        __syncthreads();
    }
    if (run_tiles == 0) return;
    const int64_t all_tiles = run_total, ctas = min((int64_t)gridDim.x, all_tiles);
    Walk walk;
    walk.b = run_b;
    walk.s = span_of(p, walk.b);
    walk.u = (int)(run_at / walk.s.tiles);
    walk.t = (int)(run_at - (int64_t)walk.u * walk.s.tiles);
    walk.unit0 = run_unit0 + (int64_t)walk.u * walk.s.tiles;
    walk.left = run_tiles;
    bool ok = true;                       // no bounded wait has given up; after one, no wait is made
    auto wait = [&](uint32_t bar, uint32_t parity) {
        if (ok) ok = mbar_wait(bar, parity);
    };

    if (wid == W || wid == W + 1) {
        // ================= producers: K tiles take the ring's even turns, V tiles the odd ones
        const bool is_v = wid == W + 1;
        const uint8_t* cache = is_v ? p.v : p.k;
        constexpr int CH = C::CH, RPI = CH >= 32 ? 1 : 32 / CH;     // rows of one warp-wide copy
        constexpr int IPR = CH > 32 ? CH / 32 : 1;                  // copies of one row
        const int chunk = CH >= 32 ? lane : lane % CH, row_in = CH >= 32 ? 0 : lane / CH;
        const int real_chunks = p.dim * C::ES / 16;
        const uint32_t page_mask = (1u << p.page_shift) - 1u;
        const uint32_t ring_u = smem_u32(ring);
        int slot = is_v ? 1 : 0;
        uint32_t phase = 0;
        while (walk.next(p, units)) {
            const Span& s = walk.s;
            const int32_t* table = p.table + (int64_t)walk.b * p.table_stride;
            const int64_t head = (int64_t)(walk.u / p.row_tiles) * p.head_bytes;
            // the offset of the cache row of key `key`, or -1: a row of zeros
            auto entry_of = [&](int key) { return key >= s.lo && key < s.hi ? table[key >> p.page_shift] : -1; };
            auto offset_of = [&](int key, int entry) -> int64_t {
                const bool seen = key >= s.lo && key < s.hi;
                if (!seen) return -1;
                if ((uint32_t)entry >= (uint64_t)p.pages) {
                    if (p.user_status) atomicOr(p.user_status, 2u);
                    return -1;
                }
                return (int64_t)entry * p.page_bytes + (int64_t)((uint32_t)key & page_mask) * p.token_bytes + head;
            };
            int key0 = s.base + walk.t0 * KEYS;
            int e0 = entry_of(key0 + lane), e1 = entry_of(key0 + 32 + lane);
            for (int t = walk.t0; t < walk.t1; ++t, key0 += KEYS) {
                const int64_t off0 = offset_of(key0 + lane, e0), off1 = offset_of(key0 + 32 + lane, e1);
                if (t + 1 < walk.t1) {
                    e0 = entry_of(key0 + KEYS + lane);
                    e1 = entry_of(key0 + KEYS + 32 + lane);
                }
                wait(empty(slot), phase ^ 1u);
                if (!ok) break;
                const uint32_t dst = ring_u + (uint32_t)slot * C::TILE;
#pragma unroll 8
                for (int i = 0; i < KEYS / RPI; ++i) {
                    const int row = i * RPI + row_in;
                    const int64_t off = __shfl_sync(~0u, i < KEYS / RPI / 2 ? off0 : off1, row & 31);
#pragma unroll
                    for (int c = 0; c < IPR; ++c) {
                        const int ch = chunk + 32 * c;
                        if (ch < real_chunks)
                            cp16(dst + chunk_at<CH>(row, ch), cache + (off < 0 ? 0 : off + ch * 16), off >= 0);
                    }
                }
                cp_arrive(full(slot));
                slot += 2;
                if (slot >= C::NS) slot -= C::NS, phase ^= 1u;
            }
            if (!ok) break;
        }
        if (!ok && lane == 0) atomicOr(p.status, 1u);
        asm volatile("cp.async.wait_all;" ::: "memory");
        return;
    }
    if (wid == W + 2) {
        // ================= q of each segment, rows (token, head of the group), in the matrix type
        int qs = 0;
        uint32_t phase = 0;
        const int rows = p.tokens * p.group;
        while (walk.next(p, units)) {
            wait(qempty(qs), phase ^ 1u);
            if (!ok) break;
            uint8_t* dst = qbuf + qs * C::QBYTES;
            const int hk = walk.u / p.row_tiles, r0 = (walk.u % p.row_tiles) * C::ROWS;
            constexpr int QCH = DP / 8;                             // 16-byte chunks of a row
            constexpr int PER = QCH > 32 ? QCH / 32 : 1;
            for (int r = 0; r < C::ROWS; ++r) {
                const bool in = r0 + r < rows;
                const int j = in ? (r0 + r) / p.group : 0, hq = hk * p.group + (r0 + r - j * p.group);
                const uint16_t* src = p.q + (int64_t)walk.b * p.q_bs + (int64_t)j * p.q_ts + (int64_t)hq * p.q_hs;
                uint4 w[PER];
#pragma unroll
                for (int c = 0; c < PER; ++c) {
                    const int ch = lane + 32 * c;
                    w[c] = (in && ch < QCH && ch * 8 < p.dim) ? *reinterpret_cast<const uint4*>(src + ch * 8)
                                                               : make_uint4(0, 0, 0, 0);
                }
                if constexpr (E4M3) {
                    // a power of two that brings the row's largest magnitude into [2^13, 2^14)
                    uint32_t big = 0;
#pragma unroll
                    for (int c = 0; c < PER; ++c) {
                        const uint32_t v[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) big = max(big, max(v[e] & 0x7fffu, (v[e] >> 16) & 0x7fffu));
                    }
                    big = __reduce_max_sync(~0u, big);
                    int up = 13 - ((int)(big >> 7) - 127);
                    if (big >= 0x7f80u) up = 0;                     // an infinity or NaN stays one
                    up = min(up, 126);
                    const float f = __uint_as_float((uint32_t)(up + 127) << 23);
                    if (lane == 0) qscale[qs * C::ROWS + r] = __uint_as_float((uint32_t)(127 - up) << 23);
#pragma unroll
                    for (int c = 0; c < PER; ++c) {
                        const int ch = lane + 32 * c;
                        uint32_t v[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            v[e] = pack2<true>(__uint_as_float(v[e] << 16) * f, __uint_as_float(v[e] & 0xffff0000u) * f);
                        if (ch < QCH) {
                            // within 16 dims, the order in which an 8-bit K fragment holds them: a thread's
                            // four bytes 4t .. 4t + 3 are k = 2t, 2t + 1, 2t + 8, 2t + 9
                            const int step = ch >> 1, h = ch & 1;   // dims 16 step + 8 h ..
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int pair = 4 * h + e;         // dims 2 pair, 2 pair + 1 of the 16
                                const int k = (pair >> 1) * 2 + (pair & 1) * 8;
                                *reinterpret_cast<uint32_t*>(dst + chunk_at<QCH>(r, 2 * step + (k >> 3)) + (k & 7) * 2) = v[e];
                            }
                        }
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < PER; ++c) {
                        const int ch = lane + 32 * c;
                        if (ch < QCH) *reinterpret_cast<uint4*>(dst + chunk_at<QCH>(r, ch)) = w[c];
                    }
                }
            }
            mbar_arrive(qfull(qs));
            if (++qs == C::QBUF) qs = 0, phase ^= 1u;
        }
        if (!ok && lane == 0) atomicOr(p.status, 1u);
        return;
    }

    // ===================== consumers
    const int g = lane >> 2, t2 = (lane & 3) * 2;
    constexpr int MT = C::MT, QCH = DP / 8;
    int slot = 0, qs = 0;
    uint32_t phase = 0, qphase = 0;
    const uint32_t ring_u = smem_u32(ring), qbuf_u = smem_u32(qbuf), pbuf_u = smem_u32(pbuf);
    uint32_t turn = 0;                       // which half of pbuf
    float acc[MT][NT][4], m[NT][2], l[NT][2];
    const float NINF = __int_as_float(0xff800000);
    auto advance = [&] {
        __syncwarp();
        if (lane == 0) mbar_arrive(empty(slot));
        if (++slot == C::NS) slot = 0, phase ^= 1u;
    };

    while (walk.next(p, units)) {
        const Span s = walk.s;
        const int hk = walk.u / p.row_tiles, r0 = (walk.u % p.row_tiles) * C::ROWS;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            m[nt][0] = m[nt][1] = NINF;
            l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[mt][nt][e] = 0.f;
        }
        wait(qfull(qs), qphase);
        const float sc_all = p.scale_log2 * (p.k_scale ? p.k_scale[hk] : 1.f);
        float sc[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) sc[nt][e] = E4M3 ? sc_all * qscale[qs * C::ROWS + 8 * nt + t2 + e] : sc_all;
        const uint32_t q_u = qbuf_u + qs * C::QBYTES;

        for (int t = walk.t0; t < walk.t1; ++t) {
            const int key0 = s.base + t * KEYS;
            // ---- S^T: this warp's 16 keys x all rows
            float sT[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) sT[nt][e] = 0.f;
            wait(full(slot), phase);
            {
                const uint32_t kt = ring_u + (uint32_t)slot * C::TILE;
                const int krow = 16 * wid + (lane & 15);
#pragma unroll
                for (int s2 = 0; s2 < DP / 32; ++s2) {               // 32 dims
                    uint32_t a0[4], a1[4];
                    if constexpr (E4M3) {
                        uint32_t r[4];
                        ldsm4(kt + chunk_at<C::CH>(krow, 2 * s2 + (lane >> 4)), r);
                        a0[0] = e4m3_f16x2(r[0]), a0[2] = e4m3_f16x2(r[0] >> 16);
                        a0[1] = e4m3_f16x2(r[1]), a0[3] = e4m3_f16x2(r[1] >> 16);
                        a1[0] = e4m3_f16x2(r[2]), a1[2] = e4m3_f16x2(r[2] >> 16);
                        a1[1] = e4m3_f16x2(r[3]), a1[3] = e4m3_f16x2(r[3] >> 16);
                    } else {
                        ldsm4(kt + chunk_at<C::CH>(krow, 4 * s2 + (lane >> 4)), a0);
                        ldsm4(kt + chunk_at<C::CH>(krow, 4 * s2 + 2 + (lane >> 4)), a1);
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        uint32_t b[4];
                        ldsm4(q_u + chunk_at<QCH>(8 * nt + (lane & 7), 4 * s2 + (lane >> 3)), b);
                        mma<E4M3>(sT[nt], a0, b[0], b[1]);
                        mma<E4M3>(sT[nt], a1, b[2], b[3]);
                    }
                }
            }
            advance();   // the K tile has been read

            // ---- scores in log2 units; what a row may not see is -inf
            // every key of the tile visible to every row?
            const bool whole = key0 + KEYS <= s.len - p.tokens + 1 && (p.window <= 0 || key0 >= s.len - p.window);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) sT[nt][e] *= sc[nt][e & 1];
            if (!whole) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int key = key0 + 16 * wid + g + (e >> 1) * 8;
                        const int end = s.len - p.tokens + (r0 + 8 * nt + t2 + (e & 1)) / p.group + 1;
                        if (key >= end || key >= s.hi || (p.window > 0 && key < end - p.window)) sT[nt][e] = NINF;
                    }
            }
            bool need = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) need |= sT[nt][e] > m[nt][e & 1] + LAZY;

            // ---- P^T = 2^(s - m), to [nt][key][row]
            uint32_t p_u = pbuf_u + turn * C::PBYTES;
            float pT[NT][4];
            auto make_p = [&] {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float mm = m[nt][e & 1] == NINF ? 0.f : m[nt][e & 1];
                        pT[nt][e] = exp2_approx(sT[nt][e] - mm);
                    }
                    const uint32_t at = p_u + nt * KEYS * 16 + (16 * wid + g) * 16 + t2 * 2;
#pragma unroll
                    for (int e = 0; e < 4; e += 2) {
                        const uint32_t hi = pack2<E4M3>(pT[nt][e], pT[nt][e + 1]);
                        st_shared(at + e * 64, hi);
                        if constexpr (!E4M3)
                            st_shared(at + e * 64 + C::LOW, pack2<false>(pT[nt][e] - __uint_as_float(hi << 16),
                                                                         pT[nt][e + 1] - __uint_as_float(hi & 0xffff0000u)));
                    }
                }
            };
            make_p();
            if (consumer_any(need)) {
                // a new maximum for every row: the four warps' maxima meet in shared memory
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float x = fmaxf(sT[nt][e], sT[nt][e + 2]);
                        x = fmaxf(x, __shfl_xor_sync(~0u, x, 4));
                        x = fmaxf(x, __shfl_xor_sync(~0u, x, 8));
                        x = fmaxf(x, __shfl_xor_sync(~0u, x, 16));
                        if (g == 0) red[wid * C::ROWS + 8 * nt + t2 + e] = x;
                    }
                consumer_sync();
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float x = m[nt][e];
#pragma unroll
                        for (int w = 0; w < W; ++w) x = fmaxf(x, red[w * C::ROWS + 8 * nt + t2 + e]);
                        const float f = m[nt][e] == x ? 1.f : exp2_approx(m[nt][e] - x);
                        m[nt][e] = x;
                        l[nt][e] *= f;
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt) acc[mt][nt][e] *= f, acc[mt][nt][e + 2] *= f;
                    }
                make_p();
                consumer_sync();
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) l[nt][e & 1] += pT[nt][e];

            // ---- O^T += V^T P^T: this warp's dims, all 64 keys
            wait(full(slot), phase);
            {
                const uint32_t vt = ring_u + (uint32_t)slot * C::TILE;
                // V^T fragments of 16-dim tile mt: keys 32 kp .. 32 kp + 31, two k-steps
                auto v_frags = [&](int kp, int mt, uint32_t (&f)[2][4]) {
                    if constexpr (E4M3) {
                        uint32_t r[4];
                        ldsm4t(vt + chunk_at<C::CH>(32 * kp + lane, wid * MT + mt), r);
#pragma unroll
                        for (int h = 0; h < 4; ++h) {
                            const uint32_t x = __byte_perm(r[h], 0, 0x3120);   // (key, key + 1) of dim 2g, then of 2g + 1
                            f[h >> 1][(h & 1) * 2] = e4m3_f16x2(x);
                            f[h >> 1][(h & 1) * 2 + 1] = e4m3_f16x2(x >> 16);
                        }
                    } else {
                        const int key = 32 * kp + (lane & 7) + ((lane >> 4) << 3);
                        const int c = 2 * (wid * MT + mt) + ((lane >> 3) & 1);
                        ldsm4t(vt + chunk_at<C::CH>(key, c), f[0]);
                        ldsm4t(vt + chunk_at<C::CH>(key + 16, c), f[1]);
                    }
                };
                auto p_frags = [&](int kp, uint32_t (&b)[C::PN][NT][4]) {
#pragma unroll
                    for (int n = 0; n < C::PN; ++n)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            ldsm4t(p_u + n * C::LOW + nt * KEYS * 16 + (32 * kp + lane) * 16, b[n][nt]);
                };
                // Keys that some rows see and others do not meet P = 0 in the others' columns, where an
                // infinity or NaN of V must not become one of the output: such a tile is added row by row.
                bool apart = false;
                if (!whole && p.tokens > 1) {
                    constexpr uint32_t EXP = E4M3 ? 0x7c00u : 0x7f80u;
#pragma unroll 1
                    for (int kp = 0; kp < 2; ++kp)
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt) {
                            uint32_t f[2][4];
                            v_frags(kp, mt, f);
#pragma unroll
                            for (int h = 0; h < 8; ++h) {
                                const uint32_t x = f[h >> 2][h & 3];
                                apart |= (x & EXP) == EXP || ((x >> 16) & EXP) == EXP;
                            }
                        }
                    apart = __any_sync(~0u, apart);
                }
                if (!apart) {
#pragma unroll
                    for (int kp = 0; kp < 2; ++kp) {
                        uint32_t b[C::PN][NT][4];
                        p_frags(kp, b);
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt) {
                            uint32_t f[2][4];
                            v_frags(kp, mt, f);
#pragma unroll
                            for (int n = 0; n < C::PN; ++n)
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt) {
                                    mma<E4M3>(acc[mt][nt], f[0], b[n][nt][0], b[n][nt][1]);
                                    mma<E4M3>(acc[mt][nt], f[1], b[n][nt][2], b[n][nt][3]);
                                }
                        }
                    }
                } else {
#pragma unroll 1
                    for (int j = 0; j < p.tokens; ++j) {
                        const int end = s.len - p.tokens + j + 1, begin = p.window > 0 ? end - p.window : 0;
#pragma unroll 1
                        for (int kp = 0; kp < 2; ++kp) {
                            uint32_t b[C::PN][NT][4];
                            p_frags(kp, b);
#pragma unroll
                            for (int mt = 0; mt < MT; ++mt) {
                                uint32_t f[2][4];
                                v_frags(kp, mt, f);
#pragma unroll
                                for (int h = 0; h < 8; ++h) {       // keys 2t, 2t + 1 (+ 8 for registers 2 and 3)
                                    const int key = key0 + 32 * kp + 16 * (h >> 2) + t2 + ((h & 2) ? 8 : 0);
                                    if (key < begin || key >= end) f[h >> 2][h & 3] &= 0xffff0000u;
                                    if (key + 1 < begin || key + 1 >= end) f[h >> 2][h & 3] &= 0x0000ffffu;
                                }
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt) {
                                    float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                                    for (int n = 0; n < C::PN; ++n) {
                                        mma<E4M3>(d, f[0], b[n][nt][0], b[n][nt][1]);
                                        mma<E4M3>(d, f[1], b[n][nt][2], b[n][nt][3]);
                                    }
#pragma unroll
                                    for (int e = 0; e < 4; ++e)
                                        if ((r0 + 8 * nt + t2 + (e & 1)) / p.group == j) acc[mt][nt][e] += d[e];
                                }
                            }
                        }
                    }
                }
            }
            advance();   // the V tile has been read
            turn ^= 1u;
        }

        // ---- the end of a segment
        __syncwarp();
        if (lane == 0) mbar_arrive(qempty(qs));
        if (++qs == C::QBUF) qs = 0, qphase ^= 1u;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float x = l[nt][e];
                x += __shfl_xor_sync(~0u, x, 4);
                x += __shfl_xor_sync(~0u, x, 8);
                x += __shfl_xor_sync(~0u, x, 16);
                if (g == 0) lred[wid * C::ROWS + 8 * nt + t2 + e] = x;
            }
        consumer_sync();
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float x = 0.f;
#pragma unroll
                for (int w = 0; w < W; ++w) x += lred[w * C::ROWS + 8 * nt + t2 + e];
                l[nt][e] = x;
            }

        bool write = true;
        if (walk.t0 > 0 || walk.t1 < s.tiles) {
            // a part of the unit: publish it, and join the parts if every other run has published
            const int64_t c_first = ((walk.unit0 + 1) * ctas - 1) / all_tiles;
            const int64_t c_last = ((walk.unit0 + s.tiles) * ctas - 1) / all_tiles;
            const int mine = 2 * blockIdx.x + (walk.t0 > 0 ? 0 : 1);
            float4* part = reinterpret_cast<float4*>(p.slots + (size_t)mine * C::SLOT_FLOATS);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    part[((wid * MT + mt) * NT + nt) * 32 + lane] =
                        make_float4(acc[mt][nt][0], acc[mt][nt][1], acc[mt][nt][2], acc[mt][nt][3]);
            float* stats = reinterpret_cast<float*>(part) + (size_t)W * MT * NT * 128;   // [row]{m, l}
            if (wid == 0 && g == 0)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    *reinterpret_cast<float4*>(stats + 2 * (8 * nt + t2)) = make_float4(m[nt][0], l[nt][0], m[nt][1], l[nt][1]);
            __threadfence();
            consumer_sync();
            if (tid == 0) {
                const uint32_t parts = (uint32_t)(c_last - c_first + 1);
                uint32_t* counter = p.counters + c_first;
                const uint32_t before = atomicAdd(counter, 1u);
                const bool last = before == parts - 1;
                if (last) *counter = 0;   // every run has counted in: zero again for the next call
                __threadfence();
                last_flag = last;
            }
            consumer_sync();
            write = last_flag != 0;
            if (write) {
                __threadfence();
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    m[nt][0] = m[nt][1] = NINF;
                    l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[mt][nt][e] = 0.f;
                }
                auto slot_of = [&](int64_t c) { return p.slots + (size_t)(2 * c + (c == c_first ? 1 : 0)) * C::SLOT_FLOATS; };
                for (int64_t c = c_first; c <= c_last; ++c) {
                    const float* st = slot_of(c) + (size_t)W * MT * NT * 128;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const float4 v = __ldcg(reinterpret_cast<const float4*>(st + 2 * (8 * nt + t2)));
                        m[nt][0] = fmaxf(m[nt][0], v.x);
                        m[nt][1] = fmaxf(m[nt][1], v.z);
                    }
                }
#pragma unroll 2
                for (int64_t c = c_first; c <= c_last; ++c) {
                    const float* base = slot_of(c);
                    const float* st = base + (size_t)W * MT * NT * 128;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const float4 v = __ldcg(reinterpret_cast<const float4*>(st + 2 * (8 * nt + t2)));
                        const float f0 = v.x == m[nt][0] ? 1.f : exp2_approx(v.x - m[nt][0]);
                        const float f1 = v.z == m[nt][1] ? 1.f : exp2_approx(v.z - m[nt][1]);
                        l[nt][0] += f0 * v.y;
                        l[nt][1] += f1 * v.w;
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt) {
                            const float4 a = __ldcg(reinterpret_cast<const float4*>(base) + ((wid * MT + mt) * NT + nt) * 32 + lane);
                            acc[mt][nt][0] += f0 * a.x;
                            acc[mt][nt][1] += f1 * a.y;
                            acc[mt][nt][2] += f0 * a.z;
                            acc[mt][nt][3] += f1 * a.w;
                        }
                    }
                }
            }
        }
        if (write && ok) {
            const float vs = p.v_scale ? p.v_scale[hk] : 1.f;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = r0 + 8 * nt + t2 + e;
                    const int j = r / p.group, hq = hk * p.group + (r - j * p.group);
                    if (j >= p.tokens) continue;
                    // a row that sees no key is zero; otherwise its sum is positive, or NaN as its scores are
                    const int end = s.len - p.tokens + j + 1;
                    const bool none = end <= 0;
                    const float inv = none ? 0.f : vs / l[nt][e];
                    uint16_t* o = p.out + (int64_t)walk.b * p.o_bs + (int64_t)j * p.o_ts + (int64_t)hq * p.o_hs;
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        const int d = (wid * MT + mt) * 16 + (E4M3 ? 2 * g : g);
                        const __nv_bfloat16 x = __float2bfloat16_rn(none ? 0.f : acc[mt][nt][e] * inv);
                        const __nv_bfloat16 y = __float2bfloat16_rn(none ? 0.f : acc[mt][nt][e + 2] * inv);
                        if (d < p.dim) {
                            if constexpr (E4M3) {
                                *reinterpret_cast<__nv_bfloat162*>(o + d) = __nv_bfloat162(x, y);
                            } else {
                                *reinterpret_cast<__nv_bfloat16*>(o + d) = x;
                                *reinterpret_cast<__nv_bfloat16*>(o + d + 8) = y;
                            }
                        }
                    }
                    if (p.lse && wid == 0 && g == 0)
                        p.lse[((int64_t)walk.b * p.tokens + j) * p.heads_q + hq] =
                            none ? NINF : (m[nt][e] == NINF ? 0.f : m[nt][e] * 0.69314718055994531f) + logf(l[nt][e]);
                }
        }
    }
    if (!ok && lane == 0) atomicOr(p.status, 1u);
}

template <int DP, int NT, bool E4M3>
cudaError_t allow() {
    return cudaFuncSetAttribute(paged_attn_kernel<DP, NT, E4M3>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)Cfg<DP, NT, E4M3>::SMEM);
}
template <int DP, int NT, bool E4M3>
AttnShape shape() {
    using C = Cfg<DP, NT, E4M3>;
    AttnShape s;
    s.ctas_per_sm = C::CPS;
    s.rows = C::ROWS;
    s.slot_floats = C::SLOT_FLOATS;
    return s;
}
template <int DP, int NT, bool E4M3>
cudaError_t launch(const AttnParams& p, int grid, cudaStream_t st) {
    return launch_pdl(paged_attn_kernel<DP, NT, E4M3>, dim3((unsigned)grid), THREADS, Cfg<DP, NT, E4M3>::SMEM, st, p);
}

// Row tiles hold 8 NT rows, the fewest that take all rows at once, up to 64
// (16 at dim 512, whose tiles fill shared memory); more rows go to several
// tiles, each of which reads the keys again.
#define AFFQMM_ATTN_SWITCH(DP, rows, CALL)                   \
    if ((rows) <= 8) { CALL(DP, 1); }                        \
    if ((rows) <= 16 || (DP) == 512) { CALL(DP, 2); }        \
    if constexpr ((DP) < 512) {                              \
        if ((rows) <= 32) { CALL(DP, 4); }                   \
        CALL(DP, 8);                                         \
    }
#define AFFQMM_ATTN_SHAPE(DP, NT) return e4m3 ? attn::shape<DP, NT, true>() : attn::shape<DP, NT, false>()
#define AFFQMM_ATTN_LAUNCH(DP, NT) \
    return e4m3 ? attn::launch<DP, NT, true>(p, grid, st) : attn::launch<DP, NT, false>(p, grid, st)
#define AFFQMM_ATTN_ALLOW(DP, NT)                                           \
    if (cudaError_t e = attn::allow<DP, NT, true>(); e != cudaSuccess) return e; \
    if (cudaError_t e = attn::allow<DP, NT, false>(); e != cudaSuccess) return e

}  // namespace attn
}  // namespace affqmm

#define AFFQMM_ATTN_DEFINE(DP)                                                                            \
    namespace affqmm {                                                                                    \
    AttnShape attn_shape_##DP(bool e4m3, int rows) {                                                      \
        AFFQMM_ATTN_SWITCH(DP, rows, AFFQMM_ATTN_SHAPE)                                                   \
        return {};                                                                                        \
    }                                                                                                     \
    cudaError_t attn_allow_smem_##DP() {                                                                  \
        AFFQMM_ATTN_ALLOW(DP, 1);                                                                         \
        AFFQMM_ATTN_ALLOW(DP, 2);                                                                         \
        if constexpr ((DP) < 512) {                                                                       \
            AFFQMM_ATTN_ALLOW(DP < 512 ? DP : 64, 4);                                                     \
            AFFQMM_ATTN_ALLOW(DP < 512 ? DP : 64, 8);                                                     \
        }                                                                                                 \
        return cudaSuccess;                                                                               \
    }                                                                                                     \
    cudaError_t launch_attn_##DP(bool e4m3, int rows, const AttnParams& p, int grid, cudaStream_t st) {    \
        AFFQMM_ATTN_SWITCH(DP, rows, AFFQMM_ATTN_LAUNCH)                                                  \
        return cudaErrorInvalidValue;                                                                     \
    }                                                                                                     \
    }
