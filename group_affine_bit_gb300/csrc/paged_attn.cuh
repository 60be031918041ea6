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
// Roles.  A CTA has four consumer warps (or two groups of four, below), two
// producer warps, one for q and, where blocks have scales, one for those.  A
// tile is 64 or 128 keys.  The producers (one for K, one for V) gather it through the block table with TMA, a box to a
// page's rows of the tile, in 128-byte panels whose swizzle keeps the fragment
// loads free of bank conflicts; K and V tiles take turns in one ring.  Rows of
// pages that no query may see are not read, an entry that is no page reads as
// zeros, and what lies in a tile beyond the visible keys is zeroed by the
// consumers.  The producers run ahead across the borders of requests, so the
// memory pipeline does not drain there.  (Gathering with 16-byte cp.async
// copies cost a producer warp 54-97 cycles for each 512 bytes: 559 MB at dim
// 256 in 117 us instead of 90, 659 MB of e4m3 in 165 us instead of 108-129.)
//
// Arithmetic.  Keys are the M side of the matrix instruction (m16n8k16) and
// query rows its N side, so that one to eight rows cost one instruction per 16
// keys x 16 dims: S^T = K Q^T, a warp to 16 (or 2 x 16) keys; then O^T = V^T
// P^T, a warp to a quarter of the dims, P^T through shared memory.  The running
// maximum is shared by the group and lazy: a tile is rescaled only if a score
// exceeds it by more than 2^8 (8-bit caches: 2^2; an OR over the barrier that P^T needs
// anyway), so most tiles cost one barrier and no shuffles.  Scores, maxima, sums and
// outputs are fp32.  P meets V in the matrix type.  Beside a bf16 cache it is
// the sum of two bf16 numbers, what the first leaves being in the second, each
// with its own matrix instruction: 16 bits of P instead of 8, so that the
// output's own rounding is what is left of the error (2-norm against 64 bits
// 0.0017; with one bf16 number 0.0023), for instructions that a memory-bound
// kernel has to spare.  The first is cut off, not rounded, and the second is
// never zero beside it: an infinite value meets two positive numbers, and stays
// infinite.  Beside an e4m3 one it is one f16, 2^13 times P: f16 has
// 11 bits from 2^-14 on and reaches 2^16, so that P keeps them down to 2^-27 of
// the running maximum, and below that is off by 2^-38 at most (a tail 18 nats
// below a key whose value is zero is the whole output; with P itself in f16 it
// came out as zero).  f16 holds the cache's values exactly, and q is brought to
// f16 with a power of two per row, so that it keeps its eight bits.  The sum of P is taken before these
// roundings.  The warp-level matrix instruction, not tcgen05: with few rows the
// pipe is far from busy, and from 32 rows on it is what bounds the kernel (64
// rows at dim 128: 192 instructions of 16 cycles a tile, 168 us of the measured
// 170).
//
// Scales of blocks.  Beside codes with a scale for each block of tokens and head
// (e4m3 or int8), K's scale multiplies a key's score, and V's enters the exponent:
//     z = log2(e) s + log2 vs,   P = 2^(z - m + lift) in f16,   l = sum P / vs
// with m the running maximum of z, so that what meets V's codes in f16 is again at
// most 2^15 whatever the scales are.  A scale is between 2^-48 and 2^48, which
// keeps P / vs within fp32.  A warp of its own brings the scales: it loads the
// next tile's (8 bytes a block, gathered through the table) while this one's wait
// for their place beside the ring, and leaves K's scale and log2 of V's, so that a
// consumer spends two multiply-adds a score and a shared load and an exponential a
// key.  (64 requests of up to 32768 keys, dim 128, int8: with the loads in K's
// producer 378 us in blocks of 32 and 839 with a scale for every token; with a
// warp of its own 310 and 367; e4m3 with a scale for each head 305.)  Four int8
// codes become f16 by two byte permutations and two packed subtractions.
// 16 rows of dim 256 fit two CTAs an SM in registers (12 requests x 5 tokens,
// window 1024: 40 -> 33 us against two groups that convert the same keys).
//
// Groups.  Where one CTA fills an SM and the rows fill two row tiles or more,
// they go to two groups of four consumer warps that share the ring and q: two
// warps to a scheduler, whose latencies overlap (64 rows at dim 128: 226 -> 204
// us).  In long tables of short rows the two groups take two neighbouring key
// heads instead (paged_api.cu says where).
//
// Split.  All tiles of all (request, key head, row tile) units, in order, are
// cut into equal runs, one per CTA, so a batch of ragged lengths loads every
// SM alike; each CTA finds its run by a prefix sum over the lengths.  The runs
// that share a unit leave their parts in slots of the workspace and count in;
// one of them joins the parts, always in run order, so that the same inputs
// give the same bits.  A part that a run begins with is counted in by the q
// warp while the consumers go on; a run that ends with a unit's first part
// keeps it in registers if the others are in by then, as they mostly are;
// else the last to count in joins.
//
// Failure.  Every wait on a barrier is bounded; one that gives up is reported in
// the workspace's status word.  A consumer warp that gave up goes on through the
// barriers it shares, with whatever shared memory holds, and frees no slot of
// the ring, so that the producers give up too and wait for their copies; what
// it had a part in is neither counted in nor written.
//
// Measured (GB300, device time): 64 requests of up to 32768 keys, dim 128, 4.47
// GB: 657 us, the measured copy rate; one request of 262143 keys 165 us, 96 % of
// it; 32 requests of up to 4096 keys, dim 256, 559 MB: 93 us, 89 %; e4m3, 659
// MB: 109 us, 89 %; one request of 577 keys 8.7 us, of which 0.7 is the launch, 3
// lead to the first tile and 4 are the join of its parts.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "affqmm_async.cuh"
#include "affqmm_internal.h"
#include "affqmm_paged.h"
#include "affqmm_tc.cuh"

namespace affqmm {
namespace attn {

constexpr int W = 4;                       // consumer warps
constexpr int GROUP = 32 * W;             // threads of a group of consumers
// Kinds of cache: bf16; e4m3 with a scale for each key head; e4m3 and int8 with a scale for each block of tokens and key head.
enum Kind { KV_BF16, KV_E4M3, KV_E4M3_BLOCKS, KV_I8_BLOCKS };
constexpr float lazy(bool bytes) { return bytes ? 2.f : 8.f; }   // log2 of how far a score may exceed the running maximum
constexpr float lift(bool bytes) { return bytes ? 13.f : 0.f; }  // log2 of what P is multiplied by: with lazy() below f16's 16
constexpr size_t SM_SMEM = 233472;         // shared memory of an SM, 1 KB of it taken by each CTA
constexpr size_t CTA_SMEM = 232448;        // and what one CTA may have of it
constexpr size_t STATIC_SMEM = 1024;       // the kernel's few static variables, and the ring's alignment
constexpr int MAX_SLOTS = 16;

// Blocks of 16 keys to a consumer warp: with two, two chains of matrix instructions overlap and the barrier comes
// half as often, but a tile has 128 keys and the cut is coarser.  Two for rows of 128 bytes or less, and for rows of
// 256 bytes with four row tiles or more (204.8 -> 170.2 us for 64 rows of dim 128), or where the tables have room for
// `lasting` tiles (dim 128: 678 -> 657 us for 64 requests of up to 32768 keys; 7.6 -> 8.2 for one of 577).
constexpr int key_blocks(int pitch, int na, bool lasting) { return pitch <= 128 || (pitch == 256 && (na >= 4 || lasting)) ? 2 : 1; }

template <int DP, int NA, int KIND, int KBLOCKS, bool PAIRED>
struct Cfg {
    static constexpr bool BYTES = KIND != KV_BF16, BLOCKS = KIND >= KV_E4M3_BLOCKS, I8 = KIND == KV_I8_BLOCKS;
    // PAIR: the two groups of consumer warps take two neighbouring key heads, whose rows lie side by side in the
    // pool, and a tile holds the keys of both.
    static constexpr bool PAIR = PAIRED;
    static constexpr int HEADS = PAIR ? 2 : 1;
    static constexpr int ES = BYTES ? 1 : 2;
    static constexpr int ROWS = 8 * NA;
    static constexpr int PITCH = DP * ES;              // bytes of a cache row in shared memory
    static constexpr int PW = PITCH < 128 ? PITCH : 128;   // bytes of a row in one panel
    static constexpr int PANELS = PITCH / PW;
    static constexpr int KB = KBLOCKS;
    static constexpr int KEYS = 16 * W * KB;
    static constexpr int HEAD_TILE = KEYS * PITCH, TILE = HEADS * HEAD_TILE;
    static constexpr int SCALES = BLOCKS ? 2 * HEADS * KEYS : 0;   // floats of a tile's scales: [head][block, at most KEYS]{K, V}
    static constexpr int QBYTES = ROWS * DP * 2;
    static constexpr int QBUF = (DP == 512 && NA > 1) ? 1 : 2;
    static constexpr int PN = BYTES ? 1 : 2;           // numbers that make one P
    static constexpr int MT = DP / (16 * W);           // 16-dim tiles of a consumer warp
    static constexpr int JOIN = 32;                    // most parts that a join takes at once
    static constexpr int BARRIER_BYTES = BLOCKS ? 448 : 512;      // more than the barriers (below) take
    static constexpr size_t FIXED = (size_t)QBUF * QBYTES + 2 * PN * NA * KEYS * 16 + 2 * W * ROWS * 4 + 5 * QBUF * ROWS * 4 +
                                    JOIN * ROWS * 4 + BARRIER_BYTES;
    // Registers allow two CTAs an SM.  Two row tiles of dim 256 beside scales of blocks fit but for 4 to 8 bytes (12 x 5 tokens,
    // window 1024: 40 -> 33 us); four of dim 64, as many accumulators but more scores, spill (12 requests of 1000 keys 12.7 -> 15.6).
    static constexpr bool LIGHT = MT * NA * 4 + NA * 8 <= (BLOCKS && DP == 256 ? 48 : 32);
    static constexpr size_t HALF = SM_SMEM / 2 - 1024 - STATIC_SMEM;
    static constexpr int CPS = (!PAIR && LIGHT && FIXED + 3 * TILE + 2 * SCALES * 4 <= HALF) ? 2 : 1;
    // With one CTA an SM, the rows go to two groups of consumer warps (where there are two row tiles), which share
    // the ring and q and nothing else: two warps to a scheduler, whose latencies overlap.
    static constexpr int NG = CPS == 1 && NA >= 2 ? 2 : 1;
    static constexpr int NT = NA / NG, GROWS = 8 * NT;           // row tiles, rows of a group
    static constexpr int CONSUMERS = 32 * W * NG, THREADS = CONSUMERS + (BLOCKS ? 128 : 96);
    static constexpr int LOW = NT * KEYS * 16;         // from P's first numbers to the second
    static constexpr int PBYTES = PN * LOW;            // of a group: [PN][NT][keys][8 rows] of 16 bits
    static constexpr size_t ROOM = (CPS == 2 ? HALF : CTA_SMEM - STATIC_SMEM) - FIXED;
    static constexpr int sets(int slots) { return (slots + 1) / 2; }   // of scales: one for each K tile that the ring can hold
    static constexpr int slots_in(size_t room) {
        int n = room / TILE > MAX_SLOTS ? MAX_SLOTS : (int)(room / TILE);
        while (n > 0 && (size_t)n * TILE + (size_t)sets(n) * SCALES * 4 > room) --n;
        return n;
    }
    static constexpr int NS = slots_in(ROOM), NSC = sets(NS);
    static constexpr size_t SMEM = FIXED + (size_t)NS * TILE + (size_t)NSC * SCALES * 4;
    static constexpr size_t STATS = (size_t)W * MT * NT * 128;  // of a group's part: the accumulators, then [row]{m, l}
    static constexpr size_t PART_FLOATS = STATS + 2 * GROWS;
    static constexpr size_t SLOT_FLOATS = NG * PART_FLOATS;
    static_assert(NS >= 3, "ring too short");
    // The barriers, in units of one: full[], empty[], qfull[2], stored[2], counted, finished, decided, joined[2], drained, never,
    // scaled[].
    static constexpr int B_EMPTY = MAX_SLOTS, B_QFULL = B_EMPTY + MAX_SLOTS, B_STORED = B_QFULL + 2, B_COUNTED = B_STORED + 2,
                         B_FINISHED = B_COUNTED + 1, B_DECIDED = B_FINISHED + 1, B_JOINED = B_DECIDED + 1, B_DRAINED = B_JOINED + 2,
                         B_NEVER = B_DRAINED + 1, B_SCALED = B_NEVER + 1, BARRIERS = B_SCALED + (BLOCKS ? NSC : 0);
    static_assert(QBUF <= 2 && NG <= 2 && 8 * BARRIERS <= BARRIER_BYTES, "more barriers than there is room for");
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
// Four codes in a word to f16, exact: the first two and the last two, or (ACROSS) the even and the odd ones.
// A signed byte b is the low byte of the f16 1024 + (b + 128).
template <bool I8, bool ACROSS>
__device__ __forceinline__ void bytes_f16(uint32_t w, uint32_t& a, uint32_t& b) {
    if constexpr (I8) {
        w ^= 0x80808080u;
        const __half2 zero = __half2half2(__ushort_as_half(0x6480));   // 1024 + 128
        const uint32_t x = __byte_perm(w, 0x64646464u, ACROSS ? 0x4240 : 0x4140), y = __byte_perm(w, 0x64646464u, ACROSS ? 0x4341 : 0x4342);
        const __half2 u = __hsub2(*reinterpret_cast<const __half2*>(&x), zero), v = __hsub2(*reinterpret_cast<const __half2*>(&y), zero);
        a = *reinterpret_cast<const uint32_t*>(&u), b = *reinterpret_cast<const uint32_t*>(&v);
    } else {
        if (ACROSS) w = __byte_perm(w, 0, 0x3120);
        a = e4m3_f16x2(w), b = e4m3_f16x2(w >> 16);
    }
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
// Count a part in: what this CTA stored before is visible to who sees the count, and what others stored to us.
__device__ __forceinline__ uint32_t count_part(uint32_t* counter) {
    uint32_t before;
    asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(before) : "l"(counter) : "memory");
    return before;
}
// n / d by m = ceil(2^32 / d), exact for n < 2^32 / d (n up to 4096 heads x 64 tokens, d up to 4096)
__device__ __forceinline__ int over(int n, int d, uint32_t m) { return d == 1 ? n : (int)__umulhi((uint32_t)n, m); }
// Whether one of the values in a word (two bf16, or four codes) is an infinity or NaN.
template <int KIND>
__device__ __forceinline__ bool not_finite(uint32_t w) {
    if constexpr (KIND == KV_I8_BLOCKS) {
        return false;
    } else if constexpr (KIND != KV_BF16) {
        bool any = false;
#pragma unroll
        for (int i = 0; i < 4; ++i) any |= ((w >> (8 * i)) & 0x7fu) == 0x7fu;
        return any;
    } else {
        return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
    }
}
__device__ __forceinline__ void st_shared(uint32_t addr, uint32_t v) {
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, int c3,
                                            uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
            dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void group_sync(int group) { asm volatile("barrier.cta.sync %0, 128;" ::"r"(1 + group) : "memory"); }
__device__ __forceinline__ bool group_any(int group, bool v) {
    uint32_t r;
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred q, %2, 128, p;\n selp.u32 %0, 1, 0, q;\n}\n"
        : "=r"(r) : "r"((uint32_t)v), "r"(1 + group) : "memory");
    return r != 0;
}
// Whether `v` holds in every consumer thread: what branches around a barrier is decided by all of them alike.
template <int THREADS>
__device__ __forceinline__ bool consumers_all(bool v) {
    uint32_t r;
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.and.pred q, 3, %2, p;\n selp.u32 %0, 1, 0, q;\n}\n"
        : "=r"(r) : "r"((uint32_t)v), "n"(THREADS) : "memory");
    return r != 0;
}
template <int THREADS>
__device__ __forceinline__ void consumers_sync() { asm volatile("barrier.cta.sync 3, %0;" ::"n"(THREADS) : "memory"); }
// Wait for the phase of parity `parity` of `bar` to complete; false if it has not within `limit` cycles.
__device__ __forceinline__ bool mbar_wait_within(uint32_t bar, uint32_t parity, long long limit) {
    if (mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    while (!mbar_try_wait(bar, parity))
        if (clock64() - t0 > limit) return false;
    return true;
}
// A block's scale as it counts: between the bounds that the append keeps to (NaN: the lower).
__device__ __forceinline__ float within_scales(float x) { return fminf(fmaxf(x, kLeastScale), kMostScale); }
// 16-byte chunk `c` of row `row` of a tile: panels of PW bytes of every row,
// swizzled as TMA swizzles rows of 128 (64) bytes, so that the eight rows that
// one fragment load reads fall into eight bank groups.
template <int PW, int KEYS>
__device__ __forceinline__ uint32_t chunk_at(int row, int c) {
    if constexpr (PW == 128) return (uint32_t)((c >> 3) * KEYS * 128 + row * 128 + ((c & 7) ^ (row & 7)) * 16);
    else return (uint32_t)(row * 64 + (c ^ ((row >> 1) & 3)) * 16);
}
// The same of q, whose rows are whole (CH chunks).
template <int CH>
__device__ __forceinline__ uint32_t qchunk_at(int row, int c) {
    return (uint32_t)(row * CH + (c ^ (row & 7))) * 16u;
}

// What a request's tiles cover: keys lo .. hi - 1, tiles counted from `base`.
struct Span {
    int len, lo, hi, base, tiles;
};
template <int KEYS>
__device__ __forceinline__ Span span_of(const AttnParams& p, int b) {
    Span s;
    const int64_t most = (int64_t)p.wide << p.page_shift;
    int len = p.lens[b];
    if (len > most) len = (int)most;
    s.len = max(len, 0);
    s.hi = s.len;
    s.lo = p.window > 0 ? max(0, s.len - p.tokens + 1 - p.window) : 0;
    s.base = s.lo & ~(KEYS - 1);
    s.tiles = max(1, (s.hi - s.base + KEYS - 1) / KEYS);
    return s;
}

// The CTA's run, segment by segment: unit (request b, u = key head * row tiles + row tile), tiles t0 .. t1 - 1.
// A unit's end takes the time of about a tile (3400 cycles against 3000 for a tile of e4m3, dim 128), so in the
// numbering that the runs are cut by, each unit has one tile more than there is to read: a run of many short
// requests gets fewer of them.
template <int KEYS>
struct Walk {
    int b, u, t, t0, t1;
    int left;          // tiles of the run not yet handed out
    uint32_t unit0;    // number of the unit's first tile
    Span s;
    __device__ __forceinline__ bool next(const AttnParams& p, int units) {
        while (left > 0) {
            if (t > s.tiles) {
                unit0 += s.tiles + 1;
                t = 0;
                if (++u == units) {
                    u = 0;
                    ++b;
                    s = span_of<KEYS>(p, b);
                }
            }
            const int from = t, n = min(s.tiles + 1 - t, left);
            left -= n;
            t += n;
            if (from < s.tiles) {
                t0 = from;
                t1 = min(t, s.tiles);
                return true;
            }
        }
        return false;
    }
};

// The CTA whose run has tile x, runs being tiles floor(c total / ctas) .. floor((c + 1) total / ctas) - 1 of CTA c.
__device__ __forceinline__ uint32_t run_of(uint32_t x, uint32_t total, uint32_t ctas) {
    const uint64_t top = (uint64_t)(x + 1) * ctas - 1;
    if (top < (uint64_t)1 << 32) return (uint32_t)top / total;
    return (uint32_t)(top / total);
}

template <int DP, int NA, int KIND, int KBLOCKS, bool PAIRED>
__global__ void __launch_bounds__(Cfg<DP, NA, KIND, KBLOCKS, PAIRED>::THREADS, Cfg<DP, NA, KIND, KBLOCKS, PAIRED>::CPS) paged_attn_kernel(
    const __grid_constant__ AttnParams p, const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map) {
    using C = Cfg<DP, NA, KIND, KBLOCKS, PAIRED>;
    constexpr bool BYTES = C::BYTES, BLOCKS = C::BLOCKS;
    constexpr int KEYS = C::KEYS, THREADS = C::THREADS, PRODUCER = C::NG * W;   // the first warp that is no consumer
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t* ring = smem;
    float* scales = reinterpret_cast<float*>(ring + (size_t)C::NS * C::TILE);   // [NSC][head][KEYS]{K, V}
    uint8_t* qbuf = reinterpret_cast<uint8_t*>(scales + (size_t)C::NSC * C::SCALES);
    uint8_t* pbuf = qbuf + C::QBUF * C::QBYTES;
    float* red = reinterpret_cast<float*>(pbuf + 2 * C::NG * C::PBYTES);      // of each group: [W][rows] maxima
    float* lred = red + W * C::ROWS;                                  // of each group: [W][rows] sums
    float* qscale = lred + W * C::ROWS;                               // [QBUF][ROWS] of 8-bit caches: scale of the row's scores
    int* row_token = reinterpret_cast<int*>(qscale + C::QBUF * C::ROWS);   // [QBUF][ROWS] token of a row, -1: none
    int* row_head = row_token + C::QBUF * C::ROWS;                    // [QBUF][ROWS] and its query head
    float* stats = reinterpret_cast<float*>(row_head + C::QBUF * C::ROWS);   // [QBUF][ROWS]{m, l} of staged rows
    float* weight = stats + 2 * C::QBUF * C::ROWS;                       // of each group: [JOIN][rows] of a join's parts
    uint64_t* bars = reinterpret_cast<uint64_t*>(weight + C::JOIN * C::ROWS);
    const uint32_t bar0 = smem_u32(bars);
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto empty = [&](int s) { return bar0 + 8u * (C::B_EMPTY + s); };
    auto qfull = [&](int s) { return bar0 + 8u * (C::B_QFULL + s); };
    auto stored = [&](int s) { return bar0 + 8u * (C::B_STORED + s); };   // a segment's rows, or the run's first part, are there
    const uint32_t counted = bar0 + 8u * C::B_COUNTED;           // the run's first part has been counted in
    const uint32_t finished = bar0 + 8u * C::B_FINISHED;         // the run's last tile has been added
    const uint32_t decided = bar0 + 8u * C::B_DECIDED;           // whether the other parts of its unit are there
    auto joined = [&](int s) { return bar0 + 8u * (C::B_JOINED + s); };  // parts of other runs are in the group's share of the ring
    const uint32_t drained = bar0 + 8u * C::B_DRAINED;           // the q warp has written every row
    const uint32_t never = bar0 + 8u * C::B_NEVER;               // completed by nothing: the fault_wait test hook waits on it
    auto scaled = [&](int s) { return bar0 + 8u * (C::B_SCALED + s); };  // a K tile's scales are there (and its V tile's), of each set
    __shared__ uint32_t sums[THREADS / 32], found_unit0;
    __shared__ float kscale[4], vscale[4];   // of each q buffer, of each key head of the unit
    __shared__ int found_b;
    __shared__ uint32_t last_flag, late_join, others_in;
    __shared__ volatile uint32_t spoilt;     // a consumer gave up: what is stored from then on is not whole

    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    if (tid == 0) {
#pragma unroll 1
        for (int s = 0; s < C::NS; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), PRODUCER);
        }
        for (int s = 0; s < C::QBUF; ++s) {
            mbar_init(qfull(s), 32);
            mbar_init(stored(s), PRODUCER);
        }
        mbar_init(counted, 1);
        mbar_init(finished, PRODUCER);
        mbar_init(decided, 1);
        for (int s = 0; s < C::NG; ++s) mbar_init(joined(s), W);
        mbar_init(drained, 1);
        mbar_init(never, 1);
        if constexpr (BLOCKS)
            for (int s = 0; s < C::NSC; ++s) mbar_init(scaled(s), 1);
        fence_mbar_init();
        spoilt = 0;
    }
    if (wid == PRODUCER && lane == 0) {
        prefetch_tmap(&k_map);
        prefetch_tmap(&v_map);
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // ---- this CTA's run of tiles: a prefix sum over the requests' tiles, which the CTA's threads share
    const int units = C::PAIR ? p.heads_kv >> 1 : p.heads_kv * p.row_tiles;
    uint32_t all_tiles = 0, ctas, run_tiles, run_unit0, run_at;
    int run_b;
    {
        const int each = (p.batch + THREADS - 1) / THREADS;
        const int b0 = min(tid * each, p.batch), b1 = min(b0 + each, p.batch);
        uint32_t mine = 0;
#pragma unroll 1
        for (int b = b0; b < b1; ++b) mine += (uint32_t)((span_of<KEYS>(p, b).tiles + 1) * units);
        uint32_t x = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t y = __shfl_up_sync(~0u, x, d);
            if (lane >= d) x += y;
        }
        uint32_t before = x - mine;
        if (lane == 31) sums[wid] = x;
        __syncthreads();
        for (int w = 0; w < THREADS / 32; ++w) {
            if (w < wid) before += sums[w];
            all_tiles += sums[w];
        }
        // no run is empty: with fewer tiles than CTAs, the first `all_tiles` CTAs take one each
        ctas = min(gridDim.x, all_tiles);
        const uint32_t c = min(blockIdx.x, ctas), per = all_tiles / ctas, over = all_tiles - per * ctas;
        const uint32_t r0 = c * per + c * over / ctas;
        run_tiles = c < ctas ? (c + 1) * per + (c + 1) * over / ctas - r0 : 0;
        if (run_tiles > 0 && before <= r0 && r0 - before < mine) {
            int b = b0;
#pragma unroll 1
            for (;; ++b) {
                const uint32_t n = (uint32_t)((span_of<KEYS>(p, b).tiles + 1) * units);
                if (r0 - before < n) break;
                before += n;
            }
            found_b = b, found_unit0 = before;
        }
        __syncthreads();
        run_b = found_b;
        run_unit0 = found_unit0;
        run_at = r0 - run_unit0;
    }
    if (blockIdx.x == 0 && p.user_status)
#pragma unroll 1
        for (int b = tid; b < p.batch; b += THREADS)
            if (p.lens[b] < 0 || p.lens[b] > ((int64_t)p.wide << p.page_shift)) atomicOr(p.user_status, 2u);
    if (run_tiles == 0) return;
    Walk<KEYS> walk;
    walk.b = run_b;
    walk.s = span_of<KEYS>(p, walk.b);
    walk.u = (int)(run_at / (uint32_t)(walk.s.tiles + 1));
    walk.t = (int)run_at - walk.u * (walk.s.tiles + 1);
    walk.unit0 = run_unit0 + (uint32_t)(walk.u * (walk.s.tiles + 1));
    walk.t0 = 1, walk.t1 = 0;
    walk.left = (int)run_tiles;
    bool ok = true;                       // no bounded wait has given up; after one, no wait is made
    auto wait = [&](uint32_t bar, uint32_t parity) {
        if (ok) ok = mbar_wait_within(bar, parity, p.wait_limit);
    };

    if (wid == PRODUCER || wid == PRODUCER + 1) {
        // ================= producers: K tiles take the ring's even turns, V tiles the odd ones
        const bool is_v = wid == PRODUCER + 1;
        const CUtensorMap* map = is_v ? &v_map : &k_map;
        const int box_shift = min(p.page_shift, KEYS == 128 ? 7 : 6), box = 1 << box_shift;
        const uint32_t page_mask = (1u << p.page_shift) - 1u;
        const uint32_t ring_u = smem_u32(ring);
        const uint32_t box_bytes = (uint32_t)box * C::PW;
        int slot = is_v ? 1 : 0;
        uint32_t phase = 0;
        int64_t turn = slot;                 // of the ring, over the whole run
        while (ok && walk.next(p, units)) {
            const Span s = walk.s;
            const int32_t* table = p.table + (int64_t)walk.b * p.table_stride;
            const int head0 = C::PAIR ? 2 * walk.u : over(walk.u, p.row_tiles, p.m_row_tiles);
            // 32 entries of the table in the lanes' registers and the next 32 on their way, so that no tile
            // waits for its entries; one that is no page becomes a page beyond the tensor, which reads as zeros
            auto entries = [&](int e) {
                int page = (int)p.pages;
                if (((int64_t)e << p.page_shift) < s.hi && (((int64_t)e + 1) << p.page_shift) > s.lo) {
                    page = table[e];
                    if ((uint32_t)page >= (uint64_t)p.pages) {
                        page = (int)p.pages;
                        if (p.user_status) atomicOr(p.user_status, 2u);
                    }
                }
                return page;
            };
            int key0 = s.base + walk.t0 * KEYS;
            int have = ((key0 >> p.page_shift) & ~31) - 64, cur = 0, nxt = 0;   // two steps before the first
#pragma unroll 1
            for (int t = walk.t0; t < walk.t1; ++t, key0 += KEYS) {
                // the tile's boxes that hold a visible key
                const int i0 = max(0, s.lo - key0) >> box_shift, i1 = (min(KEYS, s.hi - key0) + box - 1) >> box_shift;
                wait(empty(slot), phase ^ 1u);
                ok = __all_sync(~0u, ok);
                if (!ok) break;
                const uint32_t dst = ring_u + (uint32_t)slot * C::TILE, bar = full(slot);
                if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)max(0, i1 - i0) * C::HEADS * C::PANELS * box_bytes);
                __syncwarp();
#pragma unroll 1
                for (int i = i0; i < i1; ++i) {
                    const int row = i << box_shift;
                    int e = ((key0 + row) >> p.page_shift) - have;
#pragma unroll 1
                    while (e >= 32) {
                        have += 32;
                        e -= 32;
                        cur = nxt;
                        nxt = entries(have + 32 + lane);
                    }
                    const int page = __shfl_sync(~0u, cur, e);
                    const int token = (int)((uint32_t)(key0 + row) & page_mask);
#pragma unroll
                    for (int h = 0; h < C::HEADS; ++h) {
                        auto at = [&](int axis) { return axis == 0 ? token : axis == 1 ? head0 + h : page; };
                        const int c1 = at(p.axis1), c2 = at(p.axis2), c3 = at(p.axis3);
                        if (lane == 0)
#pragma unroll
                            for (int n = 0; n < C::PANELS; ++n)
                                tma_load_4d(dst + h * C::HEAD_TILE + n * KEYS * C::PW + row * C::PW, map, n * (C::PW / C::ES), c1, c2, c3,
                                            bar);
                    }
                }
                turn += 2;
                slot += 2;
                if (slot >= C::NS) slot -= C::NS, phase ^= 1u;
            }
        }
        // The next kernel's CTAs may come as this one's end: what this kernel waited for is complete.
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
        // no copy is in flight when the CTA ends, whatever its consumers did
#pragma unroll 1
        for (int64_t i = turn - 2; i >= 0 && i >= turn - C::NS; i -= 2)
            if (!mbar_wait(full((int)(i % C::NS)), (uint32_t)(i / C::NS) & 1u)) ok = false;
        if (!ok && lane == 0) atomicOr(p.status, 1u);
        return;
    }
    if (BLOCKS && wid == PRODUCER + 3) {
        // ================= scales of each tile's blocks, K's and V's, to the set that goes with the K tile's slot, within
        // bounds and V's as its logarithm.  The next tile's are loaded while this one's wait for their set.
        constexpr int EACH = (C::HEADS * KEYS + 31) / 32;     // blocks of a tile to a lane, at most
        const int count_shift = max(0, (KEYS == 128 ? 7 : 6) - p.block_shift), count = 1 << count_shift;   // of a head
        const uint32_t page_mask = (1u << p.page_shift) - 1u;
        int slot = 0, set = 0;
        uint32_t phase = 0;
        const int32_t* table = nullptr;
        int head0 = 0, key0 = 0, have = 0, cur = 0, nxt = 0;
        walk.t0 = walk.t1 = 0;
        auto entry = [&](int e) {            // of a page that a query may see, -1 of any other
            return ((int64_t)e << p.page_shift) < walk.s.hi && (((int64_t)e + 1) << p.page_shift) > walk.s.lo ? table[e] : -1;
        };
        float2 mine[EACH], next[EACH];
        auto load = [&](float2 (&x)[EACH]) {
            if (walk.t0 >= walk.t1) {
                if (!walk.next(p, units)) return false;
                table = p.table + (int64_t)walk.b * p.table_stride;
                head0 = C::PAIR ? 2 * walk.u : over(walk.u, p.row_tiles, p.m_row_tiles);
                key0 = walk.s.base + walk.t0 * KEYS;
                have = ((key0 >> p.page_shift) & ~31) - 64, cur = nxt = -1;   // as the producers have them
            }
            const int e0 = key0 >> p.page_shift;
            int tile_page = -1;              // the lane's entry of the tile, where a tile has 32 at most
            if (p.page_shift >= 2) {
#pragma unroll 1
                while (e0 - have >= 32) {
                    have += 32;
                    cur = nxt;
                    nxt = entry(have + 32 + lane);
                }
                const int e = e0 - have + lane, u = __shfl_sync(~0u, cur, e & 31), w = __shfl_sync(~0u, nxt, e & 31);
                tile_page = e < 32 ? u : w;
            }
            const bool whole = key0 >= walk.s.lo && key0 + KEYS <= walk.s.hi;
            // the lane's block `i` of the tile, of one head: where its scales are, or -1: zeros where there is no page, or
            // nothing that a query may see
            auto place = [&](int i, int head) {
                const int key = key0 + ((i & (count - 1)) << p.block_shift), e = (key >> p.page_shift) - e0;
                int page = __shfl_sync(~0u, tile_page, e & 31);
                const bool seen = whole || (key < walk.s.hi && key + (1 << p.block_shift) > walk.s.lo);
                if (p.page_shift < 2) page = seen ? table[e0 + e] : -1;
                const int in_page = (int)(((uint32_t)key & page_mask) >> p.block_shift);
                return seen && (uint32_t)page < (uint32_t)p.pages
                           ? (int64_t)page * p.s_ps + (int64_t)in_page * p.s_bs + (int64_t)(head0 + head) * p.s_hs
                           : -1;
            };
            if (C::PAIR && p.s_pairs) {
                // the two heads' scales lie side by side: registers 2j and 2j + 1 are a block's two heads
#pragma unroll
                for (int j = 0; j < EACH / 2; ++j)
                    if (32 * j < count) {
                        const int64_t at = place(32 * j + lane, 0);
                        float2 k = make_float2(0.f, 0.f), v = k;
                        if (at >= 0 && 32 * j + lane < count) {
                            k = *reinterpret_cast<const float2*>(p.k_scales + at);
                            v = *reinterpret_cast<const float2*>(p.v_scales + at);
                        }
                        x[2 * j] = make_float2(k.x, v.x);
                        x[2 * j + 1] = make_float2(k.y, v.y);
                    }
            } else {
#pragma unroll
                for (int j = 0; j < EACH; ++j)
                    if (32 * j < C::HEADS * count) {
                        const int i = 32 * j + lane, head = i >> count_shift;
                        const int64_t at = place(i, head);
                        x[j] = make_float2(0.f, 0.f);
                        if (at >= 0 && head < C::HEADS) x[j] = make_float2(p.k_scales[at], p.v_scales[at]);
                    }
            }
            key0 += KEYS;
            ++walk.t0;
            return true;
        };
        bool more = load(next);
        while (more) {
#pragma unroll
            for (int j = 0; j < EACH; ++j) mine[j] = next[j];
            more = load(next);
            wait(empty(slot), phase ^ 1u);
            ok = __all_sync(~0u, ok);
            if (!ok) break;
            float2* of = reinterpret_cast<float2*>(scales + set * C::SCALES);
            auto put = [&](int block, int head, float2 x) { of[head * KEYS + block] = make_float2(within_scales(x.x), __log2f(within_scales(x.y))); };
            if (C::PAIR && p.s_pairs) {
#pragma unroll
                for (int j = 0; j < EACH; ++j)
                    if (32 * (j >> 1) + lane < count) put(32 * (j >> 1) + lane, j & 1, mine[j]);
            } else {
#pragma unroll
                for (int j = 0; j < EACH; ++j)
                    if (32 * j + lane < C::HEADS * count) put((32 * j + lane) & (count - 1), (32 * j + lane) >> count_shift, mine[j]);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(scaled(set));
            if (++set == C::NSC) set = 0;
            slot += 2;
            if (slot >= C::NS) slot -= C::NS, phase ^= 1u;
        }
        if (!ok && lane == 0) atomicOr(p.status, 1u);
        return;
    }
    // The parts of a unit that begins at tile `unit0`: the runs from `first` on.
    struct Parts {
        uint32_t first;
        int count;
    };
    auto parts_of = [&](uint32_t unit0, int tiles) {
        Parts x;
        x.first = run_of(unit0, all_tiles, ctas);
        x.count = (int)(run_of(unit0 + tiles - 1, all_tiles, ctas) - x.first) + 1;
        return x;
    };
    // Which token and query head row r of unit u is; token >= tokens (or rows beyond the last): none.
    struct Place {
        int token, head;
    };
    auto place_of = [&](int u, int r) {
        const int hk = C::PAIR ? 2 * u + r / C::GROWS : over(u, p.row_tiles, p.m_row_tiles);
        const int at = C::PAIR ? r % C::GROWS : (u - hk * p.row_tiles) * C::ROWS + r;
        const int j = over(at, p.group, p.m_group);
        return Place{j, hk * p.group + at - j * p.group};
    };
    // Rows that are staged in q buffer `buf`, with their maxima and sums, to the output: 16 bytes a thread.
    auto copy_rows = [&](int b, int u, int buf, int first, int step) {
        constexpr int QCH = DP / 8;
        const uint8_t* stage = qbuf + buf * C::QBYTES;
        const float* stat = stats + buf * 2 * C::ROWS;
#pragma unroll 1
        for (int i = first; i < C::ROWS * QCH; i += step) {
            const int r = i / QCH, ch = i % QCH;
            const Place at = place_of(u, r);
            if (!ok || at.token >= p.tokens) continue;
            if (ch * 8 < p.dim)
                *reinterpret_cast<uint4*>(p.out + (int64_t)b * p.o_bs + (int64_t)at.token * p.o_ts + (int64_t)at.head * p.o_hs + ch * 8) =
                    *reinterpret_cast<const uint4*>(stage + qchunk_at<QCH>(r, ch));
            if (p.lse && ch == 0) {
                const float top = stat[2 * r], sum = stat[2 * r + 1];
                p.lse[((int64_t)b * p.tokens + at.token) * p.heads_q + at.head] =
                    ((top == __int_as_float(0xff800000) ? 0.f : top) + __log2f(sum) - lift(BYTES)) * 0.69314718055994531f;
            }
        }
    };
    if (wid == PRODUCER + 2) {
        // ================= q of each segment, rows (token, head of the group), and what is
        // left of a segment's end beside the stream: rows to the output, the run's first part counted in (the
        // counter of a unit's parts is the first run's)
        Walk<KEYS> ahead = walk;             // whose q is loaded next; `walk` follows the consumers
        bool more = true;
        auto load_q = [&](int qs) {
            const Walk<KEYS>& walk = ahead;
            uint8_t* dst = qbuf + qs * C::QBYTES;
            const int hk = C::PAIR ? 2 * walk.u : over(walk.u, p.row_tiles, p.m_row_tiles);
            constexpr int QCH = DP / 8;                             // 16-byte chunks of a row
            const uint16_t* base = p.q + (int64_t)walk.b * p.q_bs;
            // which token and query head each row is, for the consumers too
#pragma unroll 1
            for (int r = lane; r < C::ROWS; r += 32) {
                const Place at = place_of(walk.u, r);
                row_token[qs * C::ROWS + r] = at.token < p.tokens ? at.token : -1;
                row_head[qs * C::ROWS + r] = at.head;
            }
            __syncwarp();
            auto source = [&](int r, int ch) {
                const int j = row_token[qs * C::ROWS + r];
                return (j >= 0 && ch * 8 < p.dim) ? base + (int64_t)j * p.q_ts + (int64_t)row_head[qs * C::ROWS + r] * p.q_hs + ch * 8
                                                  : nullptr;
            };
            const uint32_t to = smem_u32(dst);
#pragma unroll 1
            for (int i = lane; i < C::ROWS * QCH; i += 32) {        // in flight together
                const uint16_t* src = source(i / QCH, i % QCH);
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + qchunk_at<QCH>(i / QCH, i % QCH)),
                             "l"(src ? src : p.q), "r"(src ? 16u : 0u) : "memory");
            }
            if constexpr (BYTES)
                if (lane < C::HEADS) {
                    kscale[2 * qs + lane] = p.k_scale ? p.k_scale[hk + lane] : 1.f;
                    vscale[2 * qs + lane] = p.v_scale ? p.v_scale[hk + lane] : 1.f;
                }
            asm volatile("cp.async.wait_all;" ::: "memory");
            mbar_arrive(qfull(qs));
        };
#pragma unroll 1
        for (int i = 0; more; ++i) {
            // q buffers in turn: the first QBUF segments' at once, then each when its buffer is free again
            if (i >= C::QBUF) {
                walk.next(p, units);
                const bool part = walk.t0 > 0 || walk.t1 < walk.s.tiles;
                if (part && walk.left <= 0) break;          // the consumers end the run
                wait(stored(i % C::QBUF), (i / C::QBUF - 1) & 1);
                ok = __all_sync(~0u, ok && !spoilt);
                if (!part) {
                    copy_rows(walk.b, walk.u, i % C::QBUF, lane, 32);
                    __syncwarp();
                } else if (lane == 0) {
                    const Parts x = parts_of(walk.unit0, walk.s.tiles);
                    late_join = ok && count_part(p.counters + x.first) == (uint32_t)x.count - 1;
                    mbar_arrive(counted);
                }
                if (walk.left <= 0) break;
            }
            if (ahead.next(p, units)) load_q(i % C::QBUF);
            else if (i == 0) more = false;                  // a run of nothing
        }
        if (walk.t0 == 0 && walk.t1 < walk.s.tiles) {
            // the run ends with its unit's first part: the other parts' runs mostly began with theirs, so
            // look for them as soon as the last tile is added, while the consumers add up their sums
            if (lane == 0) {
                const Parts x = parts_of(walk.unit0, walk.s.tiles);
                const uint32_t* counter = p.counters + x.first;
                uint32_t in = 0;
                const long long t_begin = clock64();
                for (;;) {
                    const bool over = mbar_try_wait(finished, 0);
                    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(in) : "l"(counter) : "memory");
                    if (over || in == (uint32_t)x.count - 1 || clock64() - t_begin > kWaitLimitCycles) break;
                }
                others_in = in == (uint32_t)x.count - 1;
                mbar_arrive(decided);
            }
        }
        if (lane == 0) mbar_arrive(drained);
        if (!ok && lane == 0) atomicOr(p.status, 1u);
        return;
    }

    // ===================== consumers
    const int g = lane >> 2, t2 = (lane & 3) * 2;
    constexpr int MT = C::MT, NT = C::NT, QCH = DP / 8, KB = C::KB, GROWS = C::GROWS;
    const int group = C::NG == 1 ? 0 : wid / W, cw = C::NG == 1 ? wid : wid % W, ct = C::NG == 1 ? tid : tid % GROUP;   // warp and thread of the group
    const int rb = group * GROWS;            // the group's first row
    const int own_head = C::PAIR ? group * C::HEAD_TILE : 0;   // where a tile holds the group's key head
    red += group * W * GROWS;
    lred += group * W * GROWS;
    weight += group * C::JOIN * GROWS;
    auto consumer_sync = [&] { group_sync(group); };
    auto consumer_any = [&](bool v) { return group_any(group, v); };
    int slot = 0, qs = 0, set = 0;
    uint32_t phase = 0, qphase = 0, sphase = 0;
    const uint32_t ring_u = smem_u32(ring), qbuf_u = smem_u32(qbuf), pbuf_u = smem_u32(pbuf) + group * 2 * C::PBYTES;
    uint32_t turn = 0;                       // which half of pbuf
    float acc[MT][NT][4], m[NT][2], l[NT][2];
    const float NINF = __int_as_float(0xff800000);
    auto advance = [&] {
        __syncwarp();
        if (lane == 0 && ok) mbar_arrive(empty(slot));           // its copy is complete
        if (++slot == C::NS) slot = 0, phase ^= 1u;
    };
    auto arrive_stored = [&](int buf) {
        ok = __all_sync(~0u, ok);
        if (lane != 0) return;
        if (!ok) spoilt = 1;
        mbar_arrive(stored(buf));
    };
    auto clear = [&] {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[mt][nt][e] = 0.f;
    };
    auto slot_of = [&](const Parts& x, int i) { return p.slots + (size_t)(2 * (x.first + i) + (i == 0 ? 1 : 0)) * C::SLOT_FLOATS + group * C::PART_FLOATS; };
    int join_round = 0;                      // of `joined`
    if (p.fault) wait(never, 0);

    // this run's part of a unit, to its slot
    auto store_part = [&](bool first) {
        float4* part = reinterpret_cast<float4*>(p.slots + (size_t)(2 * blockIdx.x + (first ? 1 : 0)) * C::SLOT_FLOATS + group * C::PART_FLOATS);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                __stcg(part + ((cw * MT + mt) * NT + nt) * 32 + lane,
                       make_float4(acc[mt][nt][0], acc[mt][nt][1], acc[mt][nt][2], acc[mt][nt][3]));
        if (cw == 0 && g == 0)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                __stcg(reinterpret_cast<float4*>(reinterpret_cast<float*>(part) + C::STATS + 2 * (8 * nt + t2)),
                       make_float4(m[nt][0], l[nt][0], m[nt][1], l[nt][1]));
    };

    // The parts of a unit joined, in run order: acc, m and l of the whole.  `own`: this run has the first part,
    // in registers; the same sums come out as if it were read from its slot.  The ring is free by now, so the
    // other parts come by bulk copies, as many at once as it holds: one round trip for them all.
    auto join = [&](const Parts& x, bool own) {
        constexpr uint32_t BYTES = C::PART_FLOATS * sizeof(float), SHARE = C::NS * C::TILE / C::NG;
        constexpr int ROOM = SHARE / BYTES < C::JOIN ? SHARE / BYTES : C::JOIN;
        static_assert(ROOM >= 1, "a part is larger than its share of the ring");
        constexpr int TPR = GROUP / GROWS;         // threads of a row
        const int row = ct % GROWS, p0 = ct / GROWS;
        if (own && cw == 0 && g == 0)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) red[8 * nt + t2 + e] = m[nt][e], red[GROWS + 8 * nt + t2 + e] = l[nt][e];
        consumer_sync();
        float top = NINF, sum = 0.f;
        if (own) top = red[row], sum = red[GROWS + row];
        else clear();
        consumer_sync();                                 // `red` has been read
        if (p0 > 0) sum = 0.f;                           // a row's sum is kept by its threads in pieces
#pragma unroll 1
        for (int c0 = 0; c0 < x.count; c0 += ROOM) {
            const int n = min(ROOM, x.count - c0), i0 = own && c0 == 0 ? 1 : 0;
            if (!ok) break;
            if (lane == 0) {
                asm volatile("fence.proxy.async;" ::: "memory");   // others' stores, before the copies read them
                uint32_t mine = 0;
#pragma unroll 1
                for (int i = i0 + cw; i < n; i += W) mine += BYTES;
                mbar_arrive_expect_tx(joined(group), mine);
#pragma unroll 1
                for (int i = i0 + cw; i < n; i += W) bulk_g2s(ring_u + group * SHARE + i * BYTES, slot_of(x, c0 + i), BYTES, joined(group));
            }
            const uint32_t parity = join_round++ & 1;
            wait(joined(group), parity);
            if (!ok) mbar_wait(joined(group), parity);       // no copy is in flight when the CTA ends
            const float* parts = reinterpret_cast<const float*>(ring + group * SHARE);
            const float* stats = parts + C::STATS + 2 * row;
            float high = top;
#pragma unroll 4
            for (int i = i0; i < n; ++i) high = fmaxf(high, stats[i * C::PART_FLOATS]);
            const float f = top == high ? 1.f : exp2_approx(top - high);
            sum *= f;
            top = high;
            if (p0 == 0) red[row] = f;
#pragma unroll 1
            for (int i = p0 < i0 ? p0 + TPR : p0; i < n; i += TPR) {
                const float2 st = *reinterpret_cast<const float2*>(stats + i * C::PART_FLOATS);
                const float w = st.x == top ? 1.f : exp2_approx(st.x - top);
                weight[i * GROWS + row] = w;
                sum = fmaf(w, st.y, sum);
            }
            consumer_sync();
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const float2 k = *reinterpret_cast<const float2*>(red + 8 * nt + t2);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
                    acc[mt][nt][0] *= k.x, acc[mt][nt][1] *= k.y, acc[mt][nt][2] *= k.x, acc[mt][nt][3] *= k.y;
            }
#pragma unroll (MT * NT <= 4 ? 4 : 1)
            for (int i = i0; i < n; ++i)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const float2 w = *reinterpret_cast<const float2*>(weight + i * GROWS + 8 * nt + t2);
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        const float4 a = *(reinterpret_cast<const float4*>(parts + i * C::PART_FLOATS) +
                                           ((cw * MT + mt) * NT + nt) * 32 + lane);
                        acc[mt][nt][0] = fmaf(w.x, a.x, acc[mt][nt][0]);
                        acc[mt][nt][1] = fmaf(w.y, a.y, acc[mt][nt][1]);
                        acc[mt][nt][2] = fmaf(w.x, a.z, acc[mt][nt][2]);
                        acc[mt][nt][3] = fmaf(w.y, a.w, acc[mt][nt][3]);
                    }
                }
            ok = !consumer_any(!ok);                     // the ring, `weight` and `red` serve the next parts
        }
        weight[ct] = sum;
        if (p0 == 0) red[row] = top;
        consumer_sync();
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = 8 * nt + t2 + e;
                m[nt][e] = red[r];
                float z = 0.f;
#pragma unroll
                for (int i = 0; i < TPR; ++i) z += weight[i * GROWS + r];
                l[nt][e] = z;
            }
        if (tid == 0) p.counters[x.first] = 0;           // every part has counted in: zero for the next call
        consumer_sync();                                 // `weight` and `red` serve what follows
    };

    // Rows normalised and rounded into the segment's q buffer, which has been read.  A row that sees no key
    // (whose sum is zero) is zero.
    auto stage_out = [&](float v_scale, int buf) {
        uint8_t* stage = qbuf + buf * C::QBYTES;
        float* stat = stats + buf * 2 * C::ROWS;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = rb + 8 * nt + t2 + e;
                const float inv = l[nt][e] == 0.f ? 0.f : __fdividef(v_scale, l[nt][e]);
                if (cw == 0 && g == 0) stat[2 * r] = m[nt][e], stat[2 * r + 1] = l[nt][e];
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    const int d = (cw * MT + mt) * 16 + (BYTES ? 2 * g : g);
                    uint8_t* to = stage + qchunk_at<QCH>(r, d >> 3) + (d & 7) * 2;
                    if constexpr (BYTES) {
                        *reinterpret_cast<uint32_t*>(to) = pack2<false>(acc[mt][nt][e] * inv, acc[mt][nt][e + 2] * inv);
                    } else {
                        *reinterpret_cast<__nv_bfloat16*>(to) = __float2bfloat16_rn(acc[mt][nt][e] * inv);
                        *reinterpret_cast<__nv_bfloat16*>(stage + qchunk_at<QCH>(r, (d >> 3) + 1) + (d & 7) * 2) =
                            __float2bfloat16_rn(acc[mt][nt][e + 2] * inv);
                    }
                }
            }
    };

    bool early = false;                      // the run's first segment is a part, and not the last
    int early_b = 0, early_u = 0;
    float early_scale = 1.f;
    Parts early_parts = {};
    for (;;) {
        int b, u, buf = 0;
        float v_scale;
        Parts parts = {};
        bool part, direct = false;
        if (!walk.next(p, units)) {
            // after the run: if its first segment's part was the last of its unit to be counted in, join that unit
            if (!early) break;
            early = false;
            wait(counted, 0);
            ok = consumers_all<C::CONSUMERS>(ok);
            if (!ok || late_join == 0) break;
            wait(drained, 0);                // its rows go through q buffer 0
            b = early_b, u = early_u, v_scale = early_scale, parts = early_parts, part = true;
        } else {
            const Span s = walk.s;
            const bool end_of_run = walk.left <= 0;
            b = walk.b, u = walk.u;
            part = walk.t0 > 0 || walk.t1 < s.tiles;
            if (part) parts = parts_of(walk.unit0, s.tiles);
            clear();
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                m[nt][0] = m[nt][1] = NINF;
                l[nt][0] = l[nt][1] = 0.f;
            }
            wait(qfull(qs), qphase);
            if constexpr (BYTES) {
                // q to f16, a warp to a row: times a power of two that brings the row's largest magnitude into
                // [2^13, 2^14), and within 16 dims in the order in which an 8-bit K fragment holds them: a thread's
                // four bytes 4t .. 4t + 3 are k = 2t, 2t + 1, 2t + 8, 2t + 9
                constexpr int PAIRS = DP / 64;   // of dims, of a lane
                uint8_t* rows = qbuf + qs * C::QBYTES;
                const float k_scale = p.scale_log2 * kscale[2 * qs + (C::PAIR ? group : 0)];
#pragma unroll 1
                for (int r = rb + cw; r < rb + GROWS; r += W) {
                    uint32_t w[PAIRS], big = 0;
#pragma unroll
                    for (int i = 0; i < PAIRS; ++i) {
                        const int pair = lane * PAIRS + i;
                        w[i] = *reinterpret_cast<const uint32_t*>(rows + qchunk_at<QCH>(r, pair >> 2) + (pair & 3) * 4);
                        big = max(big, max(w[i] & 0x7fffu, (w[i] >> 16) & 0x7fffu));
                    }
                    big = __reduce_max_sync(~0u, big);       // and every lane has read
                    int up = 13 - ((int)(big >> 7) - 127);
                    if (big >= 0x7f80u) up = 0;              // an infinity or NaN stays one
                    up = min(up, 126);
                    const float f = __uint_as_float((uint32_t)(up + 127) << 23);
                    if (lane == 0) qscale[qs * C::ROWS + r] = __uint_as_float((uint32_t)(127 - up) << 23) * k_scale;
#pragma unroll
                    for (int i = 0; i < PAIRS; ++i) {
                        const int pair = lane * PAIRS + i, in16 = pair & 7, k = (in16 >> 1) * 2 + (in16 & 1) * 8;
                        *reinterpret_cast<uint32_t*>(rows + qchunk_at<QCH>(r, 2 * (pair >> 3) + (k >> 3)) + (k & 7) * 2) =
                            pack2<true>(__uint_as_float(w[i] << 16) * f, __uint_as_float(w[i] & 0xffff0000u) * f);
                    }
                }
                consumer_sync();
            }
            v_scale = BYTES ? vscale[2 * qs + (C::PAIR ? group : 0)] : 1.f;
            float sc[NT][2];                     // of the scores: softmax scale, log2(e), k's scale, q's power of two
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) sc[nt][e] = BYTES ? qscale[qs * C::ROWS + rb + 8 * nt + t2 + e] : p.scale_log2;
            const uint32_t q_u = qbuf_u + qs * C::QBYTES;

#pragma unroll 1
            for (int t = walk.t0; t < walk.t1; ++t) {
                const int key0 = s.base + t * KEYS;
                // ---- S^T: this warp's 16 KB keys x all rows
                float sT[KB][NT][4];
#pragma unroll
                for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) sT[kb][nt][e] = 0.f;
                // of this thread's keys: K's scale; log2 of V's, by which P grows; and one over V's
                float ks[KB][2], lv[KB][2], rv[KB][2];
                if constexpr (BLOCKS) wait(scaled(set), sphase);
                wait(full(slot), phase);
                {
                    const uint32_t kt = ring_u + (uint32_t)slot * C::TILE + own_head;
                    // Four steps under way beside scales of blocks, whatever the rows: 16 of dim 128 take 54 us instead of 56 (e4m3 57
                    // instead of 60), 32 take 108 instead of 113, 64 take 167 instead of 170 (e4m3: 151 either way, with four 146
                    // bytes of spill), 32 of dim 256 take 186 instead of 188; 64 requests of up to 8192 keys, 4 key heads.
#pragma unroll (BLOCKS ? 4 : 2)
                    for (int s2 = 0; s2 < DP / 32; ++s2) {               // 32 dims
                        uint32_t a0[KB][4], a1[KB][4];
#pragma unroll
                        for (int kb = 0; kb < KB; ++kb) {
                            const int krow = 16 * (cw + W * kb) + (lane & 15);
                            if constexpr (BYTES) {
                                uint32_t r[4];
                                ldsm4(kt + chunk_at<C::PW, KEYS>(krow, 2 * s2 + (lane >> 4)), r);
                                bytes_f16<C::I8, false>(r[0], a0[kb][0], a0[kb][2]);
                                bytes_f16<C::I8, false>(r[1], a0[kb][1], a0[kb][3]);
                                bytes_f16<C::I8, false>(r[2], a1[kb][0], a1[kb][2]);
                                bytes_f16<C::I8, false>(r[3], a1[kb][1], a1[kb][3]);
                            } else {
                                ldsm4(kt + chunk_at<C::PW, KEYS>(krow, 4 * s2 + (lane >> 4)), a0[kb]);
                                ldsm4(kt + chunk_at<C::PW, KEYS>(krow, 4 * s2 + 2 + (lane >> 4)), a1[kb]);
                            }
                        }
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            uint32_t b[4];
                            ldsm4(q_u + qchunk_at<QCH>(rb + 8 * nt + (lane & 7), 4 * s2 + (lane >> 3)), b);
#pragma unroll
                            for (int kb = 0; kb < KB; ++kb) mma<BYTES>(sT[kb][nt], a0[kb], b[0], b[1]);
#pragma unroll
                            for (int kb = 0; kb < KB; ++kb) mma<BYTES>(sT[kb][nt], a1[kb], b[2], b[3]);
                        }
                    }
                }
                if constexpr (BLOCKS) {
                    const float2* of = reinterpret_cast<const float2*>(scales + set * C::SCALES) + (C::PAIR ? group * KEYS : 0);
#pragma unroll
                    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const float2 x = of[(16 * (cw + W * kb) + g + 8 * h) >> p.block_shift];
                            ks[kb][h] = x.x, lv[kb][h] = x.y;
                            rv[kb][h] = exp2_approx(-x.y);
                        }
                    if (++set == C::NSC) set = 0, sphase ^= 1u;
                }
                advance();   // the K tile has been read

                // ---- scores in log2 units; what a row may not see is -inf
                // every key of the tile visible to every row?
                const bool whole = key0 + KEYS <= s.len - p.tokens + 1 && (p.window <= 0 || key0 >= s.len - p.window);
#pragma unroll
                for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            sT[kb][nt][e] *= sc[nt][e & 1];
                            if constexpr (BLOCKS) sT[kb][nt][e] = fmaf(sT[kb][nt][e], ks[kb][e >> 1], lv[kb][e >> 1]);
                        }
                if (!whole) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int end = min(s.len - p.tokens + row_token[qs * C::ROWS + rb + 8 * nt + t2 + e] + 1, s.hi);
                            const int begin = p.window > 0 ? end - p.window : 0;
#pragma unroll
                            for (int kb = 0; kb < KB; ++kb) {
                                const int key = key0 + 16 * (cw + W * kb) + g;
                                if (key >= end || key < begin) sT[kb][nt][e] = NINF;
                                if (key + 8 >= end || key + 8 < begin) sT[kb][nt][e + 2] = NINF;
                            }
                        }
                }
                bool need = false;
#pragma unroll
                for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) need |= sT[kb][nt][e] > m[nt][e & 1] + lazy(BYTES);

                // ---- P^T = 2^(s - m + lift), to [nt][key][row]
                const uint32_t p_u = pbuf_u + turn * C::PBYTES;
                float sum[NT][2];                // of this lane's P, before it is rounded
                auto make_p = [&] {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const float m0 = (m[nt][0] == NINF ? 0.f : m[nt][0]) - lift(BYTES), m1 = (m[nt][1] == NINF ? 0.f : m[nt][1]) - lift(BYTES);
                        sum[nt][0] = sum[nt][1] = 0.f;
#pragma unroll
                        for (int kb = 0; kb < KB; ++kb) {
                            const uint32_t at = p_u + (nt * KEYS + 16 * (cw + W * kb) + g) * 16 + t2 * 2;
#pragma unroll
                            for (int e = 0; e < 4; e += 2) {
                                const float x = exp2_approx(sT[kb][nt][e] - m0), y = exp2_approx(sT[kb][nt][e + 1] - m1);
                                if constexpr (BLOCKS) {
                                    sum[nt][0] = fmaf(x, rv[kb][e >> 1], sum[nt][0]);
                                    sum[nt][1] = fmaf(y, rv[kb][e >> 1], sum[nt][1]);
                                } else {
                                    sum[nt][0] += x;
                                    sum[nt][1] += y;
                                }
                                if constexpr (BYTES) {
                                    st_shared(at + e * 64, pack2<true>(x, y));
                                } else {         // the upper halves, and what they leave of P (1 + 2^-23)
                                    const uint32_t bx = __float_as_uint(x), by = __float_as_uint(y);
                                    st_shared(at + e * 64, __byte_perm(bx, by, 0x7632));
                                    st_shared(at + e * 64 + C::LOW, pack2<false>(fmaf(x, 1.f + 0x1p-23f, -__uint_as_float(bx & 0xffff0000u)),
                                                                                 fmaf(y, 1.f + 0x1p-23f, -__uint_as_float(by & 0xffff0000u))));
                                }
                            }
                        }
                    }
                };
                for (bool fresh = t == walk.t0;; fresh = false) {
                    if (!fresh) {
                        make_p();
                        if (!consumer_any(need)) break;
                    }
                    // a new maximum for every row: the four warps' maxima meet in shared memory; then P again
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float x = NINF;
#pragma unroll
                            for (int kb = 0; kb < KB; ++kb) x = fmaxf(x, fmaxf(sT[kb][nt][e], sT[kb][nt][e + 2]));
                            x = fmaxf(x, __shfl_xor_sync(~0u, x, 4));
                            x = fmaxf(x, __shfl_xor_sync(~0u, x, 8));
                            x = fmaxf(x, __shfl_xor_sync(~0u, x, 16));
                            if (g == 0) red[cw * GROWS + 8 * nt + t2 + e] = x;
                        }
                    consumer_sync();
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float x = m[nt][e];
#pragma unroll
                            for (int w = 0; w < W; ++w) x = fmaxf(x, red[w * GROWS + 8 * nt + t2 + e]);
                            const float f = m[nt][e] == x ? 1.f : exp2_approx(m[nt][e] - x);
                            m[nt][e] = x;
                            l[nt][e] *= f;
#pragma unroll
                            for (int mt = 0; mt < MT; ++mt) acc[mt][nt][e] *= f, acc[mt][nt][e + 2] *= f;
                        }
                    need = false;
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) l[nt][0] += sum[nt][0], l[nt][1] += sum[nt][1];

                // ---- O^T += V^T P^T: this warp's dims, all keys of the tile
                wait(full(slot), phase);
                {
                    const uint32_t vt = ring_u + (uint32_t)slot * C::TILE + own_head;
                    // Keys that some tokens see and others do not meet P = 0 in the others' columns, where an
                    // infinity or NaN must not become one of the output: with such values among them the tokens
                    // are added one by one, each with the keys that it sees and in the same order.
                    bool apart = false;
                    if (!whole) {
                        constexpr int PCH = C::PITCH / 16;
                        uint8_t* v = ring + (size_t)slot * C::TILE + own_head;
                        // Rows outside the visible keys are not the cache's (a box reads whole pages, and skips
                        // those that nobody sees): zeros, so that P = 0 meets a number there.
                        const int z0 = max(0, min(KEYS, s.lo - key0)), z1 = max(0, min(KEYS, s.hi - key0));
#pragma unroll 1
                        for (int i = ct; i < (z0 + KEYS - z1) * PCH; i += GROUP) {
                            const int r = i / PCH, row = r < z0 ? r : z1 + r - z0;
                            *reinterpret_cast<uint4*>(v + chunk_at<C::PW, KEYS>(row, i % PCH)) = make_uint4(0, 0, 0, 0);
                        }
                        // and the rows that not every token sees: the last tokens - 1 keys, and the first of a window
                        const int a1 = p.window > 0 ? min(z1, max(z0, s.len - p.window - key0)) : z0;
                        const int b0 = max(a1, min(z1, s.len - p.tokens + 1 - key0)), n = a1 - z0 + z1 - b0;
#pragma unroll 1
                        for (int i = ct; i < n * PCH; i += GROUP) {
                            const int r = i / PCH, row = r < a1 - z0 ? z0 + r : b0 + r - (a1 - z0);
                            const uint4 w = *reinterpret_cast<const uint4*>(v + chunk_at<C::PW, KEYS>(row, i % PCH));
                            apart |= not_finite<KIND>(w.x) || not_finite<KIND>(w.y) || not_finite<KIND>(w.z) || not_finite<KIND>(w.w);
                        }
                        fence_proxy_async_smem();        // before TMA writes the slot again
                        apart = consumer_any(apart);
                    }
                    // V^T fragments of 16-dim tile mt: keys 32 kp .. 32 kp + 31, two k-steps
                    auto v_frags = [&](int kp, int mt, uint32_t (&f)[2][4]) {
                        if constexpr (BYTES) {
                            uint32_t r[4];
                            ldsm4t(vt + chunk_at<C::PW, KEYS>(32 * kp + lane, cw * MT + mt), r);
#pragma unroll
                            for (int h = 0; h < 4; ++h)              // (key, key + 1) of dim 2g, then of 2g + 1
                                bytes_f16<C::I8, true>(r[h], f[h >> 1][(h & 1) * 2], f[h >> 1][(h & 1) * 2 + 1]);
                        } else {
                            const int key = 32 * kp + (lane & 7) + ((lane >> 4) << 3);
                            const int c = 2 * (cw * MT + mt) + ((lane >> 3) & 1);
                            ldsm4t(vt + chunk_at<C::PW, KEYS>(key, c), f[0]);
                            ldsm4t(vt + chunk_at<C::PW, KEYS>(key + 16, c), f[1]);
                        }
                    };
                    auto p_frags = [&](int kp, uint32_t (&b)[C::PN][NT][4]) {
#pragma unroll
                        for (int n = 0; n < C::PN; ++n)
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                ldsm4t(p_u + n * C::LOW + (nt * KEYS + 32 * kp + lane) * 16, b[n][nt]);
                    };
                    if (!apart) {
#pragma unroll 1
                        for (int kp = 0; kp < KEYS / 32; ++kp) {
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
                                        mma<BYTES>(acc[mt][nt], f[0], b[n][nt][0], b[n][nt][1]);
                                        mma<BYTES>(acc[mt][nt], f[1], b[n][nt][2], b[n][nt][3]);
                                    }
                            }
                        }
                    } else {
#pragma unroll 1
                        for (int j = 0; j < p.tokens; ++j) {
                            const int end = s.len - p.tokens + j + 1, begin = p.window > 0 ? max(0, end - p.window) : 0;
#pragma unroll 1
                            for (int kp = 0; kp < KEYS / 32; ++kp) {
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
                                        float d[4] = {acc[mt][nt][0], acc[mt][nt][1], acc[mt][nt][2], acc[mt][nt][3]};
#pragma unroll
                                        for (int n = 0; n < C::PN; ++n) {
                                            mma<BYTES>(d, f[0], b[n][nt][0], b[n][nt][1]);
                                            mma<BYTES>(d, f[1], b[n][nt][2], b[n][nt][3]);
                                        }
#pragma unroll
                                        for (int e = 0; e < 4; ++e)
                                            if (row_token[qs * C::ROWS + rb + 8 * nt + t2 + (e & 1)] == j) acc[mt][nt][e] = d[e];
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
            buf = qs;
            if (++qs == C::QBUF) qs = 0, qphase ^= 1u;
            __syncwarp();
            if (lane == 0 && end_of_run) mbar_arrive(finished);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float x = l[nt][e];
                    x += __shfl_xor_sync(~0u, x, 4);
                    x += __shfl_xor_sync(~0u, x, 8);
                    x += __shfl_xor_sync(~0u, x, 16);
                    if (g == 0) lred[cw * GROWS + 8 * nt + t2 + e] = x;
                }
            consumer_sync();
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float x = 0.f;
#pragma unroll
                    for (int w = 0; w < W; ++w) x += lred[w * GROWS + 8 * nt + t2 + e];
                    l[nt][e] = x;
                }
            if (part && !end_of_run) {
                // the run's first part: to its slot, and on with the next segment; the q warp counts it in
                store_part(false);
                early = true;
                early_b = b, early_u = u, early_scale = v_scale, early_parts = parts;
                arrive_stored(buf);
                continue;
            }
            if (part) {
                if (walk.t0 == 0) {
                    wait(decided, 0);
                    ok = consumers_all<C::CONSUMERS>(ok);
                    direct = ok && others_in != 0;
                }
                if (!direct) {
                    store_part(walk.t0 == 0);
                    ok = consumers_all<C::CONSUMERS>(ok);
                    if (tid == 0) last_flag = ok && count_part(p.counters + parts.first) == (uint32_t)parts.count - 1;
                    consumers_sync<C::CONSUMERS>();
                    if (last_flag == 0) continue;
                }
            }
        }
        if (part) join(parts, direct);
        stage_out(v_scale, buf);
        if (!part) {
            arrive_stored(buf);                                  // the q warp writes the rows
        } else {
            ok = consumers_all<C::CONSUMERS>(ok);
            copy_rows(b, u, buf, tid, C::CONSUMERS);
            consumers_sync<C::CONSUMERS>();                                // before the buffer is staged again
        }
    }
    if (!ok) atomicOr(p.status, 1u);
}

template <int DP, int NA, int KIND, bool LASTING, bool PAIR>
struct Launch {
    static constexpr int KB = key_blocks(DP * (KIND == KV_BF16 ? 2 : 1), NA, LASTING);
    using C = Cfg<DP, NA, KIND, KB, PAIR>;
    static AttnShape shape() {
        AttnShape s;
        s.ctas_per_sm = C::CPS;
        s.rows = C::ROWS;
        s.keys = C::KEYS;
        s.slot_floats = C::SLOT_FLOATS;
        return s;
    }
    static cudaError_t allow() {
        return cudaFuncSetAttribute(paged_attn_kernel<DP, NA, KIND, KB, PAIR>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM);
    }
    static cudaError_t launch(const AttnParams& p, const CUtensorMap& k, const CUtensorMap& v, int grid, cudaStream_t st) {
        return launch_pdl(paged_attn_kernel<DP, NA, KIND, KB, PAIR>, dim3((unsigned)grid), C::THREADS, C::SMEM, st, p, k, v);
    }
};

// Row tiles hold 8 NA rows, the fewest that take all rows at once, up to 64
// (32 at dim 256, whose accumulators fill the registers, and 16 at dim 512,
// whose tiles fill shared memory); more rows go to several tiles, each of
// which reads the keys again, the later ones mostly from L2.
// BLOCKS: a scale for each block of tokens and head; bytes: e4m3 rather than bf16, with BLOCKS int8 rather than e4m3.
template <int DP, bool BLOCKS, typename Then>
auto with_rows(bool bytes, bool lasting, bool pair, int rows, Then then) {
    constexpr int MOST = DP <= 128 ? 8 : DP == 256 ? 4 : 2;
    constexpr int ONE = BLOCKS ? KV_E4M3_BLOCKS : KV_BF16, OTHER = BLOCKS ? KV_I8_BLOCKS : KV_E4M3;
    auto typed = [&](auto na) {
        constexpr int NA = decltype(na)::value;
        if (bytes) return lasting ? then(Launch<DP, NA, OTHER, true, false>{}) : then(Launch<DP, NA, OTHER, false, false>{});
        return lasting ? then(Launch<DP, NA, ONE, true, false>{}) : then(Launch<DP, NA, ONE, false, false>{});
    };
    if constexpr (DP <= 128)
        if (pair && bytes) return then(Launch<DP, 2, OTHER, true, true>{});
    if constexpr (DP <= 64 || (BLOCKS && DP <= 128))
        if (pair) return then(Launch<DP, 2, ONE, true, true>{});
    if (rows <= 8) return typed(std::integral_constant<int, 1>{});
    if (rows <= 16 || MOST == 2) return typed(std::integral_constant<int, 2>{});
    if (rows <= 32 || MOST == 4) return typed(std::integral_constant<int, MOST < 4 ? 2 : 4>{});
    return typed(std::integral_constant<int, MOST < 8 ? 2 : 8>{});
}

template <int DP, bool BLOCKS>
AttnShape shape(bool bytes, bool lasting, bool pair, int rows) {
    return with_rows<DP, BLOCKS>(bytes, lasting, pair, rows, [](auto l) { return l.shape(); });
}
template <int DP, bool BLOCKS>
cudaError_t allow_all() {
    for (int i = 0; i < 32; ++i) {
        const cudaError_t e = with_rows<DP, BLOCKS>(i & 1, i & 2, i & 4, 8 << (i >> 3), [](auto l) { return l.allow(); });
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}
template <int DP, bool BLOCKS>
cudaError_t launch(bool bytes, bool lasting, bool pair, int rows, const AttnParams& p, const CUtensorMap& k, const CUtensorMap& v, int grid,
                   cudaStream_t st) {
    return with_rows<DP, BLOCKS>(bytes, lasting, pair, rows, [&](auto l) { return l.launch(p, k, v, grid, st); });
}

}  // namespace attn
}  // namespace affqmm

#define AFFQMM_ATTN_DEFINE(DP, NAME, BLOCKS)                                                                                \
    namespace affqmm {                                                                                                      \
    AttnShape attn_shape_##NAME(bool bytes, bool lasting, bool pair, int rows) {                                            \
        return attn::shape<DP, BLOCKS>(bytes, lasting, pair, rows);                                                         \
    }                                                                                                                       \
    cudaError_t attn_allow_smem_##NAME() { return attn::allow_all<DP, BLOCKS>(); }                                          \
    cudaError_t launch_attn_##NAME(bool bytes, bool lasting, bool pair, int rows, const AttnParams& p, const CUtensorMap& k, \
                                   const CUtensorMap& v, int grid, cudaStream_t st) {                                       \
        return attn::launch<DP, BLOCKS>(bytes, lasting, pair, rows, p, k, v, grid, st);                                     \
    }                                                                                                                       \
    }
