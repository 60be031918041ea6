// paged_plan.cu -- a step's block tables and slot maps, built on the GPU from
// the requests' lengths.
//
// With P tokens a page, request i holds ceil(len_i / P) pages and needs
// ceil((len_i + new_i) / P).  Three prefix sums over the requests -- of the
// new tokens, of the pages they need and of the pages that finished requests
// give back -- say where each request's tokens and pages begin.  Free pages
// wait in a ring: a step takes its pages from the front and puts the returned
// ones behind the back, so nothing that is read here is also written, and the
// same call on the same inputs writes the same values.
//
// One launch.  Every CTA makes the prefix sums for itself, from L2, rather than
// waiting for another CTA's: its requests are loaded once, into registers (1 to
// 16 a thread, by the batch), scanned in two rounds (tokens and returned pages,
// then needed pages, which depend on which requests fit) and kept in shared
// memory, twelve bytes a request.  Then each CTA takes its share of the tokens,
// four to a thread, finds their request by bisection and writes slot, position
// and request with 16-byte stores.  The call is bound by latency: lengths,
// scans, table or ring entry, store.
#include "affqmm_internal.h"
#include "affqmm_paged.h"

namespace affqmm {
namespace {

constexpr int PL_THREADS = 1024;
constexpr uint32_t PL_LIMIT = 0x7fffffffu;      // sums saturate here: beyond every pool (below 2^30) and capacity (up to 2^30)
constexpr uint32_t PL_SERVED = 1u << 31, PL_FINISHED = 1u << 30;
constexpr uint32_t PL_PAGE = PL_FINISHED - 1;   // and below the flags, a page's place among the pages taken or given back

__device__ __forceinline__ uint32_t sat_add(uint32_t a, uint32_t b) { return min(a + b, PL_LIMIT); }

// Exclusive prefix sums of two values over the block's threads (saturating, so
// the order of the additions does not matter), and their totals.
struct Pair {
    uint32_t a, b;
};
__device__ __forceinline__ Pair block_scan(Pair v, Pair* warp_sums, Pair* total) {
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    Pair x = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const uint32_t a = __shfl_up_sync(~0u, x.a, d), b = __shfl_up_sync(~0u, x.b, d);
        if (lane >= d) x.a = sat_add(x.a, a), x.b = sat_add(x.b, b);
    }
    if (lane == 31) warp_sums[wid] = x;
    __syncthreads();
    Pair w = warp_sums[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const uint32_t a = __shfl_up_sync(~0u, w.a, d), b = __shfl_up_sync(~0u, w.b, d);
        if (lane >= d) w.a = sat_add(w.a, a), w.b = sat_add(w.b, b);
    }
    *total = {__shfl_sync(~0u, w.a, 31), __shfl_sync(~0u, w.b, 31)};
    const Pair before = {__shfl_sync(~0u, w.a, (wid + 31) & 31), __shfl_sync(~0u, w.b, (wid + 31) & 31)};
    const Pair up = {__shfl_up_sync(~0u, x.a, 1), __shfl_up_sync(~0u, x.b, 1)};
    return {sat_add(wid ? before.a : 0u, lane ? up.a : 0u), sat_add(wid ? before.b : 0u, lane ? up.b : 0u)};
}

struct Ask {
    uint32_t len, fresh;   // tokens in the cache, new tokens
    bool done, bad;
};

__device__ __forceinline__ Ask ask_of(const PlanParams& p, int i) {
    Ask a;
    const int32_t len = p.lens[i], fresh = p.fresh[i];
    a.done = p.finished && p.finished[i];
    // a length that no table row can hold, or a negative count: the request is left alone
    a.bad = len < 0 || (int64_t)len > ((int64_t)p.wide << p.page_shift) || (!a.done && fresh < 0);
    a.len = a.bad ? 0u : (uint32_t)len;
    a.fresh = (a.bad || a.done) ? 0u : (uint32_t)fresh;
    return a;
}

template <int EACH>
__global__ void __launch_bounds__(PL_THREADS) paged_plan_kernel(PlanParams p) {
    extern __shared__ uint32_t plan_smem[];
    uint32_t* starts = plan_smem;                   // [batch + 1] first token of each request
    uint32_t* first = plan_smem + p.batch + 1;      // [batch] first page taken (or given back), and the flags
    uint32_t* length = first + p.batch;             // [batch] tokens in the cache
    __shared__ Pair warp_sums[2][32];
    __shared__ uint32_t flags, taken;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int tid = threadIdx.x;
    const uint32_t page_mask = (1u << p.page_shift) - 1u;
    if (tid == 0) flags = 0, taken = 0;
    // requests i0 .. i0 + EACH - 1 are this thread's
    const int i0 = tid * EACH;
    Ask ask[EACH];
#pragma unroll
    for (int k = 0; k < EACH; ++k) {
        ask[k] = {0, 0, false, false};
        if (i0 + k < p.batch) ask[k] = ask_of(p, i0 + k);
    }
    const int32_t head_in = p.ring_state[0], free_in = p.ring_state[1];
    const bool ring_ok = head_in >= 0 && head_in < p.pool && free_in >= 0 && free_in <= p.pool;
    const uint32_t head = ring_ok ? (uint32_t)head_in : 0u, free = ring_ok ? (uint32_t)free_in : 0u;
    const uint32_t pool = (uint32_t)p.pool;

    Pair sum = {0, 0}, total, needed;
#pragma unroll
    for (int k = 0; k < EACH; ++k) {
        sum.a = sat_add(sum.a, ask[k].fresh);
        sum.b = sat_add(sum.b, ask[k].done ? (ask[k].len + page_mask) >> p.page_shift : 0u);
    }
    const Pair at0 = block_scan(sum, warp_sums[0], &total);
    const uint32_t tokens = total.a, back_total = total.b;
    const bool back_ok = (uint64_t)free + back_total <= pool;   // else the ring's count and the requests disagree
    uint32_t bits = (ring_ok ? 0u : 8u) | (back_ok ? 0u : 8u), at = at0.a;
    uint32_t need[EACH];
    bool fits[EACH];
    Pair want = {0, 0};
#pragma unroll
    for (int k = 0; k < EACH; ++k) {
        const Ask& a = ask[k];
        const uint32_t end = sat_add(at, a.fresh);
        const bool wide_ok = (uint64_t)a.len + a.fresh <= (uint64_t)p.wide << p.page_shift, room = end <= (uint32_t)p.capacity;
        need[k] = 0;
        fits[k] = false;
        if (i0 + k < p.batch) {
            starts[i0 + k] = at;
            length[i0 + k] = a.len;
            fits[k] = !a.done && !a.bad && wide_ok && room;
            if (a.bad) bits |= 8u;
            if (!a.done && !wide_ok) bits |= 2u;
            if (!a.done && !room) bits |= 4u;
            if (fits[k]) need[k] = ((a.len + a.fresh + page_mask) >> p.page_shift) - ((a.len + page_mask) >> p.page_shift);
            if (blockIdx.x == 0) p.starts[i0 + k] = (int32_t)at;
        }
        at = end;
        want.a = sat_add(want.a, need[k]);
    }
    if (tid == 0) starts[p.batch] = tokens;
    uint32_t need_at = block_scan(want, warp_sums[1], &needed).a, back_at = at0.b, got = 0;
#pragma unroll
    for (int k = 0; k < EACH; ++k) {
        const Ask& a = ask[k];
        const uint32_t before = need_at;
        need_at = sat_add(need_at, need[k]);
        const bool served = fits[k] && (need[k] == 0 || need_at <= free);
        if (fits[k] && !served) bits |= 1u;
        if (served && need[k]) got = need_at;
        uint32_t word = served ? (before | PL_SERVED) : 0u;   // before <= free, below 2^30
        if (a.done) {
            word = (back_at & PL_PAGE) | PL_FINISHED;         // used where all pages given back fit the pool
            back_at = sat_add(back_at, (a.len + page_mask) >> p.page_shift);
        }
        if (i0 + k < p.batch) {
            first[i0 + k] = word;
            if (blockIdx.x == 0)
                p.lens_out[i0 + k] = a.done ? 0 : a.bad ? p.lens[i0 + k] : (int32_t)(a.len + (served ? a.fresh : 0u));
        }
    }
    if (bits) atomicOr(&flags, bits);
    if (got) atomicMax(&taken, got);
    __syncthreads();
    if (blockIdx.x == 0 && tid == 0) {
        p.starts[p.batch] = (int32_t)tokens;
        const uint32_t moved = head + taken;
        p.ring_state_out[0] = (int32_t)(moved >= pool ? moved - pool : moved);
        p.ring_state_out[1] = (int32_t)(free - taken + (back_ok ? back_total : 0u));
        p.status[0] = (int32_t)flags;
    }

    // ---- this CTA's tokens, four at a time
    const int64_t quads = ((int64_t)p.capacity + 3) >> 2;
    for (int64_t qd = (int64_t)blockIdx.x * PL_THREADS + tid; qd < quads; qd += (int64_t)gridDim.x * PL_THREADS) {
        const uint32_t t0 = (uint32_t)qd << 2;
        int r = p.batch;
        if (t0 < tokens) {   // the last request that starts at or before t0
            int lo = 0, hi = p.batch;
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (starts[mid] <= t0) lo = mid;
                else hi = mid;
            }
            r = lo;
        }
        int32_t slot[4], pos[4], req[4];
        uint32_t len = 0, word = 0, have_pg = 0;
        int32_t page = -1;       // page have_pg of request `have`: one entry serves the tokens in it
        int have = -1;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t t = t0 + e;
            slot[e] = -1, pos[e] = 0, req[e] = -1;
            if (t < tokens) {
                while (starts[r + 1] <= t) ++r;
                bool look = false;
                if (have != r) {
                    have = r;
                    look = true;
                    len = length[r];
                    word = first[r];
                }
                const uint32_t place = len + (t - starts[r]);
                pos[e] = (int32_t)place;
                req[e] = r;
                if (word & PL_SERVED) {
                    const uint32_t held = (len + page_mask) >> p.page_shift, pg = place >> p.page_shift;
                    int32_t* entry = p.table + (int64_t)r * p.table_stride + pg;
                    if (look || pg != have_pg) {
                        have_pg = pg;
                        uint32_t x = head + (word & PL_PAGE) + (pg - held);
                        if (x >= pool) x -= pool;
                        page = pg >= held ? p.ring[x] : *entry;
                    }
                    if (pg >= held && (place & page_mask) == 0) *entry = page;
                    slot[e] = (int32_t)(((uint32_t)page << p.page_shift) | (place & page_mask));
                }
            }
        }
        if ((int64_t)t0 + 4 <= p.capacity) {
            reinterpret_cast<int4*>(p.slots)[qd] = make_int4(slot[0], slot[1], slot[2], slot[3]);
            reinterpret_cast<int4*>(p.positions)[qd] = make_int4(pos[0], pos[1], pos[2], pos[3]);
            reinterpret_cast<int4*>(p.requests)[qd] = make_int4(req[0], req[1], req[2], req[3]);
        } else {
            for (int e = 0; (int64_t)t0 + e < p.capacity; ++e)
                p.slots[t0 + e] = slot[e], p.positions[t0 + e] = pos[e], p.requests[t0 + e] = req[e];
        }
    }

    // ---- finished requests' pages go behind the free ones, a warp to a request
    if (back_total && back_ok) {
        const int lane = tid & 31, warps = (PL_THREADS / 32) * gridDim.x;
        for (int i = blockIdx.x * (PL_THREADS / 32) + (tid >> 5); i < p.batch; i += warps) {
            const uint32_t word = first[i];
            if ((word & (PL_SERVED | PL_FINISHED)) != PL_FINISHED) continue;
            const uint32_t held = (length[i] + page_mask) >> p.page_shift;
            const int32_t* row = p.table + (int64_t)i * p.table_stride;
            constexpr int GO = 8;    // loads in flight
            for (uint32_t j0 = lane; j0 < held; j0 += 32 * GO) {
                int32_t page[GO];
#pragma unroll
                for (int k = 0; k < GO; ++k)
                    if (j0 + 32 * k < held) page[k] = row[j0 + 32 * k];
#pragma unroll
                for (int k = 0; k < GO; ++k)
                    if (j0 + 32 * k < held) {
                        uint32_t x = head + free + (word & PL_PAGE) + j0 + 32 * k;
                        if (x >= pool) x -= pool;
                        if (x >= pool) x -= pool;
                        p.ring[x] = page[k];
                    }
            }
        }
    }
}

}  // namespace

namespace {
template <int EACH>
cudaError_t launch_each(const PlanParams& p, unsigned grid, size_t smem, cudaStream_t st) {
    if (smem > 40 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(paged_plan_kernel<EACH>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    return launch_pdl(paged_plan_kernel<EACH>, dim3(grid), PL_THREADS, smem, st, p);
}
}  // namespace

cudaError_t launch_paged_plan(const PlanParams& p, int sms, cudaStream_t st) {
    const size_t smem = ((size_t)3 * p.batch + 1) * sizeof(uint32_t);
    // a CTA for each 4096 tokens and for each 256 requests, up to one an SM
    int64_t grid = ((int64_t)p.capacity + 4095) / 4096;
    if (grid < (p.batch + 255) / 256) grid = (p.batch + 255) / 256;
    if (grid > sms) grid = sms;
    if (grid < 1) grid = 1;
    if (p.batch <= PL_THREADS) return launch_each<1>(p, (unsigned)grid, smem, st);
    if (p.batch <= 4 * PL_THREADS) return launch_each<4>(p, (unsigned)grid, smem, st);
    return launch_each<16>(p, (unsigned)grid, smem, st);
}

}  // namespace affqmm
