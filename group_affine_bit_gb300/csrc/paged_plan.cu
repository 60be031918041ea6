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
// One launch.  Every CTA makes the prefix sums for itself (two block scans of
// at most 16 requests a thread, from L2) and keeps them in shared memory,
// eight bytes a request, rather than waiting for another CTA's; then each
// takes its share of the tokens, four to a thread, finds their request by
// bisection and writes slot, position and request with 16-byte stores.  The
// call is bound by latency: lengths, scan, table or ring entry, store.
#include "affqmm_internal.h"
#include "affqmm_paged.h"

namespace affqmm {
namespace {

constexpr int PL_THREADS = 1024;
constexpr uint32_t PL_MOST = (1u << 30) - 1;   // sums saturate here: no pool and no capacity reaches it
constexpr uint32_t PL_SERVED = 1u << 31, PL_FINISHED = 1u << 30;

__device__ __forceinline__ uint32_t sat_add(uint32_t a, uint32_t b) { return min(a + b, PL_MOST); }

// Exclusive prefix sum over the block's threads (saturating, so the order of
// the additions does not matter); `total` gets the block's sum.
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t* warp_sums, uint32_t* total) {
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    uint32_t x = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const uint32_t y = __shfl_up_sync(~0u, x, d);
        if (lane >= d) x = sat_add(x, y);
    }
    if (lane == 31) warp_sums[wid] = x;
    __syncthreads();
    uint32_t w = warp_sums[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const uint32_t y = __shfl_up_sync(~0u, w, d);
        if (lane >= d) w = sat_add(w, y);
    }
    *total = __shfl_sync(~0u, w, 31);
    const uint32_t before_warp = __shfl_sync(~0u, w, (wid + 31) & 31);
    const uint32_t up = __shfl_up_sync(~0u, x, 1);
    return sat_add(wid ? before_warp : 0u, lane ? up : 0u);
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
    a.fresh = (a.bad || a.done) ? 0u : min((uint32_t)fresh, PL_MOST);
    return a;
}

__global__ void __launch_bounds__(PL_THREADS) paged_plan_kernel(PlanParams p) {
    extern __shared__ uint32_t plan_smem[];
    uint32_t* starts = plan_smem;                   // [batch + 1] first token of each request
    uint32_t* first = plan_smem + p.batch + 1;      // [batch] first page taken (or given back), and the flags
    __shared__ uint32_t warp_sums[4][32];
    __shared__ uint32_t flags, taken;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int tid = threadIdx.x;
    const uint32_t page_mask = (1u << p.page_shift) - 1u;
    if (tid == 0) flags = 0, taken = 0;
    const int32_t head_in = p.ring_state[0], free_in = p.ring_state[1];
    const bool ring_ok = head_in >= 0 && head_in < p.pool && free_in >= 0 && free_in <= p.pool;
    const uint32_t head = ring_ok ? (uint32_t)head_in : 0u, free = ring_ok ? (uint32_t)free_in : 0u;
    const uint32_t pool = (uint32_t)p.pool;

    // requests i0 .. i1 - 1 are this thread's
    const int each = (p.batch + PL_THREADS - 1) / PL_THREADS;
    const int i0 = min(tid * each, p.batch), i1 = min(i0 + each, p.batch);
    uint32_t sum = 0, total;
    for (int i = i0; i < i1; ++i) sum = sat_add(sum, ask_of(p, i).fresh);
    const uint32_t token0 = block_scan(sum, warp_sums[0], &total);

    uint32_t need_sum = 0, back_sum = 0, bits = ring_ok ? 0u : 8u, at = token0;
    for (int i = i0; i < i1; ++i) {
        const Ask a = ask_of(p, i);
        const uint32_t held = (a.len + page_mask) >> p.page_shift;
        starts[i] = at;
        at = sat_add(at, a.fresh);
        const bool wide_ok = (uint64_t)a.len + a.fresh <= (uint64_t)p.wide << p.page_shift;
        const bool room = at <= (uint32_t)p.capacity;
        const bool fits = !a.done && !a.bad && wide_ok && room;
        if (a.bad) bits |= 8u;
        if (!a.done && !wide_ok) bits |= 2u;
        if (!a.done && !room) bits |= 4u;
        need_sum = sat_add(need_sum, fits ? ((a.len + a.fresh + page_mask) >> p.page_shift) - held : 0u);
        back_sum = sat_add(back_sum, a.done ? held : 0u);
    }
    if (tid == 0) starts[p.batch] = total;
    uint32_t need_total, back_total;
    const uint32_t need0 = block_scan(need_sum, warp_sums[1], &need_total);
    const uint32_t back0 = block_scan(back_sum, warp_sums[2], &back_total);
    const bool back_ok = (uint64_t)free + back_total <= pool;   // else the ring's count and the requests disagree
    if (!back_ok) bits |= 8u;

    uint32_t need_at = need0, back_at = back0, got = 0;
    for (int i = i0; i < i1; ++i) {
        const Ask a = ask_of(p, i);
        const uint32_t held = (a.len + page_mask) >> p.page_shift;
        const uint32_t end = sat_add(starts[i], a.fresh);
        const bool fits = !a.done && !a.bad && (uint64_t)a.len + a.fresh <= (uint64_t)p.wide << p.page_shift &&
                          end <= (uint32_t)p.capacity;
        const uint32_t need = fits ? ((a.len + a.fresh + page_mask) >> p.page_shift) - held : 0u;
        const uint32_t before = need_at;
        need_at = sat_add(need_at, need);
        const bool served = fits && (need == 0 || need_at <= free);
        if (fits && !served) bits |= 1u;
        if (served && need) got = need_at;
        uint32_t word = served ? (before | PL_SERVED) : before;
        if (a.done) {
            word = back_at | PL_FINISHED;
            back_at = sat_add(back_at, held);
        }
        first[i] = word;
        if (blockIdx.x == 0) {
            p.starts[i] = (int32_t)starts[i];
            p.lens_out[i] = a.done ? 0 : (served ? (int32_t)(a.len + a.fresh) : p.lens[i]);
        }
    }
    if (bits) atomicOr(&flags, bits);
    if (got) atomicMax(&taken, got);
    __syncthreads();
    if (blockIdx.x == 0 && tid == 0) {
        p.starts[p.batch] = (int32_t)total;
        const uint32_t back = back_ok ? back_total : 0u;
        const uint32_t moved = head + taken;
        p.ring_state_out[0] = (int32_t)(moved >= pool ? moved - pool : moved);
        p.ring_state_out[1] = (int32_t)(free - taken + back);
        p.status[0] = (int32_t)flags;
    }

    // ---- this CTA's tokens, four at a time
    const int64_t quads = ((int64_t)p.capacity + 3) >> 2;
    for (int64_t qd = (int64_t)blockIdx.x * PL_THREADS + tid; qd < quads; qd += (int64_t)gridDim.x * PL_THREADS) {
        const uint32_t t0 = (uint32_t)qd << 2;
        int r = p.batch;
        if (t0 < total) {   // the last request that starts at or before t0
            int lo = 0, hi = p.batch;
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (starts[mid] <= t0) lo = mid;
                else hi = mid;
            }
            r = lo;
        }
        int32_t slot[4], pos[4], req[4];
        uint32_t len = 0, word = 0;
        int have = -1;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t t = t0 + e;
            slot[e] = -1, pos[e] = 0, req[e] = -1;
            if (t < total) {
                while (starts[r + 1] <= t) ++r;
                if (have != r) {
                    have = r;
                    len = (uint32_t)p.lens[r];
                    word = first[r];
                }
                const uint32_t place = len + (t - starts[r]);
                pos[e] = (int32_t)place;
                req[e] = r;
                if (word & PL_SERVED) {
                    const uint32_t held = (len + page_mask) >> p.page_shift, pg = place >> p.page_shift;
                    int32_t* entry = p.table + (int64_t)r * p.table_stride + pg;
                    int32_t page;
                    if (pg >= held) {
                        uint32_t x = head + (word & PL_MOST) + (pg - held);
                        if (x >= pool) x -= pool;
                        page = p.ring[x];
                        if ((place & page_mask) == 0) *entry = page;
                    } else {
                        page = *entry;
                    }
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
            const Ask a = ask_of(p, i);
            const uint32_t held = (a.len + page_mask) >> p.page_shift;
            for (uint32_t j = lane; j < held; j += 32) {
                uint32_t x = head + free + (word & PL_MOST) + j;
                if (x >= pool) x -= pool;
                if (x >= pool) x -= pool;
                p.ring[x] = p.table[(int64_t)i * p.table_stride + j];
            }
        }
    }
}

}  // namespace

cudaError_t launch_paged_plan(const PlanParams& p, int sms, cudaStream_t st) {
    const size_t smem = ((size_t)2 * p.batch + 1) * sizeof(uint32_t);
    // a CTA for each 4096 tokens and for each 256 requests, up to one an SM
    int64_t grid = ((int64_t)p.capacity + 4095) / 4096;
    if (grid < (p.batch + 255) / 256) grid = (p.batch + 255) / 256;
    if (grid > sms) grid = sms;
    if (grid < 1) grid = 1;
    if (smem > 40 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(paged_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   (2 * AFFQMM_PAGED_MAX_BATCH + 1) * (int)sizeof(uint32_t));
        if (e != cudaSuccess) return e;
    }
    return launch_pdl(paged_plan_kernel, dim3((unsigned)grid), PL_THREADS, smem, st, p);
}

}  // namespace affqmm
