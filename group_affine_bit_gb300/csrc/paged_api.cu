// paged_api.cu -- the C ABI of the paged key-value cache: host-side validation
// and the launches.  See include/affqmm.h for the contract.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <mutex>

#include "affqmm.h"
#include "affqmm_async.cuh"
#include "affqmm_internal.h"
#include "affqmm_paged.h"

using namespace affqmm;

namespace {

constexpr int kMaxDevices = 64;
constexpr int64_t kMost = (int64_t)1 << 30;   // tokens of a step, pages of a pool

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// The shift of a page size, or -1 if it is no power of two up to 65536.
int page_shift_of(int64_t page) {
    for (int s = 0; s <= 16; ++s)
        if (page == (int64_t)1 << s) return s;
    return -1;
}

// The cache's axes (0 token, 1 head, 2 page) in the order of their strides, those that are stepped along first.
struct Axes {
    int order[3];
    int64_t stride[3];   // elements; of an axis of one, which is never stepped along, the one before it
};
Axes axes_of(const affqmm_kv_cache* c) {
    const int64_t size[3] = {c->page, c->heads, c->pages}, stride[3] = {c->token_stride, c->head_stride, c->page_stride};
    Axes a;
    int n = 0;
    for (int i = 0; i < 3; ++i) {
        if (size[i] == 1) continue;
        int j = n++;
        for (; j > 0 && stride[i] < stride[a.order[j - 1]]; --j) a.order[j] = a.order[j - 1];
        a.order[j] = i;
    }
    for (int j = 0; j < n; ++j) a.stride[j] = stride[a.order[j]];
    for (int i = 0; i < 3; ++i)
        if (size[i] == 1) {
            a.order[n] = i;
            a.stride[n] = n ? a.stride[n - 1] : c->dim;
            ++n;
        }
    return a;
}

int check_cache(const affqmm_kv_cache* c, bool memory) {
    if (!c) return AFFQMM_E_NULL;
    if (c->type != AFFQMM_KV_BF16 && c->type != AFFQMM_KV_E4M3) return AFFQMM_E_ARG;
    if (page_shift_of(c->page) < 0) return AFFQMM_E_ARG;
    if (c->type == AFFQMM_KV_BF16 && (c->k_scale || c->v_scale)) return AFFQMM_E_ARG;
    if (c->heads < 1 || c->heads > 4096 || c->dim < 16 || c->dim > 512 || c->dim % 16) return AFFQMM_E_SHAPE;
    if (c->pages < 1 || c->pages >= kMost || c->pages * c->page >= (int64_t)1 << 31) return AFFQMM_E_SHAPE;
    const int64_t size[3] = {c->pages, c->page, c->heads}, stride[3] = {c->page_stride, c->token_stride, c->head_stride};
    for (int i = 0; i < 3; ++i)
        if (size[i] > 1 && (stride[i] < c->dim || stride[i] >= (int64_t)1 << 38)) return AFFQMM_E_SHAPE;
    if (!memory) return AFFQMM_OK;
    if (!c->k || !c->v) return AFFQMM_E_NULL;
    const int64_t each = c->type == AFFQMM_KV_E4M3 ? 16 : 8;
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))
        return AFFQMM_E_ALIGN;
    for (int i = 0; i < 3; ++i)
        if (size[i] > 1 && stride[i] % each) return AFFQMM_E_ALIGN;
    const Axes a = axes_of(c);
    for (int i = 1; i < 3; ++i)
        if (a.stride[i] % a.stride[i - 1]) return AFFQMM_E_ALIGN;
    return AFFQMM_OK;
}

int check_rows(const void* p, int64_t s0, int64_t s1, int64_t s2) {
    if (!p) return AFFQMM_E_NULL;
    if (s0 < 0 || s1 < 0 || s2 < 0) return AFFQMM_E_SHAPE;
    if (!aligned(p, 16) || s0 % 8 || s1 % 8 || s2 % 8) return AFFQMM_E_ALIGN;
    return AFFQMM_OK;
}

// Shared-memory limits of the attention kernels, set once per device and head dim.
std::once_flag g_once[kMaxDevices][4];
bool g_ok[kMaxDevices][4];

int allow_attn(int which) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return AFFQMM_E_CUDA;
    if (dev < 0 || dev >= kMaxDevices) return AFFQMM_E_DEVICE;
    std::call_once(g_once[dev][which], [&] {
        const cudaError_t e = which == 0   ? attn_allow_smem_64()
                              : which == 1 ? attn_allow_smem_128()
                              : which == 2 ? attn_allow_smem_256()
                                           : attn_allow_smem_512();
        g_ok[dev][which] = e == cudaSuccess;
    });
    return g_ok[dev][which] ? AFFQMM_OK : AFFQMM_E_CUDA;
}

// The kernels' padded head dim: 64 << this.  (e4m3 rows of 64 bytes cannot be
// TMA's destination one by one: pages of one token take the next.)
int which_dim(const affqmm_kv_cache* c) {
    if (c->dim <= 64 && c->type == AFFQMM_KV_E4M3 && c->page == 1) return 1;
    return c->dim <= 64 ? 0 : c->dim <= 128 ? 1 : c->dim <= 256 ? 2 : 3;
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encode_tiled() {
    static EncodeTiledFn fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return (EncodeTiledFn) nullptr;
        return reinterpret_cast<EncodeTiledFn>(f);
    }();
    return fn;
}

// Tensor maps of the pool's K and V: values, then tokens, heads and pages in
// the order of their strides (axis[i] says which is which: 0 token, 1 head, 2
// page), read in boxes of one panel (up to 128 bytes) of the rows that a page
// gives a tile.
int cache_maps(const affqmm_kv_cache* c, int padded, int keys, CUtensorMap* k, CUtensorMap* v, int32_t (&axis)[3]) {
    EncodeTiledFn enc = encode_tiled();
    if (!enc) return AFFQMM_E_CUDA;
    const bool e4m3 = c->type == AFFQMM_KV_E4M3;
    const int es = e4m3 ? 1 : 2, panel = padded * es < 128 ? padded * es : 128;
    const int box = c->page < keys ? c->page : keys;
    const int64_t size[3] = {c->page, c->heads, c->pages};
    const Axes a = axes_of(c);
    cuuint64_t dims[4] = {(cuuint64_t)c->dim}, strides[3];
    cuuint32_t boxes[4] = {(cuuint32_t)(panel / es)}, steps[4] = {1, 1, 1, 1};
    for (int i = 0; i < 3; ++i) {
        axis[i] = a.order[i];
        dims[i + 1] = (cuuint64_t)size[a.order[i]];
        strides[i] = (cuuint64_t)(a.stride[i] * es);
        boxes[i + 1] = a.order[i] == 0 ? (cuuint32_t)box : 1u;
    }
    for (int kv = 0; kv < 2; ++kv)
        if (enc(kv ? v : k, e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, kv ? c->v : c->k, dims,
                strides, boxes, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                panel == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return AFFQMM_E_CUDA;
    return AFFQMM_OK;
}

AttnShape attn_shape(const affqmm_kv_cache* c, int rows, bool lasting, bool pair) {
    const bool e4m3 = c->type == AFFQMM_KV_E4M3;
    switch (which_dim(c)) {
        case 0: return attn_shape_64(e4m3, lasting, pair, rows);
        case 1: return attn_shape_128(e4m3, lasting, pair, rows);
        case 2: return attn_shape_256(e4m3, lasting, pair, rows);
        default: return attn_shape_512(e4m3, lasting, pair, rows);
    }
}

uint32_t reciprocal(int d) { return d > 1 ? (uint32_t)((((uint64_t)1 << 32) + d - 1) / d) : 0u; }

int check_heads(const affqmm_kv_cache* c, int tokens, int heads_q) {
    if (tokens < 1 || tokens > AFFQMM_PAGED_MAX_TOKENS) return AFFQMM_E_ARG;
    if (heads_q < 1 || heads_q > 4096 || heads_q % c->heads) return AFFQMM_E_SHAPE;
    return AFFQMM_OK;
}

// Whether a CTA may take two key heads: their rows of 128 bytes or less lie side by side in the pool, and DRAM reads
// both at once better than either (e4m3, dim 128, 64 requests of up to 16384 keys, pages of 32: 202 -> 168 us; dim 64,
// pages of 64: 173 -> 113).  Not for pages below 32 tokens, whose small boxes want the producers of two CTAs an SM
// (pages of 16: 207 us with one head to a CTA, 262 with two).
bool pairable(const affqmm_kv_cache* c, int rows) {
    const int row_bytes = (64 << which_dim(c)) * (c->type == AFFQMM_KV_E4M3 ? 1 : 2);
    return rows <= 8 && c->heads % 2 == 0 && row_bytes <= 128 && c->page >= 32 && c->head_stride < c->token_stride;
}

// Two partial slots for each CTA that the SMs hold, of whichever kernel a call may take.
size_t attn_workspace(const affqmm_kv_cache* c, int rows, int sms) {
    size_t most = 0;
    for (const bool lasting : {false, true})
        for (const bool pair : {false, true}) {
            if (pair && !(lasting && pairable(c, rows))) continue;
            const AttnShape s = attn_shape(c, rows, lasting, pair);
            const size_t floats = (size_t)2 * s.ctas_per_sm * sms * s.slot_floats;
            if (floats > most) most = floats;
        }
    return kSlotsOffset + most * sizeof(float);
}

// Whether the tables have room for eight tiles of 128 keys to a CTA (two CTAs an SM): only then does a coarser cut
// cost nothing.
bool lasting_tiles(const affqmm_kv_cache* c, int64_t batch, int64_t keys, int sms) {
    return batch * c->heads * ((keys + 127) / 128) >= (int64_t)8 * 2 * sms;
}

// Tiles of all units, with two more for each: keys are counted from a multiple of a tile on, and a unit's end counts
// as one (paged_attn.cuh).
int64_t count_tiles(const AttnShape& s, int64_t batch, int heads, int rows, int64_t keys) {
    return batch * heads * ((rows + s.rows - 1) / s.rows) * ((keys + s.keys - 1) / s.keys + 2);
}

}  // namespace

extern "C" {

int affqmm_paged_plan(int64_t batch, const int32_t* lens, const int32_t* fresh, const uint8_t* finished,
                      int32_t* table, int64_t table_stride, int64_t wide, int32_t* ring, int64_t pool,
                      const int32_t* ring_state, int page, const affqmm_paged_step* step, void* stream) {
    if (!step) return AFFQMM_E_NULL;
    if (batch < 0 || batch > AFFQMM_PAGED_MAX_BATCH) return AFFQMM_E_SHAPE;
    if (wide < 0 || pool < 0 || table_stride < 0 || (batch > 1 && table_stride < wide)) return AFFQMM_E_SHAPE;
    const int shift = page_shift_of(page);
    if (shift < 0) return AFFQMM_E_ARG;
    if (wide * page > kMost || wide > kMost || pool >= kMost || (pool << shift) >= (int64_t)1 << 31)
        return AFFQMM_E_SHAPE;
    if (step->capacity < 0 || step->capacity > kMost) return AFFQMM_E_ARG;
    if (!step->starts || !step->ring_state || !step->status || !ring_state) return AFFQMM_E_NULL;
    if (batch > 0 && (!lens || !fresh || !step->lens)) return AFFQMM_E_NULL;
    if (batch > 0 && wide > 0 && !table) return AFFQMM_E_NULL;
    if (pool > 0 && !ring) return AFFQMM_E_NULL;
    if (step->capacity > 0 && (!step->slots || !step->positions || !step->requests)) return AFFQMM_E_NULL;
    const void* words[] = {lens, fresh, table, ring, ring_state, step->starts, step->lens, step->ring_state, step->status};
    for (const void* w : words)
        if (!aligned(w, 4)) return AFFQMM_E_ALIGN;
    if (!aligned(step->slots, 16) || !aligned(step->positions, 16) || !aligned(step->requests, 16)) return AFFQMM_E_ALIGN;
    if (step->ring_state == ring_state || (batch > 0 && step->lens == lens)) return AFFQMM_E_ARG;
    int sms = 0;
    const int rc = device_sms(&sms);
    if (rc) return rc;
    PlanParams p = {};
    p.lens = lens;
    p.fresh = fresh;
    p.finished = finished;
    p.table = table;
    p.table_stride = table_stride;
    p.ring = ring;
    p.ring_state = ring_state;
    p.batch = (int32_t)batch;
    p.wide = (int32_t)wide;
    p.pool = (int32_t)pool;
    p.page_shift = shift;
    p.capacity = (int32_t)step->capacity;
    p.starts = step->starts;
    p.lens_out = step->lens;
    p.ring_state_out = step->ring_state;
    p.slots = step->slots;
    p.positions = step->positions;
    p.requests = step->requests;
    p.status = step->status;
    return launch_paged_plan(p, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? AFFQMM_OK : AFFQMM_E_CUDA;
}

int affqmm_rope_append(const affqmm_kv_cache* cache, const affqmm_rope* rope, const affqmm_rows* q,
                       const affqmm_rows* k, const affqmm_rows* v, const affqmm_rows* out, int64_t tokens, int heads_q,
                       const int32_t* positions, int64_t position_stride, const int32_t* slots, uint32_t* status,
                       void* stream) {
    int rc = check_cache(cache, true);
    if (rc) return rc;
    if (!rope || !q || !k || !v || !out) return AFFQMM_E_NULL;
    if (rope->rotary < 0 || rope->rotary % 2 || rope->rotary > cache->dim) return AFFQMM_E_SHAPE;
    if ((rope->neighbour != 0 && rope->neighbour != 1) || rope->axes < 1 || rope->axes > 256) return AFFQMM_E_ARG;
    if (tokens < 0 || tokens >= kMost || heads_q < 1 || heads_q > 4096 || position_stride < 0) return AFFQMM_E_SHAPE;
    if (tokens == 0) return AFFQMM_OK;
    if (!positions || !slots || (rope->rotary > 0 && !rope->turns)) return AFFQMM_E_NULL;
    if (!aligned(positions, 4) || !aligned(slots, 4) || !aligned(rope->turns, 8) || !aligned(status, 4))
        return AFFQMM_E_ALIGN;
    for (const affqmm_rows* r : {q, k, v, out})
        if ((rc = check_rows(r->p, r->token_stride, r->head_stride, 0))) return rc;
    if (out->p == q->p && (out->token_stride != q->token_stride || out->head_stride != q->head_stride))
        return AFFQMM_E_ARG;
    int sms = 0;
    rc = device_sms(&sms);
    if (rc) return rc;
    const int es = cache->type == AFFQMM_KV_E4M3 ? 1 : 2;
    RopeParams p = {};
    p.q = q->p, p.q_ts = q->token_stride, p.q_hs = q->head_stride;
    p.k = k->p, p.k_ts = k->token_stride, p.k_hs = k->head_stride;
    p.v = v->p, p.v_ts = v->token_stride, p.v_hs = v->head_stride;
    p.out = out->p, p.o_ts = out->token_stride, p.o_hs = out->head_stride;
    p.positions = positions;
    p.pos_stride = position_stride;
    p.axes = rope->axes;
    p.slots = slots;
    p.turns = reinterpret_cast<const int64_t*>(rope->turns);
    p.axis = rope->axis;
    p.rotary = rope->rotary;
    p.neighbour = rope->neighbour;
    p.tokens = tokens;
    p.heads_q = heads_q;
    p.heads_kv = cache->heads;
    p.dim = cache->dim;
    p.page_shift = page_shift_of(cache->page);
    p.e4m3 = es == 1;
    p.kc = static_cast<uint8_t*>(cache->k);
    p.vc = static_cast<uint8_t*>(cache->v);
    p.page_bytes = cache->page_stride * es;
    p.token_bytes = cache->token_stride * es;
    p.head_bytes = cache->head_stride * es;
    p.pages = cache->pages;
    p.k_scale = cache->k_scale;
    p.v_scale = cache->v_scale;
    p.status = status;
    p.stream = tokens * (heads_q * 2 + (int64_t)cache->heads * 2 * es) * cache->dim > (int64_t)63 << 20;
    return launch_rope_append(p, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? AFFQMM_OK : AFFQMM_E_CUDA;
}

int affqmm_paged_attention_workspace_bytes(const affqmm_kv_cache* cache, int tokens, int heads_q, size_t* bytes) {
    if (!bytes) return AFFQMM_E_NULL;
    int rc = check_cache(cache, false);
    if (rc) return rc;
    if ((rc = check_heads(cache, tokens, heads_q))) return rc;
    int sms = 0;
    if ((rc = device_sms(&sms))) return rc;
    *bytes = attn_workspace(cache, tokens * (heads_q / cache->heads), sms);
    return AFFQMM_OK;
}

int affqmm_paged_attention(const affqmm_kv_cache* cache, const affqmm_lanes* q, const affqmm_lanes* out, float* lse,
                           int64_t batch, int tokens, int heads_q, const int32_t* table, int64_t table_stride,
                           int64_t wide, const int32_t* lens, float scale, int window, uint32_t* status,
                           void* workspace, size_t ws_bytes, void* stream) {
    int rc = check_cache(cache, true);
    if (rc) return rc;
    if ((rc = check_heads(cache, tokens, heads_q))) return rc;
    if (!q || !out) return AFFQMM_E_NULL;
    if (batch < 0 || batch > AFFQMM_PAGED_MAX_BATCH || wide < 0 || table_stride < 0) return AFFQMM_E_SHAPE;
    if (wide * cache->page >= ((int64_t)1 << 31) - 1024 || wide >= kMost) return AFFQMM_E_SHAPE;   // room to count tiles past the end
    if (!std::isfinite(scale) || window < 0) return AFFQMM_E_ARG;
    if (batch == 0) return AFFQMM_OK;
    if (!lens || (wide > 0 && !table)) return AFFQMM_E_NULL;
    if (!aligned(lens, 4) || !aligned(table, 4) || !aligned(lse, 4) || !aligned(status, 4)) return AFFQMM_E_ALIGN;
    for (const affqmm_lanes* r : {q, out})
        if ((rc = check_rows(r->p, r->batch_stride, r->token_stride, r->head_stride))) return rc;
    const int group = heads_q / cache->heads, rows = tokens * group;
    int64_t keys = wide * cache->page;       // that a request can have, and a window sees
    if (window >= keys) window = 0;          // it hides nothing (and the kernel's sums of lengths and windows stay within 32 bits)
    if (window > 0 && keys > (int64_t)window + tokens) keys = (int64_t)window + tokens;
    // so many tiles are always lasting ones
    if (count_tiles(attn_shape(cache, rows, true, false), batch, cache->heads, rows, keys) >= (int64_t)1 << 31) return AFFQMM_E_SHAPE;
    int sms = 0;
    if ((rc = device_sms(&sms))) return rc;
    const bool lasting = lasting_tiles(cache, batch, keys, sms);
    const bool pair = lasting && pairable(cache, rows);
    const AttnShape shape = attn_shape(cache, rows, lasting, pair);
    if (!workspace || ws_bytes < attn_workspace(cache, rows, sms)) return AFFQMM_E_WORKSPACE;
    if (!aligned(workspace, 256)) return AFFQMM_E_ALIGN;
    const int which = which_dim(cache);
    if ((rc = allow_attn(which))) return rc;

    const bool e4m3 = cache->type == AFFQMM_KV_E4M3;
    AttnParams p = {};
    CUtensorMap k_map, v_map;
    int32_t axis[3];
    if ((rc = cache_maps(cache, 64 << which, shape.keys, &k_map, &v_map, axis))) return rc;
    p.axis1 = axis[0], p.axis2 = axis[1], p.axis3 = axis[2];
    p.q = q->p, p.q_bs = q->batch_stride, p.q_ts = q->token_stride, p.q_hs = q->head_stride;
    p.out = out->p, p.o_bs = out->batch_stride, p.o_ts = out->token_stride, p.o_hs = out->head_stride;
    p.lse = lse;
    p.pages = cache->pages;
    p.k_scale = cache->k_scale;
    p.v_scale = cache->v_scale;
    p.table = table;
    p.table_stride = table_stride;
    p.lens = lens;
    p.batch = (int32_t)batch;
    p.tokens = tokens;
    p.heads_q = heads_q;
    p.heads_kv = cache->heads;
    p.group = group;
    p.dim = cache->dim;
    p.wide = (int32_t)wide;
    p.page_shift = page_shift_of(cache->page);
    p.window = window;
    p.row_tiles = (rows + shape.rows - 1) / shape.rows;
    p.m_group = reciprocal(p.group), p.m_row_tiles = reciprocal(p.row_tiles);
    p.scale_log2 = scale * 1.4426950408889634f;
    const int64_t fault = decode_fault_wait();
    p.fault = fault > 0;
    p.wait_limit = fault > 0 ? fault : kWaitLimitCycles;
    p.user_status = status;
    uint8_t* base = static_cast<uint8_t*>(workspace);
    p.status = reinterpret_cast<uint32_t*>(base);
    p.counters = reinterpret_cast<uint32_t*>(base + kStatusBytes);
    p.slots = reinterpret_cast<float*>(base + kSlotsOffset);
    // one CTA for each that the SMs hold, or for each tile that the tables have room for
    const int64_t tiles = count_tiles(shape, batch, cache->heads, rows, keys);
    const int64_t most = (int64_t)sms * shape.ctas_per_sm;
    const int grid = (int)(tiles < most ? tiles : most);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    switch (which) {
        case 0: e = launch_attn_64(e4m3, lasting, pair, rows, p, k_map, v_map, grid, st); break;
        case 1: e = launch_attn_128(e4m3, lasting, pair, rows, p, k_map, v_map, grid, st); break;
        case 2: e = launch_attn_256(e4m3, lasting, pair, rows, p, k_map, v_map, grid, st); break;
        default: e = launch_attn_512(e4m3, lasting, pair, rows, p, k_map, v_map, grid, st); break;
    }
    return e == cudaSuccess ? AFFQMM_OK : AFFQMM_E_CUDA;
}

}  // extern "C"
