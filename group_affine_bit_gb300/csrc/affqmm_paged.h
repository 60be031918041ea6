// affqmm_paged.h -- host-side declarations shared by the paged cache's
// translation units (not part of the public ABI).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "affqmm.h"

namespace affqmm {

// Between which the scale of a block lies, so that 2^(score + log2 of V's scale) and one over that scale stay within
// fp32 whatever the blocks that a row sees.
constexpr float kLeastScale = 0x1p-48f, kMostScale = 0x1p48f;

// ---- paged_plan.cu
struct PlanParams {
    const int32_t* lens;
    const int32_t* fresh;        // new tokens of each request
    const uint8_t* finished;     // or null
    int32_t* table;
    int64_t table_stride;
    int32_t* ring;
    const int32_t* ring_state;   // {head, count}
    int32_t batch, wide, pool, page_shift, capacity;
    int32_t *starts, *lens_out, *ring_state_out, *slots, *positions, *requests, *status;
};
cudaError_t launch_paged_plan(const PlanParams& p, int sms, cudaStream_t st);

// ---- rope_append.cu
struct RopeParams {
    const uint16_t *q, *k, *v;
    int64_t q_ts, q_hs, k_ts, k_hs, v_ts, v_hs, o_ts, o_hs;   // token and head strides, elements
    uint16_t* out;
    const int32_t* positions;
    int64_t pos_stride;          // between axes
    int32_t axes;
    const int32_t* slots;
    const int64_t* turns;        // [rotary / 2]
    const uint8_t* axis;         // [rotary / 2] or null
    int32_t rotary, neighbour;
    int64_t tokens;
    int32_t heads_q, heads_kv, dim, page_shift, e4m3;
    uint8_t *kc, *vc;
    int64_t page_bytes, token_bytes, head_bytes, pages;
    const float *k_scale, *v_scale;
    uint32_t* status;
    int32_t stream;              // more is written than L2 keeps
};
cudaError_t launch_rope_append(const RopeParams& p, int sms, cudaStream_t st);

// ---- block_append.cu
struct BlockParams {
    RopeParams rope;             // e4m3: the codes' type, else int8; no scales of heads
    float *k_scales, *v_scales;
    int64_t s_ps, s_bs, s_hs;    // page, block and head strides of the two, elements
    int32_t block_shift;
};
cudaError_t launch_block_append(const BlockParams& p, int sms, cudaStream_t st);

// ---- paged_read.cu
enum { READ_BF16, READ_E4M3, READ_E4M3_BLOCKS, READ_I8_BLOCKS };
struct ReadParams {
    const uint8_t *kc, *vc;
    int64_t page_bytes, token_bytes, head_bytes, pages;
    const float *k_scale, *v_scale;     // of heads, or null; or of blocks and heads
    int64_t s_ps, s_bs, s_hs;
    int32_t block_shift, page_shift, heads, dim;
    uint16_t *k, *v;
    int64_t k_ts, k_hs, v_ts, v_hs;
    int64_t rows;
    int32_t batch, wide;
    const int32_t* table;
    int64_t table_stride;
    const int32_t *starts, *first;
    uint32_t* status;
};
cudaError_t launch_paged_read(const ReadParams& p, int kind, int sms, cudaStream_t st);

// ---- paged_attn_*.cu (paged_attn.cuh)
struct AttnParams {
    const uint16_t* q;
    uint16_t* out;
    float* lse;                  // [batch, tokens, heads_q] or null
    int64_t q_bs, q_ts, q_hs, o_bs, o_ts, o_hs;   // elements
    int64_t pages;
    int32_t axis1, axis2, axis3; // what the cache's tensor maps have as axes 1 .. 3: 0 token, 1 head, 2 page
    const float *k_scale, *v_scale;     // of each head, or null
    const float *k_scales, *v_scales;   // of each block of tokens and head
    int32_t s_ps, s_bs, s_hs;           // page, block and head strides of the two, elements
    int32_t block_shift;
    int32_t s_pairs;                    // the scales of heads 2i and 2i + 1 lie side by side, eight bytes on their boundary
    const int32_t* table;
    int64_t table_stride;
    const int32_t* lens;
    int32_t batch, tokens, heads_q, heads_kv, group, dim, wide, page_shift;
    int32_t window;              // 0, or less than wide << page_shift (which is below 2^31 - 1024)
    int32_t row_tiles;           // tiles of 8 NT (token, head) rows
    uint32_t m_group, m_row_tiles;   // ceil(2^32 / d) of the two
    float scale_log2;            // softmax scale times log2(e)
    int64_t wait_limit;          // cycles after which a wait gives up
    int32_t fault;               // test hook: the consumers wait on a barrier that nothing completes
    uint32_t* user_status;       // or null
    uint32_t* status;            // workspace: status word, merge counters, partial slots
    uint32_t* counters;
    float* slots;
};

// A launch's shape: how many CTAs an SM holds and the floats of one partial slot.
struct AttnShape {
    int ctas_per_sm = 0;
    int rows = 0;                // rows of a tile (8 NT)
    int keys = 0;                // and its keys
    size_t slot_floats = 0;
};
// NAME: head dim padded to 64, 128, 256 or 512, of a cache with scales for each block after `blocks_`; bytes: e4m3 rather than
// bf16, with blocks int8 rather than e4m3; rows: (token, head) rows that share a key head; lasting: the tables have room for
// many tiles; pair: two key heads to a CTA.
#define AFFQMM_ATTN_DECL(NAME)                                                                          \
    AttnShape attn_shape_##NAME(bool bytes, bool lasting, bool pair, int rows);                         \
    cudaError_t attn_allow_smem_##NAME();                                                               \
    cudaError_t launch_attn_##NAME(bool bytes, bool lasting, bool pair, int rows, const AttnParams& p, const CUtensorMap& k, \
                                   const CUtensorMap& v, int grid, cudaStream_t st);
AFFQMM_ATTN_DECL(64)
AFFQMM_ATTN_DECL(128)
AFFQMM_ATTN_DECL(256)
AFFQMM_ATTN_DECL(512)
AFFQMM_ATTN_DECL(blocks_64)
AFFQMM_ATTN_DECL(blocks_128)
AFFQMM_ATTN_DECL(blocks_256)
AFFQMM_ATTN_DECL(blocks_512)
#undef AFFQMM_ATTN_DECL

// affqmm_api.cu: the current device's SM count (AFFQMM_E_DEVICE where it is no sm_103 GPU).
int device_sms(int* sms);

}  // namespace affqmm
