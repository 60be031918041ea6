// Attention over the paged cache with a scale for each block of tokens and head, head dim padded to 128 (paged_attn.cuh).
#include "paged_attn.cuh"

AFFQMM_ATTN_DEFINE(128, blocks_128, true)
