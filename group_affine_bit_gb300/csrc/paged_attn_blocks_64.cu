// Attention over the paged cache with a scale for each block of tokens and head, head dim padded to 64 (paged_attn.cuh).
#include "paged_attn.cuh"

AFFQMM_ATTN_DEFINE(64, blocks_64, true)
