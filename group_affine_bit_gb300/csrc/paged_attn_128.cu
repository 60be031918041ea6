// Attention over the paged cache, head dim padded to 128 (paged_attn.cuh).
#include "paged_attn.cuh"

AFFQMM_ATTN_DEFINE(128, 128, false)
