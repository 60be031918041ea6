// Attention over the paged cache, head dim padded to 64 (paged_attn.cuh).
#include "paged_attn.cuh"

AFFQMM_ATTN_DEFINE(64, 64, false)
