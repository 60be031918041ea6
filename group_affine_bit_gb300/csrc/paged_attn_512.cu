// Attention over the paged cache, head dim padded to 512 (paged_attn.cuh).
#include "paged_attn.cuh"

AFFQMM_ATTN_DEFINE(512, 512, false)
