// Attention over a paged cache of f32 rows, keys of width 256 (kernels in gdn_paged_attn.cuh).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#define GDN_PAGED_ATTN_T float
#define GDN_PAGED_ATTN_DK 256
#include "gdn_paged_attn.cuh"
