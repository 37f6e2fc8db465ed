// Attention over a paged cache of bf16 rows, keys of width 128 (kernels in gdn_paged_attn.cuh).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#define GDN_PAGED_ATTN_T __nv_bfloat16
#define GDN_PAGED_ATTN_DK 128
#include "gdn_paged_attn.cuh"
