// attn_paged.cuh -- the two paths of the paged block attention.
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>

#include "orthrus_paged.h"

namespace orthrus {

// bf16, tensor cores (attn_paged.cu)
size_t paged_tc_workspace(const orthrus_paged_attn_args& a);
int paged_tc_launch(const orthrus_paged_attn_args& a, cudaStream_t st);
// fp32, CUDA cores (attn_paged_f32.cu)
size_t paged_f32_workspace(const orthrus_paged_attn_args& a);
int paged_f32_launch(const orthrus_paged_attn_args& a, cudaStream_t st);

}  // namespace orthrus
