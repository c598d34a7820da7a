// attn.cuh -- launch interfaces of the attention calls (rope_append.cu,
// step_attention.cu, prompt_attention.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "dspark.h"

namespace dspark {

constexpr int kAttnMaxCtas = 160;  // CTAs of an attention launch (152 SMs)

// Workspace of the attention calls: word 0 is the device status.
size_t attn_workspace_bytes(int Hq, int Hkv, int D, int q_max);

// Can the cache be copied key by key (pages of no multiple of 8 positions)?
bool step_strides_ok(const dspark_attn &a);

// Is the list of a step's tiles counted in 32 bits?
bool step_list_fits(const dspark_attn &a);

cudaError_t launch_rope_append(const dspark_attn &a, int sms, cudaStream_t s);
cudaError_t launch_step_attention(const dspark_attn &a, int sms, uint64_t wait_ns, cudaStream_t s);
cudaError_t launch_prompt_attention(const dspark_attn &a, int sms, uint64_t wait_ns, cudaStream_t s);

}  // namespace dspark
