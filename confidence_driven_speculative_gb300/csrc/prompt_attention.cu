// prompt_attention.cu -- dspark_prompt_attention: the kernel of
// prompt_attention.cuh, causal or with a window.
#include "prompt_attention.cuh"

namespace dspark {

cudaError_t launch_prompt_attention(const dspark_attn &a, int sms, uint64_t wait_ns, cudaStream_t s) {
    return a.window > 0 ? launch_prompts<kWindow>(a, 0, sms, wait_ns, s) : launch_prompts<kCausal>(a, 0, sms, wait_ns, s);
}

}  // namespace dspark
