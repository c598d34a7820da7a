// prompt_attention_sinks.cu -- dspark_prompt_attention_sinks: the kernel of
// prompt_attention.cuh for windows with sinks.
#include "prompt_attention.cuh"

namespace dspark {

cudaError_t launch_prompt_attention_sinks(const dspark_attn &a, int sinks, int sms, uint64_t wait_ns, cudaStream_t s) {
    return launch_prompts<kSinks>(a, sinks, sms, wait_ns, s);
}

}  // namespace dspark
