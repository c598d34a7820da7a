// step_attention_sinks.cu -- dspark_step_attention_sinks: the kernel of
// step_attention.cuh for windows with sinks.
#include "step_attention.cuh"

namespace dspark {

cudaError_t launch_step_attention_sinks(const dspark_attn &a, int sinks, int sms, uint64_t wait_ns, cudaStream_t s) {
    return launch_rows<kSinks>(a, sinks, sms, wait_ns, s);
}

}  // namespace dspark
