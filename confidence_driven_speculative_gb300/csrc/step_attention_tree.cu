// step_attention_tree.cu -- dspark_step_attention_tree: the kernel of
// step_attention.cuh for drafted trees.
#include "step_attention.cuh"

namespace dspark {

cudaError_t launch_step_attention_tree(const dspark_attn &a, const uint64_t *row_seen, int sinks, int sms,
                                       uint64_t wait_ns, cudaStream_t s) {
    return launch_rows<kTree>(a, row_seen, sinks, sms, wait_ns, s);
}

}  // namespace dspark
