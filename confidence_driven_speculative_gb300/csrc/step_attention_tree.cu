// step_attention_tree.cu -- dspark_step_attention_tree: for few columns the
// kernel of step_attention.cuh, else that of tree_attention.cu.
#include "step_attention.cuh"

namespace dspark {

// Columns of a unit (rows of the longest tree times query heads of a cached head) up to which the keys are
// the tensor core's M side.  8 cached heads of 128, 4 query heads each: one request of 4095 keys with 4, 8 and 16
// rows 15.1, 18.9 and 28.1 us, with the queries there 18.9, 19.2 and 21.1; 32 of 2048 keys with 8, 16 and 32 rows
// 57, 61 and 82 us against 60, 64 and 74.
constexpr int kFewColumns = 48;

cudaError_t launch_step_attention_tree(const dspark_attn &a, const uint64_t *row_seen, int sinks, int sms,
                                       uint64_t wait_ns, cudaStream_t s) {
    if (a.q_max * (a.Hq / a.Hkv) > kFewColumns) return launch_tree_attention(a, row_seen, sinks, sms, wait_ns, s);
    return launch_rows<kTree>(a, row_seen, sinks, sms, wait_ns, s);
}

}  // namespace dspark
