// step_attention.cu -- dspark_step_attention: the kernel of step_attention.cuh
// for chains, and the limits of all its callers.
#include "step_attention.cuh"

namespace dspark {

size_t attn_workspace_bytes(int Hq, int Hkv, int D, int q_max) {
    if (q_max > DSPARK_MAX_STEP_ROWS) return kHeaderBytes;  // dspark_prompt_attention's
    const size_t cols = size_t(step_columns(Hq, Hkv, q_max));
    return kHeaderBytes + align256(2 * kAttnMaxCtas * cols * D * sizeof(float)) +
           align256(2 * kAttnMaxCtas * 2 * cols * sizeof(float));
}

bool step_strides_ok(const dspark_attn &a) {
    int64_t row, page_rows, head_rows, head_x;
    return gcd(a.page_size, kTile) >= 8 || step_gather_rows(a, &row, &page_rows, &head_rows, &head_x);
}

bool step_list_fits(const dspark_attn &a) {
    const long long blocks = (a.q_max + step_rows(a.Hq, a.Hkv, a.q_max) - 1) / step_rows(a.Hq, a.Hkv, a.q_max) + 1;
    const long long places = (long long)a.max_pages * a.page_size / kTile + 2 + kUnitCost;
    return places * blocks * a.Hkv <= INT32_MAX / a.B;
}

cudaError_t launch_step_attention(const dspark_attn &a, int sms, uint64_t wait_ns, cudaStream_t s) {
    return launch_rows<kChain>(a, 0, sms, wait_ns, s);
}

}  // namespace dspark
