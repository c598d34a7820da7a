// step_attention.cu -- the step's rows over the paged cache.
//
// One warp per (row, query head): an online softmax over the row's keys.
#include "attn.cuh"
#include "dspark_internal.cuh"

namespace dspark {
namespace {

template <int D>
__global__ void __launch_bounds__(128) step_attention_kernel(const dspark_attn A) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int h = int(w % A.Hq);
    const int j = int(w / A.Hq % A.q_max);
    const int64_t b = w / A.Hq / A.q_max;
    if (b >= A.B) return;
    const int r = A.row_off[b] + j;
    if (r >= A.row_off[b + 1] || r < 0 || r >= A.rows) return;
    const int pos = (A.seq_lens ? A.seq_lens[b] : 0) + j;
    const int kvh = h / (A.Hq / A.Hkv);
    const uint16_t *q = static_cast<const uint16_t *>(A.q_rot) + ((int64_t)r * A.Hq + h) * D + lane * E;
    float x[E], o[E];
    for (int e = 0; e < E; ++e) { x[e] = bf16_lo(q[e]); o[e] = 0.f; }
    const float sc = A.scale * 1.4426950408889634f;
    float m = -INFINITY, l = 0.f;
    const int first = A.window > 0 ? max(0, pos - A.window + 1) : 0;
    for (int k = first; k <= pos; ++k) {
        const int pi = k / A.page_size;
        if (pi >= A.max_pages) break;
        const int page = A.block_table[b * A.max_pages + pi];
        if (page < 0 || page >= A.num_pages) continue;
        const int64_t at = page * A.page_stride + (k % A.page_size) * A.slot_stride + kvh * A.head_stride + lane * E;
        const uint16_t *kp = static_cast<const uint16_t *>(A.k_cache) + at;
        const uint16_t *vp = static_cast<const uint16_t *>(A.v_cache) + at;
        float d = 0.f;
        for (int e = 0; e < E; ++e) d += x[e] * bf16_lo(kp[e]);
        d = warp_sum(d) * sc;
        const float mn = fmaxf(m, d);
        const float f = mn == -INFINITY ? 1.f : exp2_approx(m - mn);
        const float p = mn == -INFINITY ? 0.f : exp2_approx(d - mn);
        l = l * f + p;
        for (int e = 0; e < E; ++e) o[e] = o[e] * f + p * bf16_lo(vp[e]);
        m = mn;
    }
    uint16_t *out = static_cast<uint16_t *>(A.out) + ((int64_t)r * A.Hq + h) * D + lane * E;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    for (int e = 0; e < E; ++e) {
        uint32_t y;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(y) : "f"(0.f), "f"(o[e] * inv));
        out[e] = uint16_t(y);
    }
}

}  // namespace

size_t attn_workspace_bytes() { return 256; }

cudaError_t launch_step_attention(const dspark_attn &a, int sms, uint64_t wait_ns, cudaStream_t s) {
    (void)sms; (void)wait_ns;
    const int64_t warps = (int64_t)a.B * a.q_max * a.Hq;
    const unsigned grid = unsigned((warps + 3) / 4);
    if (a.D == 128) step_attention_kernel<128><<<grid, 128, 0, s>>>(a);
    else step_attention_kernel<64><<<grid, 128, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace dspark
