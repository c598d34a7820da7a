// prompt_attention.cu -- whole prompts, causal, packed one after the other.
//
// One warp per (row, query head): an online softmax over the row's keys.
#include "attn.cuh"
#include "dspark_internal.cuh"

namespace dspark {
namespace {

template <int D>
__global__ void __launch_bounds__(128) prompt_attention_kernel(const dspark_attn A) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int h = int(w % A.Hq);
    const int64_t r = w / A.Hq;
    if (r >= A.rows) return;
    int lo = 0, hi = A.B;  // the request of row r
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (A.row_off[mid] <= r) lo = mid; else hi = mid;
    }
    const int r0 = A.row_off[lo];
    if (r < r0 || r >= A.row_off[lo + 1] || r - r0 >= A.q_max) return;
    const int kvh = h / (A.Hq / A.Hkv);
    const uint16_t *q = static_cast<const uint16_t *>(A.q_rot) + (r * A.Hq + h) * D + lane * E;
    float x[E], o[E];
    for (int e = 0; e < E; ++e) { x[e] = bf16_lo(q[e]); o[e] = 0.f; }
    const float sc = A.scale * 1.4426950408889634f;
    float m = -INFINITY, l = 0.f;
    const int64_t first = A.window > 0 ? max((int64_t)r0, r - A.window + 1) : r0;
    for (int64_t k = first; k <= r; ++k) {
        const uint16_t *kp = static_cast<const uint16_t *>(A.k_rot) + (k * A.Hkv + kvh) * D + lane * E;
        const uint16_t *vp = static_cast<const uint16_t *>(A.v) + k * A.v_stride + kvh * D + lane * E;
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
    uint16_t *out = static_cast<uint16_t *>(A.out) + (r * A.Hq + h) * D + lane * E;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    for (int e = 0; e < E; ++e) {
        uint32_t y;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(y) : "f"(0.f), "f"(o[e] * inv));
        out[e] = uint16_t(y);
    }
}

}  // namespace

cudaError_t launch_prompt_attention(const dspark_attn &a, int sms, uint64_t wait_ns, cudaStream_t s) {
    (void)sms; (void)wait_ns;
    const int64_t warps = (int64_t)a.rows * a.Hq;
    const unsigned grid = unsigned((warps + 3) / 4);
    if (a.D == 128) prompt_attention_kernel<128><<<grid, 128, 0, s>>>(a);
    else prompt_attention_kernel<64><<<grid, 128, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace dspark
