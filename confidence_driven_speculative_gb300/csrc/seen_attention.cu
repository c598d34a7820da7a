// seen_attention.cu -- attention of rows that do not see every key before
// them: drafted trees, and windows with sinks, over the paged cache or packed
// prompts.
//
// One CTA for each row and query head walks the keys in blocks of 128 with
// a running maximum m, l = sum 2^(s - m) and o = sum 2^(s - m) v.
#include <algorithm>

#include "attn.cuh"
#include "dspark_internal.cuh"
#include "tcgen05.cuh"

namespace dspark {
namespace {

constexpr int kBlock = 128;

struct SeenArgs {
    int B, rows, q_max, Hq, Hkv, G, D, page_size, num_pages, max_pages, window, sinks;
    float scale2;
    int64_t k_row, v_row, page_stride, slot_stride, head_stride;
    const uint16_t *q, *k, *v;   // paged: the caches; else packed rows
    const int32_t *row_off, *seq_lens, *block_table, *packed_pos;
    const uint64_t *row_seen;
    uint16_t *out;
    int paged;
};

__global__ void __launch_bounds__(kBlock) seen_attention_kernel(const SeenArgs A) {
    __shared__ float q[128], p[kBlock], red[kBlock / 32];
    __shared__ int64_t at[kBlock];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tid = threadIdx.x, r = blockIdx.x / A.Hq, h = blockIdx.x - r * A.Hq;
    int b = 0;
    {   // the request that owns the row
        int lo = 0, hi = A.B;
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (A.row_off[mid] <= r) lo = mid; else hi = mid;
        }
        b = lo;
    }
    const int row0 = max(A.row_off[b], 0), n = min(min(A.row_off[b + 1], A.rows) - row0, A.q_max), j = r - row0;
    if (j < 0 || j >= n) return;
    const int start = A.paged && A.seq_lens ? min(max(A.seq_lens[b], 0), INT32_MAX - 65536) : 0;
    int pos = start + j, end = pos + 1;
    if (A.row_seen) {
        end = start + n;
        pos = A.window ? max(A.packed_pos[r], start) : start;
    }
    if (A.paged) end = min(end, A.max_pages * A.page_size);
    const uint64_t seen = A.row_seen ? A.row_seen[r] : 0;
    for (int d = tid; d < A.D; d += kBlock) q[d] = bf16_lo(A.q[(int64_t(r) * A.Hq + h) * A.D + d]);
    float m = -INFINITY, l = 0.f, o = 0.f;
    for (int k0 = 0; k0 < end; k0 += kBlock) {
        const int t = k0 + tid;
        bool here = t < end;
        if (A.row_seen && t >= start) here = here && (seen >> (t - start)) & 1;
        else here = here && (A.window == 0 || t > pos - A.window || t < A.sinks);
        int64_t entry = -1;
        if (here && A.paged) {
            const int page = A.block_table[int64_t(b) * A.max_pages + t / A.page_size];
            if (page >= 0 && page < A.num_pages)
                entry = page * A.page_stride + (t % A.page_size) * A.slot_stride + (h / A.G) * A.head_stride;
        } else if (here) {
            entry = int64_t(row0 + t);
        }
        __syncthreads();
        float s = -INFINITY;
        if (entry >= 0) {
            const uint16_t *k = A.paged ? A.k + entry : A.k + entry * A.k_row + (h / A.G) * A.D;
            s = 0.f;
            for (int d = 0; d < A.D; d += 8) {
                float x[8];
                Vec<uint16_t>::unpack(*reinterpret_cast<const uint4 *>(k + d), x);
#pragma unroll
                for (int e = 0; e < 8; ++e) s = fmaf(q[d + e], x[e], s);
            }
        }
        at[tid] = entry;
        float top = s;
#pragma unroll
        for (int w = 16; w > 0; w >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
        if ((tid & 31) == 0) red[tid >> 5] = top;
        __syncthreads();
        const float now = fmaxf(m, fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
        const float f = m == -INFINITY ? 0.f : exp2f((m - now) * A.scale2);
        p[tid] = s == -INFINITY ? 0.f : exp2f((s - now) * A.scale2);
        m = now;
        __syncthreads();
        l *= f;
        o *= f;
        for (int i = 0; i < kBlock; ++i) {
            if (at[i] < 0) continue;
            l += p[i];
            if (tid < A.D)
                o = fmaf(p[i], bf16_lo(A.paged ? A.v[at[i] + tid] : A.v[at[i] * A.v_row + (h / A.G) * A.D + tid]), o);
        }
    }
    if (tid < A.D) A.out[(int64_t(r) * A.Hq + h) * A.D + tid] = uint16_t(pack_bf16x2(l == 0.f ? 0.f : o / l, 0.f));
}

}  // namespace

cudaError_t launch_seen_attention(const dspark_attn &a, const uint64_t *row_seen, int sinks, bool paged,
                                  cudaStream_t s) {
    SeenArgs A{a.B, a.rows, a.q_max, a.Hq, a.Hkv, a.Hq / a.Hkv, a.D, a.page_size, a.num_pages, a.max_pages,
               a.window, sinks, float(double(a.scale) * 1.4426950408889634), int64_t(a.Hkv) * a.D, a.v_stride,
               a.page_stride, a.slot_stride, a.head_stride, static_cast<const uint16_t *>(a.q_rot),
               static_cast<const uint16_t *>(paged ? a.k_cache : a.k_rot),
               static_cast<const uint16_t *>(paged ? a.v_cache : a.v), a.row_off, a.seq_lens, a.block_table,
               a.packed_pos, row_seen, static_cast<uint16_t *>(a.out), paged};
    return launch_overlapped(seen_attention_kernel, a.rows * a.Hq, kBlock, 0, s, A);
}

}  // namespace dspark
