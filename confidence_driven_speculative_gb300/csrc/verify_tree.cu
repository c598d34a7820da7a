// verify_tree.cu -- the walk that the target goes down a drafted tree.
//
// y_j = argmax of the target's row j, the lowest id on ties; the walk goes on
// to the lowest child whose token is y of the present row.  Only the rows of the
// walk are needed, so they are read one after the other, as the walk comes to
// them.
//
// Bound: bytes of the walks' rows, or the latency of one row after the other.
#include "cache.cuh"
#include "dspark_internal.cuh"
#include "tcgen05.cuh"

namespace dspark {
namespace {

constexpr int kThreadsTree = 1024;

struct TreeArgs {
    int B, rows, q_max, V;
    const void *logits;
    const int32_t *row_off, *parent, *ids;
    int32_t *accept_len, *num_emitted, *path, *out_tokens, *commit;
};

// A CTA walks one request's tree.
template <typename T>
__global__ void __launch_bounds__(kThreadsTree) verify_tree_kernel(const TreeArgs A) {
    constexpr int E = Vec<T>::kElems;
    __shared__ float best_v[32];
    __shared__ int best_i[32], next, token;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int row0 = min(max(A.row_off[b], 0), A.rows);
    const int n = min(min(max(A.row_off[b + 1], row0), A.rows) - row0, A.q_max);
    int32_t *const path = A.path + int64_t(b) * A.q_max, *const out = A.out_tokens + int64_t(b) * A.q_max;
    int at = n > 0 ? 0 : -1, len = 0;
    while (at >= 0) {
        const uint4 *row = reinterpret_cast<const uint4 *>(static_cast<const T *>(A.logits) + int64_t(row0 + at) * A.V);
        float v = -INFINITY;
        int i = 0x7fffffff;
        for (int c = tid; c < A.V / E; c += kThreadsTree) {
            float x[E];
            Vec<T>::unpack(row[c], x);
#pragma unroll
            for (int e = 0; e < E; ++e) am_combine(v, i, x[e], c * E + e);
        }
        warp_am_reduce(v, i);
        if (lane == 0) {
            best_v[warp] = v;
            best_i[warp] = i;
        }
        __syncthreads();
        if (warp == 0) {
            v = best_v[lane];
            i = best_i[lane];
            warp_am_reduce(v, i);
            // the lowest child with that token
            int child = -1;
            for (int j0 = at + 1; j0 < n && child < 0; j0 += 32) {
                const int j = j0 + lane;
                const uint32_t hit = __ballot_sync(
                    0xffffffffu, j < n && A.parent[row0 + j] == at && A.ids[row0 + j] == i);
                if (hit) child = j0 + __ffs(hit) - 1;
            }
            if (lane == 0) {
                path[len] = at;
                out[len] = i;
                next = child;
            }
        }
        __syncthreads();
        at = next;
        ++len;
    }
    for (int j = len + tid; j < A.q_max; j += kThreadsTree) path[j] = out[j] = -1;
    if (tid == 0) {
        A.accept_len[b] = max(len - 1, 0);
        A.num_emitted[b] = len;
        if (A.commit) A.commit[b] += len;
    }
}

}  // namespace

size_t tree_workspace_bytes(int, int, int) { return 256; }

cudaError_t launch_verify_tree(const dspark_tree &t, int, cudaStream_t s) {
    const TreeArgs A{t.B, t.rows, t.q_max, t.V, t.target_logits, t.row_off, t.parent, t.packed_ids,
                     t.accept_len, t.num_emitted, t.path, t.out_tokens, t.seq_lens_commit};
    return t.logit_dtype == DSPARK_BF16 ? launch_overlapped(verify_tree_kernel<uint16_t>, t.B, kThreadsTree, 0, s, A)
                                        : launch_overlapped(verify_tree_kernel<float>, t.B, kThreadsTree, 0, s, A);
}

}  // namespace dspark
