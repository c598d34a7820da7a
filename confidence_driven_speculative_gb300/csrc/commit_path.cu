// commit_path.cu -- the entries of an accepted path move to their places, in
// the caches of all layers.
//
// Position s + j receives what s + path[j] held, path[j] >= j.  So no entry is
// written before the ones in front of it have been read, whichever order
// the path has: place j is the source of places <= j only.  A thread that walks the
// places in ascending order, a batch of loads before the batch's stores,
// needs no barrier.
//
// Bound: bytes, each moved entry read and written once.
#include <algorithm>

#include "cache.cuh"
#include "dspark_internal.cuh"
#include "tcgen05.cuh"

namespace dspark {
namespace {

constexpr int kThreadsCommit = 256;
constexpr int kInFlight = 8;  // entries that a thread has asked for before it stores

struct CommitArgs {
    int B, q_max, max_pages, layers, group, groups, heads, chunks, page_size, num_pages;
    int64_t layer_stride, page_stride, slot_stride, head_stride;
    uint16_t *k, *v;
    const int32_t *block_table, *seq_lens, *path;
};

// A CTA takes one request in a group of layers.
__global__ void __launch_bounds__(kThreadsCommit) commit_path_kernel(const CommitArgs A) {
    __shared__ int64_t from[DSPARK_MAX_STEP_ROWS], to[DSPARK_MAX_STEP_ROWS];
    __shared__ int moves;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int b = blockIdx.x / A.groups, layer0 = (blockIdx.x - b * A.groups) * A.group, tid = threadIdx.x;
    if (tid < 32) {
        // the moves, in ascending places
        const int32_t *path = A.path + int64_t(b) * A.q_max, *table = A.block_table + int64_t(b) * A.max_pages;
        const int64_t start = A.seq_lens ? max(A.seq_lens[b], 0) : 0;
        auto entry = [&](int64_t pos) -> int64_t {
            const int64_t i = pos < INT32_MAX ? int64_t(uint32_t(pos) / uint32_t(A.page_size)) : A.max_pages;
            if (i >= A.max_pages) return -1;
            const int page = table[i];
            if (page < 0 || page >= A.num_pages) return -1;
            return page * A.page_stride + (pos - i * A.page_size) * A.slot_stride;
        };
        int n = 0;
        bool ended = false;
        for (int j0 = 0; j0 < A.q_max && !ended; j0 += 32) {
            const int j = j0 + tid, x = j < A.q_max ? path[j] : -1;
            const uint32_t stop = __ballot_sync(0xffffffffu, x < 0);
            const bool before = !(stop & ((2u << tid) - 1u));  // no negative one up to here
            int64_t src = -1, dst = -1;
            if (before && x > j) {
                src = entry(start + x);
                dst = entry(start + j);
            }
            const uint32_t go = __ballot_sync(0xffffffffu, src >= 0 && dst >= 0);
            if (src >= 0 && dst >= 0) {
                const int at = n + __popc(go & ((1u << tid) - 1u));
                from[at] = src;
                to[at] = dst;
            }
            n += __popc(go);
            ended = stop != 0;
        }
        if (tid == 0) moves = n;
    }
    __syncthreads();
    const int n = moves, per = A.heads * A.chunks, all = n * min(A.group, A.layers - layer0);
    if (n == 0) return;
    for (int x = tid; x < 2 * per; x += kThreadsCommit) {
        const int kv = x >= per, in = x - kv * per, head = in / A.chunks;
        uint16_t *const base = (kv ? A.v : A.k) + layer0 * A.layer_stride + head * A.head_stride + (in - head * A.chunks) * 8;
        // all moves of all layers of the group, layer by layer
        int64_t next = 0;  // the layer of the next move, and the move
        for (int m0 = 0, i = 0; m0 < all; m0 += kInFlight) {
            uint4 v[kInFlight];
            int64_t layer = next;
            int at = i;
#pragma unroll
            for (int m = 0; m < kInFlight; ++m) {
                if (m0 + m < all) v[m] = *reinterpret_cast<const uint4 *>(base + next + from[i]);
                if (++i == n) {
                    i = 0;
                    next += A.layer_stride;
                }
            }
#pragma unroll
            for (int m = 0; m < kInFlight; ++m) {
                if (m0 + m < all) *reinterpret_cast<uint4 *>(base + layer + to[at]) = v[m];
                if (++at == n) {
                    at = 0;
                    layer += A.layer_stride;
                }
            }
        }
    }
}

}  // namespace

cudaError_t launch_commit_path(const dspark_cache &c, int B, int q_max, int max_pages, const int32_t *block_table,
                               const int32_t *seq_lens, const int32_t *path, int sms, cudaStream_t s) {
    // As many layers to a CTA as let all CTAs run at once: their path and pages are looked up once.
    const int group = std::max(1, std::min<int>(c.layers, int64_t(B) * c.layers / (8 * sms)));
    const int groups = (c.layers + group - 1) / group;
    const CommitArgs A{B, q_max, max_pages, c.layers, group, groups, c.Hkv, c.D / 8, c.page_size, c.num_pages,
                       c.layer_stride, c.page_stride, c.slot_stride, c.head_stride,
                       static_cast<uint16_t *>(c.k_cache), static_cast<uint16_t *>(c.v_cache),
                       block_table, seq_lens, path};
    return launch_overlapped(commit_path_kernel, B * groups, kThreadsCommit, 0, s, A);
}

}  // namespace dspark
