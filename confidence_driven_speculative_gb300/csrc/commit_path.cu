// commit_path.cu -- the entries of an accepted path move to their places, in
// the caches of all layers.
//
// Position s + j receives what s + path[j] held, path[j] >= j.  So no entry is
// written before the ones in front of it have been read, whichever order
// the path has: place j is the source of places <= j only.  A thread that walks the
// places in ascending order, a batch of loads before the batch's stores,
// needs no barrier.
//
// Bound: bytes, each moved entry read and written once.  256 requests in 16
// layers of 8 heads of 128, 1.9 moves each, 12.8 us (a copy of as many bytes 9.2:
// the moves are pieces of 2 KB, and three trips come first); one request 2.9 in a
// captured graph, a launch and three trips to memory, path to page to entry, and 5.1 to
// 5.8 by plain calls, which the host's part bounds.
#include <algorithm>

#include "cache.cuh"
#include "dspark_internal.cuh"
#include "tcgen05.cuh"

namespace dspark {
namespace {

constexpr int kThreadsCommit = 256;
constexpr int kMoves = 4;  // of each layer, that a thread has asked for before it stores

struct CommitArgs {
    int B, q_max, max_pages, layers, groups, heads, chunks, page_size, num_pages;
    int64_t layer_stride, page_stride, slot_stride, head_stride;
    uint16_t *k, *v;
    const int32_t *block_table, *seq_lens, *path;
};

// A CTA takes one request in kLayers layers.
template <int kLayers>
__global__ void __launch_bounds__(kThreadsCommit, kLayers == 2 ? 5 : 6) commit_path_kernel(const CommitArgs A) {
    __shared__ int64_t from[DSPARK_MAX_STEP_ROWS], to[DSPARK_MAX_STEP_ROWS];
    __shared__ int moves;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int b = blockIdx.x / A.groups, layer0 = (blockIdx.x - b * A.groups) * kLayers, tid = threadIdx.x;
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
    // Many moves go past L2, few do not: see launch_commit_path.
    auto load = [](const uint16_t *p) {
        const uint4 *const x = reinterpret_cast<const uint4 *>(p);
        return kLayers == 2 ? __ldcs(x) : *x;
    };
    auto store = [](uint16_t *p, const uint4 &y) {
        uint4 *const x = reinterpret_cast<uint4 *>(p);
        if (kLayers == 2) __stcs(x, y);
        else *x = y;
    };
    const int n = moves, per = A.heads * A.chunks;
    const bool both = kLayers == 2 && layer0 + 1 < A.layers;
    for (int x = tid; n > 0 && x < 2 * per; x += kThreadsCommit) {
        const int kv = x >= per, in = x - kv * per, head = in / A.chunks;
        uint16_t *const base = (kv ? A.v : A.k) + layer0 * A.layer_stride + head * A.head_stride + (in - head * A.chunks) * 8;
        for (int m0 = 0; m0 < n; m0 += kMoves) {
            uint4 v[kLayers][kMoves];
#pragma unroll
            for (int m = 0; m < kMoves; ++m) {
                if (m0 + m >= n) break;
                const uint16_t *src = base + from[m0 + m];
                v[0][m] = load(src);
                if (kLayers == 2 && both) v[kLayers - 1][m] = load(src + A.layer_stride);
            }
#pragma unroll
            for (int m = 0; m < kMoves; ++m) {
                if (m0 + m >= n) break;
                uint16_t *dst = base + to[m0 + m];
                store(dst, v[0][m]);
                if (kLayers == 2 && both) store(dst + A.layer_stride, v[kLayers - 1][m]);
            }
        }
    }
}

}  // namespace

cudaError_t launch_commit_path(const dspark_cache &c, int B, int q_max, int max_pages, const int32_t *block_table,
                               const int32_t *seq_lens, const int32_t *path, int sms, cudaStream_t s) {
    // Where there are CTAs enough, two layers to one, whose path and pages are looked up once, and the moves go past
    // L2; else a CTA a layer, and moves that stay in L2.  Requests in layers, microseconds of both and (of the two
    // that this rule never takes) of two layers through L2 and one past it: 4 in 32 3.1 against 2.6 (2.7, 3.0), 64 in
    // 32 7.0 against 6.2 (6.5, 6.6), 80 in 32 7.3 against 7.0, 128 in 18 8.0 against 8.4, 160 in 16 8.4 against 9.5, 96
    // in 32 9.4 against 10.6 (10.0, 9.8), 256 in 16 11.4 against 14.7 (13.1, 12.5), 256 in 32 20.5 against 25.8.
    const bool two = int64_t(B) * c.layers > 16 * sms;
    const int groups = two ? (c.layers + 1) / 2 : c.layers;
    const CommitArgs A{B, q_max, max_pages, c.layers, groups, c.Hkv, c.D / 8, c.page_size, c.num_pages,
                       c.layer_stride, c.page_stride, c.slot_stride, c.head_stride,
                       static_cast<uint16_t *>(c.k_cache), static_cast<uint16_t *>(c.v_cache),
                       block_table, seq_lens, path};
    return launch_overlapped(two ? commit_path_kernel<2> : commit_path_kernel<1>, B * groups, kThreadsCommit, 0, s, A);
}

}  // namespace dspark
