// verify_tree.cu -- the walk that the target goes down a drafted tree.
//
// y_j = argmax of the target's row j, the lowest id on ties; the walk goes on
// to the lowest child whose token is y of the present row.  Maxima are taken
// over 64-bit keys, the logit in an order-preserving form above the
// complement of its id, so that the largest key is the lowest id of the
// largest logit, whatever the order of the comparisons.
//
// Only the walk's own rows are needed, and a walk seldom goes far, so
// verify_tree_kernel reads one row after the other: a cluster of CTAs shares the
// present row, each warp hands its key to every CTA of the cluster, and one
// cluster barrier later all know the next row.  Bound: bytes of the walks'
// rows while many walk, later the latency of a level (a load, a reduction, a
// barrier).  Clusters are as large as still lets all requests walk at once.  So
// late a level takes 1.4 us however short its row, and what a cluster has in
// flight at once counts: most loads go through shared memory (cp.async), each to
// a place that only its own thread reads, and leave the registers to more CTAs
// (seven an SM with 4 + 12 loads a thread; 16 to registers in four 28.0 us against
// 22.9 to 24.7 for 128 requests of 129280 ids, 77.5 against 57.8 for 400, 17.2 against
// 18.5 for 64; the walks' own rows take 11.4 at a copy's rate).
//
// Few rows are read all at once (verify_tree_all_kernel): every CTA
// takes a part of a row and merges its key by atomicMax, and the one that
// finishes a request's last part walks in registers.  Reading more than needed
// costs less than waiting once per level: one tree of 32 rows and 129280 ids
// takes 4.9 us.
#include <algorithm>

#include "cache.cuh"
#include "dspark_internal.cuh"
#include "tcgen05.cuh"

namespace dspark {
namespace {

constexpr int kThreadsAll = 256;    // verify_tree_all_kernel
constexpr int kThreadsWalk = 128;   // verify_tree_kernel
constexpr int kResident = 7;        // its CTAs of an SM
constexpr int kMaxCluster = 16;
// Bytes of all rows up to which they are read at once: 64 rows of 129280 ids, 16.5 MB, 5.5 us (one after the other,
// seven in a row accepted, 6.0), 2 x 40 rows, 20.7 MB, 6.9 (6.0).
constexpr size_t kAllBytes = size_t(18) << 20;
constexpr int kAllRequests = 1024;  // and requests
constexpr int kAllItems = 1280;     // and rows that they may have: B * q_max, 8 to an SM of 160
constexpr int kLoadsAll = 8, kLoadsWalk = 4;  // 16-byte loads of a thread in flight to registers
constexpr int kLaterWalk = 12;                // and to shared memory

struct TreeArgs {
    int B, rows, q_max, V;
    const void *logits;
    const int32_t *row_off, *parent, *ids;
    int32_t *accept_len, *num_emitted, *path, *out_tokens, *commit;
    unsigned long long *key;  // [B, q_max]: verify_tree_all_kernel, 0 between calls
    int32_t *done;            // [B]: parts read, 0 between calls
    int parts;                // of a row
};

struct Rows { int row0, n; };
__device__ __forceinline__ Rows rows_of(const TreeArgs &A, int b) {
    const int a0 = A.row_off[b], a1 = A.row_off[b + 1];
    const int row0 = min(max(a0, 0), A.rows);
    return {row0, min(min(max(a1, row0), A.rows) - row0, A.q_max)};
}

using Key = unsigned long long;
__device__ __forceinline__ Key make_key(float v, int i) {
    const uint32_t x = __float_as_uint(v + 0.f);  // -0 is 0
    return (Key(x ^ (x >> 31 ? 0xffffffffu : 0x80000000u)) << 32) | uint32_t(~i);
}
__device__ __forceinline__ int id_of(Key k) { return int(~uint32_t(k)); }
__device__ __forceinline__ Key warp_max(Key k) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) k = max(k, __shfl_xor_sync(0xffffffffu, k, o));
    return k;
}

// The largest of a 16-byte vector's elements.
template <typename T> __device__ __forceinline__ float vector_max(const uint4 &x);
template <> __device__ __forceinline__ float vector_max<uint16_t>(const uint4 &x) {
    uint32_t m;
    asm("{\n\t.reg .b32 a, b;\n\t"
        "max.bf16x2 a, %1, %2;\n\tmax.bf16x2 b, %3, %4;\n\tmax.bf16x2 %0, a, b;\n\t}"
        : "=r"(m) : "r"(x.x), "r"(x.y), "r"(x.z), "r"(x.w));
    return fmaxf(bf16_lo(m), bf16_hi(m));
}
template <> __device__ __forceinline__ float vector_max<float>(const uint4 &x) {
    return fmaxf(fmaxf(__uint_as_float(x.x), __uint_as_float(x.y)), fmaxf(__uint_as_float(x.z), __uint_as_float(x.w)));
}

// The vector with the largest element so far, of those that a thread has met.
template <typename T>
struct Best {
    float v = -INFINITY;
    int at = -1;
    uint4 x = make_uint4(0, 0, 0, 0);
    __device__ __forceinline__ void meet(const uint4 &y, int c) {
        const float m = vector_max<T>(y);
        if (m > v || at < 0) {  // vectors ascend, so the first of equals stays
            v = m;
            at = c;
            x = y;
        }
    }
    // A vector is taken apart only here, the one that holds the maximum.
    __device__ __forceinline__ Key key() const {
        constexpr int E = Vec<T>::kElems;
        if (at < 0) return 0;
        float z[E];
        Vec<T>::unpack(x, z);
        int e = 0;
#pragma unroll
        for (int k = E - 1; k >= 0; --k)
            if (z[k] == v) e = k;
        return make_key(v, at * E + e);
    }
};

// The largest key of the 16-byte vectors first, first + stride, .. below end of a row, for this thread: kRegs
// loads in flight to registers and kShared to its own places of shared memory, kThreads apart.
template <typename T, int kRegs, int kShared, int kThreads>
__device__ __forceinline__ Key best_of(const uint4 *row, int first, int end, int stride, uint32_t mine) {
    Best<T> best;
    for (int c0 = first; c0 < end; c0 += (kRegs + kShared) * stride) {
#pragma unroll
        for (int k = 0; k < kShared; ++k) {
            const int c = c0 + (kRegs + k) * stride;
            if (c < end)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;"
                             ::"r"(mine + k * kThreads * 16), "l"(row + c) : "memory");
        }
        uint4 x[kRegs];
#pragma unroll
        for (int k = 0; k < kRegs; ++k)
            if (c0 + k * stride < end) x[k] = __ldcs(row + c0 + k * stride);
#pragma unroll
        for (int k = 0; k < kRegs; ++k) {
            if (c0 + k * stride >= end) break;
            best.meet(x[k], c0 + k * stride);
        }
        if (kShared > 0) {
            asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll
            for (int k = 0; k < kShared; ++k) {
                const int c = c0 + (kRegs + k) * stride;
                if (c >= end) break;
                // its own copies, which wait_all has seen land; the next round's are issued behind these reads
                best.meet(ld_shared16(mine + k * kThreads * 16), c);
            }
        }
    }
    return best.key();
}

// The lowest child of row `at` whose token is y; -1: none.  Lane j holds rows j and 32 + j.
__device__ __forceinline__ int child_of(int at, int y, const int (&parent)[2], const int (&id)[2], int lane) {
    const uint32_t lo = __ballot_sync(0xffffffffu, parent[0] == at && id[0] == y);
    const uint32_t hi = __ballot_sync(0xffffffffu, parent[1] == at && id[1] == y);
    return lo ? __ffs(lo) - 1 : hi ? 31 + __ffs(hi) : -1;
}
// Those rows of a request; a parent that is not below its row is none.
__device__ __forceinline__ void load_tree(const TreeArgs &A, const Rows &r, int lane, int (&parent)[2], int (&id)[2]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int j = 32 * h + lane;
        parent[h] = -1;
        id[h] = -1;
        if (j > 0 && j < r.n) {
            parent[h] = A.parent[r.row0 + j];
            id[h] = A.ids[r.row0 + j];
            if (parent[h] >= j) parent[h] = -1;
        }
    }
}

// A walk on its way out: lane j keeps entries j and 32 + j.
struct Walk {
    int len = 0, path[2] = {-1, -1}, token[2] = {-1, -1};
    __device__ __forceinline__ void add(int at, int y, int lane) {
        if (len == lane) {
            path[0] = at;
            token[0] = y;
        } else if (len == 32 + lane) {
            path[1] = at;
            token[1] = y;
        }
        ++len;
    }
    __device__ __forceinline__ void write(const TreeArgs &A, int b, int lane) const {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int j = 32 * h + lane;
            if (j < A.q_max) {
                A.path[int64_t(b) * A.q_max + j] = path[h];
                A.out_tokens[int64_t(b) * A.q_max + j] = token[h];
            }
        }
        if (lane == 0) {
            A.accept_len[b] = max(len - 1, 0);
            A.num_emitted[b] = len;
            if (A.commit) A.commit[b] += len;
        }
    }
};

// A cluster walks one request's tree, row by row.
template <typename T>
__global__ void __launch_bounds__(kThreadsWalk, kResident) verify_tree_kernel(const TreeArgs A) {
    constexpr int kWarpsTree = kThreadsWalk / 32;
    __shared__ uint4 later[kLaterWalk][kThreadsWalk];
    __shared__ Key keys[2][kMaxCluster * kWarpsTree];  // by level % 2: of all warps of the cluster
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int rank, size;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(size));
    // all CTAs of the cluster are there before one writes to another's memory (waited for below)
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int b = blockIdx.x / size, vecs = A.V / Vec<T>::kElems;
    const Rows r = rows_of(A, b);
    int parent[2], id[2];
    load_tree(A, r, lane, parent, id);
    Walk walk;
    int at = r.n > 0 ? 0 : -1;
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    while (at >= 0) {
        const uint4 *row = reinterpret_cast<const uint4 *>(static_cast<const T *>(A.logits) + int64_t(r.row0 + at) * A.V);
        Key k = warp_max(best_of<T, kLoadsWalk, kLaterWalk, kThreadsWalk>(
            row, rank * kThreadsWalk + tid, vecs, size * kThreadsWalk, smem_addr(&later[0][tid])));
        Key *const mine = &keys[walk.len & 1][rank * kWarpsTree + warp];
        if (lane < size)
            asm volatile(
                "{\n\t.reg .b32 a;\n\t"
                "mapa.shared::cluster.u32 a, %0, %1;\n\t"
                "st.shared::cluster.b64 [a], %2;\n\t}"
                ::"r"(smem_addr(mine)), "r"(lane), "l"(k) : "memory");
        // One barrier a level: the other buffer is written only by warps that have passed the next one.
        asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
        k = 0;
        for (int w = lane; w < size * kWarpsTree; w += 32) k = max(k, keys[walk.len & 1][w]);
        const int y = id_of(warp_max(k));
        const int next = child_of(at, y, parent, id, lane);
        walk.add(at, y, lane);
        at = next;
    }
    if (rank == 0 && warp == 0) walk.write(A, b, lane);
    // no CTA ends while others may still write to it: the last barrier came after the last write
}

// All rows at once.
template <typename T>
__global__ void __launch_bounds__(kThreadsAll) verify_tree_all_kernel(const TreeArgs A) {
    __shared__ Key keys[kThreadsAll / 32];
    __shared__ int last;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int item = blockIdx.x / A.parts, part = blockIdx.x - item * A.parts;
    const int b = item / A.q_max, j = item - b * A.q_max;
    const Rows r = rows_of(A, b);
    if (j >= r.n) {
        if (r.n == 0 && j == 0 && part == 0 && warp == 0) Walk().write(A, b, lane);
        return;
    }
    const int vecs = A.V / Vec<T>::kElems, each = (vecs + A.parts - 1) / A.parts;
    const uint4 *row = reinterpret_cast<const uint4 *>(static_cast<const T *>(A.logits) + int64_t(r.row0 + j) * A.V);
    Key k = warp_max(best_of<T, kLoadsAll, 0, kThreadsAll>(row, part * each + tid, min((part + 1) * each, vecs),
                                                              kThreadsAll, 0));
    if (lane == 0) keys[warp] = k;
    __syncthreads();
    if (warp > 0) return;
    k = warp_max(lane < kThreadsAll / 32 ? keys[lane] : 0);
    if (lane == 0) {
        atomicMax(A.key + item, k);
        __threadfence();
        last = atomicAdd(A.done + b, 1) == r.n * A.parts - 1;
    }
    __syncwarp();
    if (!last) return;
    __threadfence();
    int parent[2], id[2], best[2] = {0, 0};
    load_tree(A, r, lane, parent, id);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if (32 * h + lane < r.n) {
            Key *const at = A.key + b * A.q_max + 32 * h + lane;
            best[h] = id_of(__ldcg(at));
            *at = 0;  // as the next call wants it
        }
    }
    if (lane == 0) A.done[b] = 0;
    Walk walk;
    for (int at = 0; at >= 0;) {
        const int lo = __shfl_sync(0xffffffffu, best[0], at & 31), hi = __shfl_sync(0xffffffffu, best[1], at & 31);
        const int y = at < 32 ? lo : hi;
        walk.add(at, y, lane);
        at = child_of(at, y, parent, id, lane);
    }
    walk.write(A, b, lane);
}

template <typename T>
cudaError_t launch(TreeArgs A, bool together, int sms, cudaStream_t s) {
    // all in one wave of CTAs
    if (together && A.B * A.q_max <= std::min(8 * sms, kAllItems)) {
        A.parts = std::max(1, std::min(4 * sms / (A.B * A.q_max), A.V / 2048));
        return launch_overlapped(verify_tree_all_kernel<T>, A.B * A.q_max * A.parts, kThreadsAll, 0, s, A);
    }
    int size = kMaxCluster;
    // one wave too, and no thread without a vector of the row
    while (size > 1 && (A.B * size > kResident * sms || size / 2 * kThreadsWalk >= A.V / Vec<T>::kElems)) size /= 2;
    if (size > 8) {
        const cudaError_t e =
            cudaFuncSetAttribute(verify_tree_kernel<T>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
    }
    return launch_clusters(verify_tree_kernel<T>, A.B * size, kThreadsWalk, size, s, A);
}

}  // namespace

// The workspace: status; parts done by request; keys by request and row.  As large for every shape, so that one serves all.
constexpr size_t kDoneAt = 256, kKeysAt = kDoneAt + sizeof(int32_t) * kAllRequests;
size_t tree_workspace_bytes() { return kKeysAt + sizeof(Key) * kAllItems; }

cudaError_t launch_verify_tree(const dspark_tree &t, int sms, cudaStream_t s) {
    char *ws = static_cast<char *>(t.workspace);
    const bool bf16 = t.logit_dtype == DSPARK_BF16;
    const size_t bytes = size_t(t.rows) * t.V * (bf16 ? 2 : 4);
    const TreeArgs A{t.B, t.rows, t.q_max, t.V, t.target_logits, t.row_off, t.parent, t.packed_ids,
                     t.accept_len, t.num_emitted, t.path, t.out_tokens, t.seq_lens_commit,
                     reinterpret_cast<Key *>(ws + kKeysAt), reinterpret_cast<int32_t *>(ws + kDoneAt), 1};
    const bool together = t.rows > 0 && t.B <= kAllRequests && bytes <= kAllBytes;
    return bf16 ? launch<uint16_t>(A, together, sms, s) : launch<float>(A, together, sms, s);
}

}  // namespace dspark
