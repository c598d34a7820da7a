// update_pages.cu -- the pages of a batch's next step: kept, shared, copied
// where two requests would write one, given out and freed.
//
// The free pages are not kept anywhere; each call derives them.  A word per
// page in the workspace, zero between calls, takes the largest claim on it: all
// ones of a request that names the page without writing it, else
// kWriters - b of the lowest request b whose tail it is.  A page without a
// claim is free.  Then the wanted pages are counted by request, the free ones by
// page, both are summed up, and the n-th wanted one gets the n-th free one.
// Claims are maxima of whole numbers and ranks are sums of them, so the result
// does not depend on timing.
//
// Bound: latency.  The work is a few words per page in use, in four steps that
// each need the whole of the one before.  One cluster does them with
// hardware barriers in between; a second kernel on all SMs copies the tails' entries.
#include "cache.cuh"
#include "dspark_internal.cuh"
#include "tcgen05.cuh"

namespace dspark {
namespace {

constexpr int kThreadsPages = 1024;
constexpr int kSeg = 256;               // entries of a table that a warp takes at once
constexpr int kPages = 8;               // pages in a row that a thread looks at
constexpr int kFull = 0x7fffffff;       // claim of a request that only reads
constexpr int kWriters = 1 << 17;       // kWriters - b: claim of request b that writes

struct PagesArgs {
    int B_in, B, max_pages, num_pages, page_size, sink_pages;
    const int32_t *table_in, *parent, *keep_len, *want_len, *first_pos, *held;
    int32_t *table_out, *granted_len, *tail_src, *tail_dst, *totals;
    int32_t *claim;   // [num_pages], 0 between calls
    int32_t *free_list;  // [num_pages]
    int2 *start;      // [B] rank of the request's first wanted page, does its tail need one?
    int4 *copies;     // [B] source, destination, entries
    int32_t *n_copies;
};

// A request: whose pages it takes over, and which.
struct Want {
    int parent, keep, want;       // row of table_in or -1; positions
    int keep_pages, want_pages;   // pages that hold them
    int first;                    // pages before it are dropped, but for the sinks'
    int tail;                     // the page that keep lies inside and that is written; or -1
};

__device__ __forceinline__ Want load_want(const PagesArgs &A, int b) {
    Want w;
    const int cap = A.max_pages * A.page_size;
    w.parent = A.parent ? A.parent[b] : b;
    if (w.parent >= A.B_in) w.parent = -1;
    w.keep = min(max(A.keep_len[b], 0), cap);
    w.want = min(max(A.want_len[b], w.keep), cap);
    w.first = A.first_pos ? max(A.first_pos[b], 0) / A.page_size : 0;
    w.keep_pages = (w.keep + A.page_size - 1) / A.page_size;
    w.want_pages = (w.want + A.page_size - 1) / A.page_size;
    w.tail = w.want > w.keep && w.keep % A.page_size ? w.keep_pages - 1 : -1;
    return w;
}

// New pages of a request: places [keep_pages, low_end) of the sinks, then [high, want_pages).
struct Fresh {
    int low, high, count;  // the sinks' number, first place of the others, all
    __device__ __forceinline__ Fresh(const PagesArgs &A, const Want &w) {
        low = max(min(w.want_pages, A.sink_pages) - w.keep_pages, 0);
        high = max(max(w.keep_pages, w.first), A.sink_pages);
        count = low + max(w.want_pages - high, 0);
    }
    __device__ __forceinline__ int place(const Want &w, int i) const {
        return i < low ? w.keep_pages + i : high + i - low;
    }
};

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ int cluster_rank() {
    int r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// A word of another CTA's shared memory.
__device__ __forceinline__ int remote(const int *p, int rank) {
    int v;
    asm volatile(
        "{\n\t.reg .b32 a;\n\t"
        "mapa.shared::cluster.u32 a, %1, %2;\n\t"
        "ld.shared::cluster.b32 %0, [a];\n\t}"
        : "=r"(v) : "r"(smem_addr(p)), "r"(rank) : "memory");
    return v;
}

template <int kCtas>
__global__ void __launch_bounds__(kThreadsPages, 1) update_pages_kernel(const PagesArgs A) {
    constexpr int kAll = kCtas * kThreadsPages, kAllWarps = kAll / 32;
    __shared__ int warp_sum[2][32], cta_sum[2];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rank = cluster_rank();
    // Warps of one number lie in different CTAs, so that few requests keep all CTAs busy.
    const int g = rank * kThreadsPages + tid, gw = warp * kCtas + rank;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // ---- what is kept, and the claims on it --------------------------------
    if (g == 0) *A.n_copies = 0;
    const int segs = (A.max_pages + kSeg - 1) / kSeg;
    for (int64_t s = gw; s < int64_t(A.B) * segs; s += kAllWarps) {
        const int b = int(s / segs), i0 = int(s - int64_t(b) * segs) * kSeg + lane;
        const Want w = load_want(A, b);
        const int32_t *in = A.table_in + int64_t(max(w.parent, 0)) * A.max_pages;
        int32_t *out = A.table_out + int64_t(b) * A.max_pages;
        int page[kSeg / 32];
#pragma unroll
        for (int k = 0; k < kSeg / 32; ++k) {
            const int i = i0 + 32 * k;
            page[k] = -1;
            if (w.parent >= 0 && i < w.keep_pages && (i >= w.first || i < A.sink_pages)) page[k] = in[i];
            if (page[k] >= A.num_pages) page[k] = -1;
        }
#pragma unroll
        for (int k = 0; k < kSeg / 32; ++k) {
            const int i = i0 + 32 * k;
            if (i >= A.max_pages) break;
            if (page[k] >= 0) atomicMax(A.claim + page[k], i == w.tail ? kWriters - b : kFull);
            out[i] = max(page[k], -1);
        }
    }
    cluster_sync();

    // ---- ranks of the wanted pages and of the free ones ---------------------
    // A thread counts the pages of `per` requests, and of every kAll * kPages
    // pages kPages in a row.
    const int per = (A.B + kAll - 1) / kAll;
    const int b_lo = min(g * per, A.B), b_hi = min(b_lo + per, A.B);
    // Does request b's tail need a page of its own?
    auto shares = [&](int b, const Want &w) {
        if (w.tail < 0) return false;
        const int page = __ldcg(A.table_out + int64_t(b) * A.max_pages + w.tail);
        return page >= 0 && (__ldcg(A.claim + page) != kWriters - b || (A.held && A.held[page]));
    };
    const int64_t chunk = int64_t(kAll) * kPages;
    // Bits of the free ones of a thread's pages p .. p + kPages - 1; their claims go back to zero in `clear`.
    auto free_bits = [&](int64_t p) {
        uint32_t bits = 0;
        if (p + kPages <= A.num_pages) {
            int4 c[kPages / 4], h[kPages / 4];
#pragma unroll
            for (int k = 0; k < kPages / 4; ++k) {
                c[k] = __ldcg(reinterpret_cast<const int4 *>(A.claim + p) + k);
                h[k] = make_int4(0, 0, 0, 0);
            }
            if (A.held) {
#pragma unroll
                for (int k = 0; k < kPages; ++k) reinterpret_cast<int *>(h)[k] = A.held[p + k];
            }
#pragma unroll
            for (int k = 0; k < kPages / 4; ++k) {
                bits |= uint32_t((c[k].x | h[k].x) == 0) << (4 * k) | uint32_t((c[k].y | h[k].y) == 0) << (4 * k + 1) |
                        uint32_t((c[k].z | h[k].z) == 0) << (4 * k + 2) | uint32_t((c[k].w | h[k].w) == 0) << (4 * k + 3);
            }
        } else {
            for (int k = 0; k < kPages; ++k)
                if (p + k < A.num_pages && __ldcg(A.claim + p + k) == 0 && !(A.held && A.held[p + k])) bits |= 1u << k;
        }
        return bits;
    };
    // Exclusive sums over the cluster's threads, and the totals.
    auto scan = [&](const int (&mine)[2], int (&before)[2], int (&total)[2]) {
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            int x = mine[k];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += y;
            }
            if (lane == 31) warp_sum[k][warp] = x;
            before[k] = x - mine[k];
        }
        __syncthreads();
        if (warp < 2) {
            int x = warp_sum[warp][lane];
            const int own = x;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += y;
            }
            warp_sum[warp][lane] = x - own;
            if (lane == 31) cta_sum[warp] = x;
        }
        cluster_sync();
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int x = lane < kCtas ? remote(&cta_sum[k], lane) : 0;
            before[k] += warp_sum[k][warp] + __reduce_add_sync(0xffffffffu, lane < rank ? x : 0);
            total[k] = __reduce_add_sync(0xffffffffu, x);
        }
    };
    int count[2] = {0, 0}, at[2], total[2];
    for (int b = b_lo; b < b_hi; ++b) {
        const Want w = load_want(A, b);
        count[0] += Fresh(A, w).count + shares(b, w);
    }
    uint32_t bits = free_bits(int64_t(g) * kPages);
    count[1] = __popc(bits);
    scan(count, at, total);
    const int wanted = total[0];
    for (int b = b_lo; b < b_hi; ++b) {
        const Want w = load_want(A, b);
        const int share = shares(b, w);
        A.start[b] = make_int2(at[0], share);
        at[0] += Fresh(A, w).count + share;
    }
    int there = 0;
    for (int64_t p0 = 0;;) {
        for (int left = bits, n = there + at[1]; left && n < wanted; left &= left - 1)
            A.free_list[n++] = int(p0 + int64_t(g) * kPages) + __ffs(left) - 1;
        there += total[1];
        if ((p0 += chunk) >= A.num_pages) break;
        bits = free_bits(p0 + int64_t(g) * kPages);
        count[0] = 0;
        count[1] = __popc(bits);
        cluster_sync();  // the sums are read
        scan(count, at, total);
    }
    if (g == 0) {
        A.totals[0] = max(there - wanted, 0);
        A.totals[1] = max(wanted - there, 0);
    }
    cluster_sync();

    // ---- the wanted pages, and the claims back to zero ----------------------
    for (int64_t p = int64_t(g) * kPages; p < A.num_pages; p += chunk) {
        if (p + kPages <= A.num_pages) {
#pragma unroll
            for (int k = 0; k < kPages / 4; ++k) reinterpret_cast<int4 *>(A.claim + p)[k] = make_int4(0, 0, 0, 0);
        } else {
            for (int k = 0; p + k < A.num_pages; ++k) A.claim[p + k] = 0;
        }
    }
    for (int b = gw; b < A.B; b += kAllWarps) {
        const int2 s = __ldcg(A.start + b);
        const Want w = load_want(A, b);
        const Fresh f(A, w);
        const int share = s.y, count = f.count + share, given = min(max(there - s.x, 0), count);
        int32_t *out = A.table_out + int64_t(b) * A.max_pages;
        for (int i = lane; i < f.count; i += 32)
            if (i + share < given) out[f.place(w, i)] = __ldcg(A.free_list + s.x + share + i);
        if (lane == 0) {
            int src = -1, dst = -1;
            if (share && given > 0) {
                src = __ldcg(out + w.tail);
                dst = __ldcg(A.free_list + s.x);
                out[w.tail] = dst;
                A.copies[atomicAdd(A.n_copies, 1)] = make_int4(src, dst, w.keep % A.page_size, 0);
            }
            A.tail_src[b] = src;
            A.tail_dst[b] = dst;
            A.granted_len[b] = given == count ? w.want
                               : given < share ? w.keep
                                               : max(f.place(w, given - share) * A.page_size, w.keep);
        }
    }
}

struct CopyArgs {
    int layers, heads, chunks;  // chunks: 16-byte parts of an entry
    int64_t layer_stride, page_stride, slot_stride, head_stride;
    uint16_t *k, *v;
    const int4 *copies;
    const int32_t *n_copies;
};

constexpr int kThreadsCopy = 256;
constexpr int kCopies = 8;  // 16-byte parts that a thread has asked for before it stores

// A CTA takes one tail of one layer, of k or v, at a time.
__global__ void __launch_bounds__(kThreadsCopy) copy_tails_kernel(const CopyArgs A) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int n = *A.n_copies, tid = threadIdx.x;
    const int64_t units = int64_t(n) * A.layers * 2;
    // A thread keeps its place in an entry and walks the slots, `step` at a time.
    const int per_slot = A.heads * A.chunks, step = max(kThreadsCopy / per_slot, 1), slot0 = tid / per_slot;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int lk = int(u / n);
        const int4 c = A.copies[u - int64_t(lk) * n];
        uint16_t *const base = (lk & 1 ? A.v : A.k) + (lk >> 1) * A.layer_stride;
        if (slot0 >= step) continue;
        for (int in = tid - slot0 * per_slot; in < per_slot; in += kThreadsCopy) {
            const int head = in / A.chunks;
            uint16_t *const at = base + head * A.head_stride + (in - head * A.chunks) * 8;
            const uint16_t *const from = at + c.x * A.page_stride;
            uint16_t *const to = at + c.y * A.page_stride;
            for (int s = slot0; s < c.z; s += step * kCopies) {
                uint4 x[kCopies];
#pragma unroll
                for (int k = 0; k < kCopies; ++k)
                    if (s + k * step < c.z) x[k] = __ldcs(reinterpret_cast<const uint4 *>(from + (s + k * step) * A.slot_stride));
#pragma unroll
                for (int k = 0; k < kCopies; ++k)
                    if (s + k * step < c.z) *reinterpret_cast<uint4 *>(to + (s + k * step) * A.slot_stride) = x[k];
            }
        }
    }
}

// The workspace: status word, number of copies; copies; ranks; claims; free pages.
struct PagesLayout { size_t copies, start, claim, free_list, total; };
PagesLayout pages_layout(int B, int num_pages) {
    PagesLayout l;
    l.copies = 256;
    l.start = l.copies + align256(sizeof(int4) * size_t(B));
    l.claim = l.start + align256(sizeof(int2) * size_t(B));
    l.free_list = l.claim + align256(sizeof(int32_t) * size_t(num_pages));
    l.total = l.free_list + align256(sizeof(int32_t) * size_t(num_pages));
    return l;
}

}  // namespace

size_t pages_workspace_bytes(int B, int num_pages) { return pages_layout(B, num_pages).total; }

cudaError_t launch_update_pages(const dspark_pages &p, int sms, cudaStream_t s) {
    const dspark_cache &c = p.cache;
    char *ws = static_cast<char *>(p.workspace);
    const PagesLayout l = pages_layout(p.B, c.num_pages);
    PagesArgs A{p.B_in, p.B, p.max_pages, c.num_pages, c.page_size,
                int((int64_t(p.sinks) + c.page_size - 1) / c.page_size), p.table_in, p.parent, p.keep_len,
                p.want_len, p.first_pos, p.held, p.table_out, p.granted_len, p.tail_src, p.tail_dst, p.totals,
                reinterpret_cast<int32_t *>(ws + l.claim), reinterpret_cast<int32_t *>(ws + l.free_list),
                reinterpret_cast<int2 *>(ws + l.start), reinterpret_cast<int4 *>(ws + l.copies),
                reinterpret_cast<int32_t *>(ws) + 1};
    constexpr int kCtas = 16;
    cudaError_t e = cudaFuncSetAttribute(update_pages_kernel<kCtas>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    e = launch_clusters(update_pages_kernel<kCtas>, kCtas, kThreadsPages, kCtas, s, A);
    if (e != cudaSuccess || !c.k_cache) return e;
    const CopyArgs C{c.layers, c.Hkv, c.D / 8, c.layer_stride, c.page_stride, c.slot_stride, c.head_stride,
                     static_cast<uint16_t *>(c.k_cache), static_cast<uint16_t *>(c.v_cache), A.copies, A.n_copies};
    return launch_overlapped(copy_tails_kernel, 8 * sms, kThreadsCopy, 0, s, C);
}

}  // namespace dspark
