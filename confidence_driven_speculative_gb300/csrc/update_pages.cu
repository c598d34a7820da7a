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
//
// Measured: 256 requests of 16 to 4095 positions in pages of 16 that grow by 17,
// 12.0 us (with one CTA in place of the cluster of 16, some 5 more), most of it six trips
// to L2 or through the cluster and a second launch; the same in pages of one position
// 86 (half a million entries on 16 SMs); 8 requests forked 8 ways with tails of 32 layers,
// 8 heads of 128, pages of 64, 50 (a copy of as many bytes 54.6; seven requests
// read each source, which L2 serves, so 31 would be the least): 12 CTAs an SM for the
// copies (with 3, 4, 6 and 9: 66, 66, 61 and 56 against then 54, the step 14.3 to
// 15.3), their stores streaming (54 without; units taken off a counter by 3 or 4 CTAs
// an SM 55 and 52).
#include <algorithm>

#include "cache.cuh"
#include "dspark_internal.cuh"
#include "tcgen05.cuh"

namespace dspark {
namespace {

constexpr int kThreadsPages = 1024;
static_assert(kThreadsPages == 32 * 32, "the scan takes a warp's sums from a lane each");
constexpr int kSeg = 256;               // entries of a table that a warp takes at once
constexpr int kPages = 8;               // pages in a row that a thread looks at
constexpr int kFull = 0x7fffffff;       // claim of a request that only reads
constexpr int kWriters = 1 << 17;       // kWriters - b: claim of request b that writes

struct PagesArgs {
    int B_in, B, max_pages, num_pages, page_size, sink_pages;
    uint32_t page_mul, page_shift;  // position / page_size = position * mul >> shift
    const int32_t *table_in, *parent, *keep_len, *want_len, *first_pos, *held;
    int32_t *table_out, *granted_len, *tail_src, *tail_dst, *totals;
    int32_t *claim;   // [num_pages], 0 between calls
    int32_t *free_list;  // [num_pages]
    int4 *copies;        // [B] source, destination, entries
    int32_t *first_rank; // [B] rank of a request's first new page
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
    auto page_of = [&](int pos) { return int((uint64_t(uint32_t(pos)) * A.page_mul) >> A.page_shift); };
    Want w;
    const int cap = A.max_pages * A.page_size;
    w.parent = A.parent ? A.parent[b] : b;
    if (w.parent >= A.B_in) w.parent = -1;
    w.keep = w.parent < 0 ? 0 : min(max(A.keep_len[b], 0), cap);  // nothing is kept of no parent
    w.want = min(max(A.want_len[b], w.keep), cap);
    w.first = A.first_pos ? page_of(max(A.first_pos[b], 0)) : 0;
    w.keep_pages = page_of(w.keep + A.page_size - 1);
    w.want_pages = page_of(w.want + A.page_size - 1);
    const int last = page_of(w.keep);
    w.tail = w.want > w.keep && last < w.keep_pages ? last : -1;
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
    __shared__ int warp_sum[2][32], cta_sum[2], cta_before[2], cluster_sum[2];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rank = cluster_rank();
    // Warps of one number lie in different CTAs, so that few requests keep all CTAs busy.
    const int g = rank * kThreadsPages + tid, gw = warp * kCtas + rank;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // A thread looks after `per` requests; of the first it keeps what it knows.
    if (g == 0) *A.n_copies = 0;
    const int per = (A.B + kAll - 1) / kAll;
    const int b_lo = min(g * per, A.B), b_hi = min(b_lo + per, A.B);
    auto tail_kept = [&](const Want &w) { return w.tail >= 0 && (w.tail >= w.first || w.tail < A.sink_pages); };
    auto tail_page = [&](const Want &w) {  // that the tail lies in, or -1
        if (w.parent < 0 || !tail_kept(w)) return -1;
        const int page = A.table_in[int64_t(w.parent) * A.max_pages + w.tail];
        return page < A.num_pages ? page : -1;
    };
    Want w0{};
    int tail0 = -1;
    if (b_lo < b_hi) {
        w0 = load_want(A, b_lo);
        tail0 = tail_page(w0);
    }

    // ---- what is kept, and the claims on it --------------------------------
    const int segs = (A.max_pages + kSeg - 1) / kSeg;
    for (int b = gw / segs, seg = gw % segs; b < A.B;) {
        const int i0 = seg * kSeg + lane;
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
        b += kAllWarps / segs;
        seg += kAllWarps % segs;
        if (seg >= segs) {
            seg -= segs;
            ++b;
        }
    }
    cluster_sync();

    // ---- ranks of the wanted pages and of the free ones ---------------------
    // Does request b's tail, in `page`, need a page of its own?
    auto shares = [&](int b, int page) {
        return page >= 0 && (__ldcg(A.claim + page) != kWriters - b || (A.held && A.held[page]));
    };
    const int claim0 = tail0 >= 0 ? __ldcg(A.claim + tail0) : 0, held0 = tail0 >= 0 && A.held ? A.held[tail0] : 0;
    // Of every kAll * kPages pages a thread looks at kPages in a row.
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
        if (warp < 2) {  // one reader a CTA: all warps at once take 5 us
            const int x = lane < kCtas ? remote(&cta_sum[warp], lane) : 0;
            const int below = __reduce_add_sync(0xffffffffu, lane < rank ? x : 0);
            const int all = __reduce_add_sync(0xffffffffu, x);
            if (lane == 0) {
                cta_before[warp] = below;
                cluster_sum[warp] = all;
            }
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            before[k] += warp_sum[k][warp] + cta_before[k];
            total[k] = cluster_sum[k];
        }
    };
    int count[2] = {0, 0}, at[2], total[2];
    for (int b = b_lo + 1; b < b_hi; ++b) {
        const Want w = load_want(A, b);
        count[0] += Fresh(A, w).count + shares(b, tail_page(w));
    }
    uint32_t bits = free_bits(int64_t(g) * kPages);
    count[1] = __popc(bits);
    const int share0 = tail0 >= 0 && (claim0 != kWriters - b_lo || held0);
    if (b_lo < b_hi) count[0] += Fresh(A, w0).count + share0;
    scan(count, at, total);
    const int wanted = total[0], start0 = at[0];  // rank of the thread's first wanted page
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
    int start = start0;
    for (int b = b_lo; b < b_hi; ++b) {
        const Want w = b == b_lo ? w0 : load_want(A, b);
        const int share = b == b_lo ? share0 : shares(b, tail_page(w));
        A.first_rank[b] = start + share;
        start += Fresh(A, w).count + share;
    }
    cluster_sync();

    // ---- the wanted pages, and the claims back to zero ----------------------
    auto finish = [&](int b, const Want &w, const Fresh &f, int start, int share, int page) {
        const int all = f.count + share, given = min(max(there - start, 0), all);
        int src = -1, dst = -1;
        if (share && given > 0) {
            src = page;
            dst = __ldcg(A.free_list + start);
            A.table_out[int64_t(b) * A.max_pages + w.tail] = dst;
            A.copies[atomicAdd(A.n_copies, 1)] = make_int4(src, dst, w.keep - w.tail * A.page_size, 0);
        }
        A.tail_src[b] = src;
        A.tail_dst[b] = dst;
        A.granted_len[b] = (tail_kept(w) && page < 0) || given < share ? w.keep  // where keep lies has no memory
                           : given == all ? w.want
                                           : max(f.place(w, given - share) * A.page_size, w.keep);
    };
    start = start0;
    for (int b = b_lo; b < b_hi; ++b) {
        const Want w = b == b_lo ? w0 : load_want(A, b);
        const int page = b == b_lo ? tail0 : tail_page(w), share = b == b_lo ? share0 : shares(b, page);
        const Fresh f(A, w);
        finish(b, w, f, start, share, page);
        start += f.count + share;
    }
    // New pages, a request to a warp.  (By the threads that know the requests, which are neighbours, the others of a
    // warp waiting: 192 requests that want up to 47 each 41 us against 12.5.)
    for (int b = gw; b < A.B; b += kAllWarps) {
        const Want w = load_want(A, b);
        const Fresh f(A, w);
        const int first = __ldcg(A.first_rank + b), given = min(max(there - first, 0), f.count);
        for (int i = lane; i < given; i += 32)
            A.table_out[int64_t(b) * A.max_pages + f.place(w, i)] = __ldcg(A.free_list + first + i);
    }
    if (per > 1) cluster_sync();  // claims are read up to here
    for (int64_t p = int64_t(g) * kPages; p < A.num_pages; p += chunk) {
        if (p + kPages <= A.num_pages) {
#pragma unroll
            for (int k = 0; k < kPages / 4; ++k) reinterpret_cast<int4 *>(A.claim + p)[k] = make_int4(0, 0, 0, 0);
        } else {
            for (int k = 0; p + k < A.num_pages; ++k) A.claim[p + k] = 0;
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
                    if (s + k * step < c.z) __stcs(reinterpret_cast<uint4 *>(to + (s + k * step) * A.slot_stride), x[k]);
            }
        }
    }
}

// The workspace: status word, number of copies; claims; free pages; copies; first ranks.  The claims, which are zero between
// calls, lie where they do for every B.
struct PagesLayout { size_t claim, free_list, copies, first_rank, total; };
PagesLayout pages_layout(int B, int num_pages) {
    PagesLayout l;
    l.claim = 256;
    l.free_list = l.claim + align256(sizeof(int32_t) * size_t(num_pages));
    l.copies = l.free_list + align256(sizeof(int32_t) * size_t(num_pages));
    l.first_rank = l.copies + align256(sizeof(int4) * size_t(B));
    l.total = l.first_rank + align256(sizeof(int32_t) * size_t(B));
    return l;
}

}  // namespace

size_t pages_workspace_bytes(int B, int num_pages) { return pages_layout(B, num_pages).total; }

cudaError_t launch_update_pages(const dspark_pages &p, int sms, cudaStream_t s) {
    const dspark_cache &c = p.cache;
    char *ws = static_cast<char *>(p.workspace);
    const PagesLayout l = pages_layout(p.B, c.num_pages);
    uint32_t shift = 31;  // exact below 2^31: mul = ceil(2^shift / page_size) < 2^32
    while ((1u << (shift - 31)) < unsigned(c.page_size)) ++shift;
    const uint32_t mul = uint32_t(((1ull << shift) + c.page_size - 1) / c.page_size);
    PagesArgs A{p.B_in, p.B, p.max_pages, c.num_pages, c.page_size,
                int((int64_t(p.sinks) + c.page_size - 1) / c.page_size), mul, shift, p.table_in, p.parent, p.keep_len,
                p.want_len, p.first_pos, p.held, p.table_out, p.granted_len, p.tail_src, p.tail_dst, p.totals,
                reinterpret_cast<int32_t *>(ws + l.claim), reinterpret_cast<int32_t *>(ws + l.free_list),
                reinterpret_cast<int4 *>(ws + l.copies), reinterpret_cast<int32_t *>(ws + l.first_rank),
                reinterpret_cast<int32_t *>(ws) + 1};
    constexpr int kCtas = 16;
    cudaError_t e = cudaFuncSetAttribute(update_pages_kernel<kCtas>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    e = launch_clusters(update_pages_kernel<kCtas>, kCtas, kThreadsPages, kCtas, s, A);
    if (e != cudaSuccess || !c.k_cache) return e;
    const CopyArgs C{c.layers, c.Hkv, c.D / 8, c.layer_stride, c.page_stride, c.slot_stride, c.head_stride,
                     static_cast<uint16_t *>(c.k_cache), static_cast<uint16_t *>(c.v_cache), A.copies, A.n_copies};
    const int ctas = int(std::min<int64_t>(12 * sms, int64_t(2) * c.layers * p.B));  // no more than there may be tails
    return launch_overlapped(copy_tails_kernel, ctas, kThreadsCopy, 0, s, C);
}

}  // namespace dspark
