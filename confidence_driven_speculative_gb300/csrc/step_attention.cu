// step_attention.cu -- the step's rows over the paged cache.
//
// Mathematics.  One request and one cached head give a block of
// cols = rows * G query vectors (G query heads share the cached head) over the
// request's keys.  The keys are walked in tiles of 128 with a running
// reference m and, per column, o = sum 2^(x - m) v and l = sum 2^(x - m),
// x = scale * log2(e) * q.k; the output is o / l.
//
// Layout.  A step has few columns (4 to a few tens) and many keys, so the
// products are taken transposed: the 128 keys of a tile are the M side of the
// tensor core, the columns the N side, padded only to a multiple of 16:
//     S^T [128 keys x N]  = K [128 x D] Q^T          (K and Q K-major)
//     O^T [D x N]        += V^T [D x 128] P^T        (V and P MN-major)
//     L   [D x N]        += 1 [D x 128] P^T          (sum of the rounded weights)
// Each softmax thread owns one key, so the exponentials are spread over all
// 128 threads however few the columns are.  S, O and L live in TMEM.  The
// reference is the first tile's maximum and moves only when some score
// passes it by 2^8 (the weights stay in range of fp32 and bfloat16 keeps its
// relative step), so an ordinary tile needs no reduction over keys at all:
// one vote of the 128 threads.
//
// Bound: bytes of the cache.  One persistent CTA per SM keeps a ring of
// 32 KB K and V tiles (128 keys x 128) filled by TMA; a tile's chain (S, softmax, O)
// is shorter than its copy, so one chain in flight is enough.
//
// Split.  The tiles of all (request, cached head, block of columns) units
// form one list, cut evenly over the CTAs; the cut points come from a scan of
// the lengths in every CTA, on the device.  A unit that is cut leaves partial
// (o, m, l) in the workspace, in fp32, and step_join_kernel adds them in the order of
// the keys, so the result does not depend on timing.
#include <algorithm>

#include "attn.cuh"
#include "dspark_internal.cuh"
#include "tcgen05.cuh"

namespace dspark {
namespace {

constexpr int kTile = 128;      // keys of a tile
constexpr int kMaxCols = 160;   // columns of a unit: 3 x 160 <= 512 TMEM columns
constexpr int kMaxSlots = 12;   // ring slots (one K or one V tile each)
constexpr int kWords = 16;      // ring of the tiles' bad-key words
constexpr int kSoftThreads = 128;
constexpr int kThreadsStep = 192;  // 4 softmax warps, the producer, the MMA issuer
constexpr uint32_t kColS = 0, kColO = kMaxCols, kColL = 2 * kMaxCols;
constexpr uint32_t kTmemCols = 512;
constexpr float kRefMin = -1e30f;  // reference of a column without a score yet
constexpr float kRefSlack = 8.0f;  // log2: how far a score may pass the reference
constexpr int kJoinThreads = 128;

// What step_join_kernel needs of the unit that is cut before CTA i.
struct CutInfo {
    int32_t first, last;      // the CTAs that share it; first < i <= last, or last = -1: no cut
    int32_t slot_first;       // partial slot of the first one (the others': 2 * CTA)
    int32_t row0, head0;      // packed row of the request, first query head of the group
    int32_t c0, ncols;
    int32_t pad;
};

struct StepArgs {
    int B, rows, q_max, Hq, Hkv, G;
    int page_size, num_pages, max_pages, window;
    int box;                   // keys of a TMA box (divides the page and the tile); 0: gather
    int ncap;                  // columns of a unit at most, a multiple of 16
    int slots;
    int page_rows, head_rows;  // gather: rows of the 2-D view per page and head
    int head_x;                // gather: entries of a row per head
    float scale2;              // scale * log2(e)
    int64_t page_stride, slot_stride, head_stride;
    const uint16_t *q, *v_cache;
    const int32_t *row_off, *seq_lens, *block_table;
    uint16_t *out;
    float *part;               // [2 * CTAs][ncap][D]
    float *stat;               // [2 * CTAs][2][ncap]: reference, sum
    CutInfo *cut;              // [CTAs]
    int32_t *status;
    uint64_t wait_ns;
};

// A request's block of work.
struct Req {
    int row0, n;     // packed rows
    int pos0;        // position of the first one
    int kbeg, kend;  // keys that some row sees
    int t0, nt;      // tiles
    int rt, per;     // blocks of columns, columns of one
};

__device__ __forceinline__ Req load_req(const StepArgs &A, int b) {
    Req r;
    const int a0 = A.row_off[b], a1 = A.row_off[b + 1];
    r.row0 = min(max(a0, 0), A.rows);
    r.n = min(min(max(a1, r.row0), A.rows) - r.row0, A.q_max);
    // far past any table, where nothing is seen, stays in 32 bits
    r.pos0 = A.seq_lens ? min(max(A.seq_lens[b], 0), INT32_MAX - 65536) : 0;
    const int cap = A.max_pages * A.page_size;
    r.kend = int(min((long long)r.pos0 + r.n, (long long)cap));
    r.kbeg = A.window > 0 ? min(max(r.pos0 - A.window + 1, 0), r.kend) : 0;
    r.t0 = r.kbeg / kTile;
    r.nt = max((r.kend + kTile - 1) / kTile - r.t0, 1);
    const int cols = r.n * A.G;
    const int blocks = (cols + A.ncap - 1) / A.ncap;
    r.per = blocks ? (((cols + blocks - 1) / blocks + 15) & ~15) : 16;
    r.rt = (cols + r.per - 1) / r.per;
    return r;
}

// Walks the CTA's tiles.
struct Walk {
    Req q;
    int b, h, rt, t;
    __device__ __forceinline__ void start(const StepArgs &A, int b_, long long off) {
        b = b_;
        q = load_req(A, b);
        const int per_head = q.rt * q.nt;
        h = int(off / per_head);
        const int rem = int(off % per_head);
        rt = rem / q.nt;
        t = rem % q.nt;
    }
    // To the next tile; the caller stops after the last one.
    __device__ __forceinline__ void next(const StepArgs &A) {
        if (++t < q.nt) return;
        t = 0;
        if (++rt < q.rt) return;
        rt = 0;
        if (++h < A.Hkv) return;
        h = 0;
        do {
            if (++b >= A.B) { b = A.B - 1; return; }
            q = load_req(A, b);
        } while (q.rt == 0);
    }
    __device__ __forceinline__ int c0() const { return rt * q.per; }
    __device__ __forceinline__ int ncols(const StepArgs &A) const { return min(q.per, q.n * A.G - c0()); }
};

struct Ctrl {
    uint64_t full[kMaxSlots], empty[kMaxSlots];
    uint64_t q_full, s_full, p_full, pv_done, drained;
    uint32_t tmem;
    int gave_up, poison;
    long long warp_total[kThreadsStep / 32];
    long long total, start_base;
    int start_b;
    alignas(16) uint32_t bad[kWords][4];  // keys of a tile whose page is no memory
    alignas(16) float ref[kMaxCols];
    alignas(16) float fac[kMaxCols];
    alignas(16) float colmax[4][kMaxCols];
};

__device__ __forceinline__ void soft_sync() { asm volatile("barrier.cta.sync 1, 128;" ::: "memory"); }
__device__ __forceinline__ bool soft_any(bool x) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 q, %1, 0;\n\t"
        "barrier.cta.red.or.pred p, 1, 128, q;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r) : "r"(uint32_t(x)) : "memory");
    return r != 0;
}

__device__ __forceinline__ void st_shared16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
                 : "memory");
}
__device__ __forceinline__ uint4 ld_shared16(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}
// Does either half of the word hold a NaN or an infinity?
__device__ __forceinline__ uint32_t nonfinite_mask(uint32_t w) {
    uint32_t m = 0;
    if ((w & 0x7f80u) == 0x7f80u) m |= 0xffffu;
    if ((w & 0x7f800000u) == 0x7f800000u) m |= 0xffff0000u;
    return m;
}

// The columns [lo, hi) of the block that see the key at `kpos`.
__device__ __forceinline__ void visible_columns(const StepArgs &A, const Walk &w, int c0, int ncols,
                                                int kpos, bool bad, int &lo, int &hi) {
    lo = min(max(max(kpos - w.q.pos0, 0) * A.G - c0, 0), ncols);
    hi = ncols;
    if (A.window > 0) {
        const long long j = (long long)kpos - w.q.pos0 + A.window;  // rows below see it
        hi = int(min(max(min(j, (long long)w.q.n) * A.G - c0, 0ll), (long long)ncols));
    }
    if (bad || kpos < w.q.kbeg || kpos >= w.q.kend) hi = lo;
}

template <int D>
__global__ void __launch_bounds__(kThreadsStep, 1)
step_attention_kernel(const __grid_constant__ StepArgs A, const __grid_constant__ CUtensorMap k_map,
                      const __grid_constant__ CUtensorMap v_map) {
    constexpr int kHalves = D / 64;
    constexpr uint32_t kHalfBytes = kTile * 128;
    constexpr uint32_t kSlotBytes = kHalves * kHalfBytes;
    extern __shared__ uint8_t dyn[];
    __shared__ Ctrl C;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the join waits for this grid's end

    // Shared memory: ring, P, Q, ones.
    const uint32_t base = (smem_addr(dyn) + 1023) & ~1023u;
    const uint32_t ring = base;
    const uint32_t p_smem = ring + A.slots * kSlotBytes;
    const uint32_t p_groups = (A.ncap + 63) / 64;
    const uint32_t q_smem = p_smem + p_groups * kHalfBytes;
    const uint32_t q_half = A.ncap * 128;
    const uint32_t ones = q_smem + kHalves * q_half;

    // ---- set-up: barriers, TMEM, the constant operand, the CTA's tiles -----
    if (tid == 0) {
        for (int s = 0; s < A.slots; ++s) {
            mbar_init(&C.full[s], 1);
            mbar_init(&C.empty[s], 1);
        }
        mbar_init(&C.q_full, kSoftThreads);
        mbar_init(&C.s_full, 2);
        mbar_init(&C.p_full, 1);
        mbar_init(&C.pv_done, 1);
        mbar_init(&C.drained, 1);
        C.gave_up = 0;
        C.poison = 0;
        C.start_b = 0;
        C.start_base = 0;
        fence_barrier_init();
    }
    if (tid < 64) st_shared16(ones + tid * 16, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u);
    fence_async_shared();
    if (warp == 5) tmem_alloc(&C.tmem, kTmemCols);
    if (warp == 4 && lane == 0) {
        prefetch_map(&k_map);
        prefetch_map(&v_map);
    }

    const int per = (A.B + kThreadsStep - 1) / kThreadsStep;
    const int b_lo = min(tid * per, A.B), b_hi = min(b_lo + per, A.B);
    long long mine = 0;
    for (int b = b_lo; b < b_hi; ++b) {
        const Req r = load_req(A, b);
        mine += (long long)r.rt * r.nt * A.Hkv;
    }
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
    }
    if (lane == 31) C.warp_total[warp] = incl;
    __syncthreads();
    long long before = 0, total = 0;
    for (int w = 0; w < kThreadsStep / 32; ++w) {
        if (w < warp) before += C.warp_total[w];
        total += C.warp_total[w];
    }
    // every CTA that takes part has a tile
    const long long ctas = min((long long)gridDim.x, max(total, 1ll)), me = blockIdx.x;
    const long long start = me < ctas ? total * me / ctas : total;
    const long long end = me < ctas ? total * (me + 1) / ctas : total;
    const long long excl = before + incl - mine;
    if (start < end && excl <= start && start < excl + mine) {
        long long at = excl;
        for (int b = b_lo; b < b_hi; ++b) {
            const Req r = load_req(A, b);
            const long long x = (long long)r.rt * r.nt * A.Hkv;
            if (start < at + x) {
                C.start_b = b;
                C.start_base = at;
                break;
            }
            at += x;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const int left = int(end - start);
    const uint32_t tmem = C.tmem;
    Walk w;
    if (left > 0) w.start(A, C.start_b, start - C.start_base);

    if (tid == 0) {
        // The unit that is cut before this CTA, for the join.
        CutInfo ci{};
        ci.last = -1;
        if (left > 0 && w.t > 0) {
            const long long u0 = start - w.t, u1 = u0 + w.q.nt;
            ci.first = int(((u0 + 1) * ctas - 1) / total);
            ci.last = int((u1 * ctas - 1) / total);
            const long long s0 = total * ci.first / ctas;
            ci.slot_first = s0 == u0 ? 2 * ci.first : 2 * ci.first + 1;
            ci.row0 = w.q.row0;
            ci.head0 = w.h * A.G;
            ci.c0 = w.c0();
            ci.ncols = w.ncols(A);
        }
        A.cut[me] = ci;
    }

    volatile int *gave_up = &C.gave_up;
    if (left > 0 && warp == 4) {
        // ---- producer: K and V tiles into the ring ---------------------------
        // A lane owns one TMA box of the tile (or four keys: gather), and
        // looks up its pages one tile ahead.
        struct Ids { int page[4]; };
        const int boxes = A.box ? kTile / A.box : 32;
        const int span = A.box ? A.box : 4;
        auto look_up = [&](const Walk &x, Ids &ids) {
            const int key0 = (x.q.t0 + x.t) * kTile + lane * span;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                ids.page[i] = -1;
                const int key = key0 + i;
                if ((i == 0 || !A.box) && lane < boxes) {
                    const int pi = key / A.page_size;
                    if (pi < A.max_pages && key0 < x.q.kend && key0 + span > x.q.kbeg)
                        ids.page[i] = A.block_table[(int64_t)x.b * A.max_pages + pi];
                }
            }
        };
        Ids ids;
        look_up(w, ids);
        int issued = 0;
        for (int i = 0; i < left; ++i) {
            Walk x = w;
            if (i + 1 < left) x.next(A);
            Ids ahead;
            look_up(x, ahead);

            const int key0 = (w.q.t0 + w.t) * kTile + lane * span;
            const bool here = lane < boxes && key0 < w.q.kend && key0 + span > w.q.kbeg;
            uint32_t bad_bits = 0;  // of the lane's keys (gather) or of the whole box
            int row[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                bool ok = ids.page[j] >= 0 && ids.page[j] < A.num_pages;
                if (!ok) bad_bits |= 1u << j;
                const int page = ok ? ids.page[j] : 0;  // masked; any memory will do
                row[j] = A.box ? page
                               : page * A.page_rows + w.h * A.head_rows + (key0 + j) % A.page_size;
            }
            const int slot_in_page = A.box ? key0 % A.page_size : 0;
            const bool lane_bad = here && (A.box ? (bad_bits & 1) : bad_bits != 0);
            uint32_t words[4] = {0, 0, 0, 0};
            if (__any_sync(0xffffffffu, lane_bad)) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t m = 0;
                    if (lane_bad) {
                        if (A.box) {
                            const int lo = max(lane * span - 32 * q, 0), hi = min(lane * span + span - 32 * q, 32);
                            if (lo < hi) m = (hi - lo == 32 ? 0xffffffffu : ((1u << (hi - lo)) - 1u)) << lo;
                        } else if (lane / 8 == q) {
                            m = bad_bits << (4 * (lane % 8));
                        }
                    }
                    words[q] = __reduce_or_sync(0xffffffffu, m);
                }
            }
            const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, here)) * uint32_t(span) * D * 2;
            bool ok = true;
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
                const int s = issued % A.slots;
                if (issued >= A.slots)
                    ok = wait_or_give_up(&C.empty[s], (issued / A.slots - 1) & 1, A.wait_ns, gave_up);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                if (lane == 0) {
                    if (kv == 0)
                        for (int q = 0; q < 4; ++q) C.bad[i % kWords][q] = words[q];
                    mbar_arrive_expect_tx(&C.full[s], bytes);
                }
                __syncwarp();
                if (here) {
                    const CUtensorMap *map = kv ? &v_map : &k_map;
                    const uint32_t dst = ring + s * kSlotBytes + lane * span * 128;
#pragma unroll
                    for (int hf = 0; hf < kHalves; ++hf) {
                        if (A.box)
                            tma_load_4d(dst + hf * kHalfBytes, map, &C.full[s], hf * 64, slot_in_page,
                                        w.h, row[0]);
                        else
                            tma_gather4(dst + hf * kHalfBytes, map, &C.full[s],
                                        w.h * A.head_x + hf * 64, row[0], row[1], row[2], row[3]);
                    }
                }
                ++issued;
            }
            if (!ok) break;
            w = x;
            ids = ahead;
        }
        if (C.gave_up) {
            // Let the copies in flight land before the CTA ends.
            for (int k = max(issued - A.slots, 0); k < issued; ++k)
                mbar_wait_bounded(&C.full[k % A.slots], (k / A.slots) & 1, kDrainTimeoutNs);
        }
    } else if (left > 0 && warp == 5) {
        // ---- MMA issuer -----------------------------------------------------
        if (lane == 0) {
            const uint32_t s_tm = tmem + kColS, o_tm = tmem + kColO, l_tm = tmem + kColL;
            bool first = true, ok = true;
            int unit = 0;
            const uint64_t ones_desc = smem_desc(ones, 0, 0);
            for (int i = 0; i < left; ++i) {
                const int N = (w.ncols(A) + 15) & ~15;
                const uint32_t id_s = mma_idesc(128, N, false, false);
                const uint32_t id_o = mma_idesc(128, N, true, true);
                const uint32_t id_l = mma_idesc(128, N, false, true);
                const int ks = (2 * i) % A.slots, vs = (2 * i + 1) % A.slots;
                if (first) ok = wait_or_give_up(&C.q_full, unit & 1, A.wait_ns, gave_up);
                ok = ok && wait_or_give_up(&C.full[ks], ((2 * i) / A.slots) & 1, A.wait_ns, gave_up);
                if (!ok) break;
                tc_fence_after();
                mbar_arrive(&C.s_full);  // passes the producer's words on
                const uint32_t kb = ring + ks * kSlotBytes;
#pragma unroll
                for (int d = 0; d < D / 16; ++d) {
                    const uint32_t in = (d % 4) * 32;
                    mma_ss(s_tm, smem_desc(kb + (d / 4) * kHalfBytes + in, 16, 1024),
                           smem_desc(q_smem + (d / 4) * q_half + in, 16, 1024), id_s, d > 0);
                }
                mma_commit(&C.empty[ks]);
                mma_commit(&C.s_full);
                ok = wait_or_give_up(&C.p_full, i & 1, A.wait_ns, gave_up) &&
                     wait_or_give_up(&C.full[vs], ((2 * i + 1) / A.slots) & 1, A.wait_ns, gave_up);
                if (!ok) break;
                tc_fence_after();
                const uint32_t vb = ring + vs * kSlotBytes;
                // D = 64: the second group of 64 rows repeats the first
                const uint32_t v_lbo = kHalves == 2 ? kHalfBytes : 0;
#pragma unroll
                for (int k = 0; k < kTile / 16; ++k) {
                    const uint64_t pd = smem_desc(p_smem + k * 2048, kHalfBytes, 1024);
                    mma_ss(o_tm, smem_desc(vb + k * 2048, v_lbo, 1024), pd, id_o, !(first && k == 0));
                    mma_ss(l_tm, ones_desc, pd, id_l, !(first && k == 0));
                }
                mma_commit(&C.empty[vs]);
                mma_commit(&C.pv_done);
                const int t = w.t;
                if (i + 1 < left) w.next(A);
                first = w.t != t + 1;
                if (first) ++unit;
            }
            if (C.gave_up) {
                mma_commit(&C.drained);
                mbar_wait_bounded(&C.drained, 0, kDrainTimeoutNs);
            }
        }
        __syncwarp();
    } else if (left > 0) {
        // ---- softmax: thread = key of the tile ---------------------------------
        const uint32_t lane_tm = tmem + (uint32_t(warp * 32) << 16);
        bool first = true;
        int unit = 0, unit_tile0 = 0;
        bool ok = true;
        for (int i = 0; i < left; ++i) {
            const int c0 = w.c0(), ncols = w.ncols(A), N = (ncols + 15) & ~15;
            if (first) {
                unit_tile0 = w.t;
                // The block's queries, K-major; columns past the last are zeros.
                constexpr int kChunks = D / 8;
                for (int e = tid; e < N * kChunks; e += kSoftThreads) {
                    const int n = e / kChunks, ch = e % kChunks;
                    uint4 x = make_uint4(0, 0, 0, 0);
                    if (n < ncols) {
                        const int c = c0 + n, j = c / A.G, g = c - j * A.G;
                        x = *reinterpret_cast<const uint4 *>(
                            A.q + ((int64_t)(w.q.row0 + j) * A.Hq + w.h * A.G + g) * D + ch * 8);
                    }
                    st_shared16(q_smem + (ch / 8) * q_half + n * 128 + (((ch % 8) ^ (n & 7)) << 4),
                                x.x, x.y, x.z, x.w);
                }
                fence_async_shared();
                mbar_arrive(&C.q_full);
            }
            ok = wait_or_give_up(&C.s_full, i & 1, A.wait_ns, gave_up);
            if (ok && !first) ok = wait_or_give_up(&C.pv_done, (i - 1) & 1, A.wait_ns, gave_up);
            if (soft_any(!ok)) break;
            tc_fence_after();

            const int kbase = (w.q.t0 + w.t) * kTile, kpos = kbase + tid;
            const uint4 bw = *reinterpret_cast<const uint4 *>(C.bad[i % kWords]);
            const int jmin = c0 / A.G, jmax = (c0 + ncols - 1) / A.G;
            const bool whole = (bw.x | bw.y | bw.z | bw.w) == 0 && kbase >= w.q.kbeg &&
                               kbase + kTile <= w.q.kend && kbase + kTile - 1 <= w.q.pos0 + jmin &&
                               (A.window == 0 || (long long)kbase > (long long)w.q.pos0 + jmax - A.window);
            int lo = 0, hi = N;
            if (!whole) {
                const uint32_t word = warp == 0 ? bw.x : warp == 1 ? bw.y : warp == 2 ? bw.z : bw.w;
                visible_columns(A, w, c0, ncols, kpos, (word >> lane) & 1, lo, hi);
                // Masked keys must not reach O through 0 * infinity: a value
                // row that no column sees is cleared, and one that some
                // columns see loses its NaN and infinities, which the
                // epilogue adds to the columns that do see them.
                const int vs = (2 * i + 1) % A.slots;
                ok = wait_or_give_up(&C.full[vs], ((2 * i + 1) / A.slots) & 1, A.wait_ns, gave_up);
                if (soft_any(!ok)) break;
                if (lo > 0 || hi < ncols) {
                    const uint32_t vb = ring + vs * kSlotBytes + tid * 128;
                    for (int ch = 0; ch < 8 * kHalves; ++ch) {
                        const uint32_t at = vb + (ch / 8) * kHalfBytes + (((ch % 8) ^ (tid & 7)) << 4);
                        if (lo >= hi) {
                            st_shared16(at, 0, 0, 0, 0);
                            continue;
                        }
                        const uint4 x = ld_shared16(at);
                        const uint32_t mx = nonfinite_mask(x.x), my = nonfinite_mask(x.y),
                                       mz = nonfinite_mask(x.z), mw = nonfinite_mask(x.w);
                        if (mx | my | mz | mw) {
                            st_shared16(at, x.x & ~mx, x.y & ~my, x.z & ~mz, x.w & ~mw);
                            C.poison = 1;
                        }
                    }
                }
            }

            // Weights of the tile against the reference; a unit's first tile
            // sets the reference before, a tile that passes it moves it.
            bool move = first;
            for (;;) {
                if (move) {
                    for (int n = 0; n < N; n += 16) {
                        float s[16];
                        tmem_ld16(s, lane_tm + kColS + n);
                        tmem_wait_ld(s);
                        float keep = 0.f;
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            float x = s[e] * A.scale2;
                            if (n + e < lo || n + e >= hi) x = -INFINITY;
                            asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(x) : "f"(x));
                            if (lane == e) keep = x;
                        }
                        if (lane < 16) C.colmax[warp][n + lane] = keep;
                    }
                    soft_sync();
                    for (int n = tid; n < N; n += kSoftThreads) {
                        const float old = first ? kRefMin : C.ref[n];
                        const float now = fmaxf(fmaxf(fmaxf(C.colmax[0][n], C.colmax[1][n]),
                                                      fmaxf(C.colmax[2][n], C.colmax[3][n])), old);
                        C.ref[n] = n < ncols ? now : 0.f;  // the zero columns' scores
                        C.fac[n] = exp2_approx(old - now);
                    }
                    soft_sync();
                    if (!first) {
                        for (int n = 0; n < N; n += 16) {
                            float o[16], l[16];
                            tmem_ld16(o, lane_tm + kColO + n);
                            tmem_ld16(l, lane_tm + kColL + n);
                            tmem_wait_ld(o);
                            tmem_use16(l);
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                o[e] *= C.fac[n + e];
                                l[e] *= C.fac[n + e];
                            }
                            tmem_st16(lane_tm + kColO + n, o);
                            tmem_st16(lane_tm + kColL + n, l);
                        }
                        tmem_wait_st();
                    }
                }
                float top = 0.f;
                for (int n = 0; n < N; n += 16) {
                    float s[16];
                    tmem_ld16(s, lane_tm + kColS + n);
                    float ref[16];
#pragma unroll
                    for (int e = 0; e < 16; e += 4)
                        *reinterpret_cast<float4 *>(ref + e) = *reinterpret_cast<const float4 *>(C.ref + n + e);
                    tmem_wait_ld(s);
                    uint32_t p[8];
#pragma unroll
                    for (int e = 0; e < 16; e += 2) {
                        float x = fmaf(s[e], A.scale2, -ref[e]), y = fmaf(s[e + 1], A.scale2, -ref[e + 1]);
                        if (!whole) {
                            if (n + e < lo || n + e >= hi) x = -INFINITY;
                            if (n + e + 1 < lo || n + e + 1 >= hi) y = -INFINITY;
                        }
                        top = fmaxf(top, fmaxf(x, y));
                        p[e / 2] = pack_bf16x2(exp2_approx(x), exp2_approx(y));
                    }
                    const uint32_t at = p_smem + (n / 64) * kHalfBytes + tid * 128;
                    const int ch = (n % 64) / 8;
                    st_shared16(at + ((ch ^ (tid & 7)) << 4), p[0], p[1], p[2], p[3]);
                    st_shared16(at + (((ch + 1) ^ (tid & 7)) << 4), p[4], p[5], p[6], p[7]);
                }
                fence_async_shared();
                tc_fence_before();
                move = soft_any(top > kRefSlack);
                if (!move) break;
                first = false;  // O and L hold earlier tiles, or nothing that counts yet
            }
            if (tid == 0) mbar_arrive(&C.p_full);

            // ---- the unit's end in this CTA ----------------------------------
            const Walk u = w;
            if (i + 1 < left) w.next(A);
            const bool done = i + 1 == left || w.t != u.t + 1;
            first = done;
            if (!done) continue;
            ++unit;
            ok = wait_or_give_up(&C.pv_done, i & 1, A.wait_ns, gave_up);
            if (soft_any(!ok)) break;
            tc_fence_after();
            const bool split = unit_tile0 > 0 || u.t + 1 < u.q.nt;
            const int d = D == 128 ? tid : tid % 64;
            const bool writer = tid < D;
            // the unit at the CTA's start uses the first of its two slots
            const int slot = 2 * int(me) + (unit == 1 ? 0 : 1);
            const bool poison = C.poison;
            int j = u.c0() / A.G, g = u.c0() % A.G;
            uint16_t *out = A.out + ((int64_t)(u.q.row0 + j) * A.Hq + u.h * A.G + g) * D + d;
            float *part = A.part + (int64_t)slot * A.ncap * D + d;
            for (int n = 0; n < N; n += 16) {
                float o[16], l[16];
                tmem_ld16(o, lane_tm + kColO + n);
                tmem_ld16(l, lane_tm + kColL + n);
                tmem_wait_ld(o);
                tmem_use16(l);
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    if (n + e >= ncols) break;
                    float x = o[e];
                    if (poison) {
                        // keys of this CTA's tiles that some columns see and others do not
                        const int k0 = max((u.q.t0 + unit_tile0) * kTile, u.q.kbeg);
                        const int k1 = min((u.q.t0 + u.t + 1) * kTile, u.q.kend);
                        for (int key = k0; key < k1; ++key) {
                            int vlo, vhi;
                            visible_columns(A, u, u.c0(), ncols, key, false, vlo, vhi);
                            if (vlo == 0 && vhi == ncols) continue;
                            if (n + e < vlo || n + e >= vhi) continue;
                            const int page = A.block_table[(int64_t)u.b * A.max_pages + key / A.page_size];
                            if (page < 0 || page >= A.num_pages) continue;
                            const float v = bf16_lo(A.v_cache[page * A.page_stride + (key % A.page_size) * A.slot_stride +
                                                              u.h * A.head_stride + d]);
                            if (!isfinite(v)) x += v;
                        }
                    }
                    if (split) {
                        if (writer) part[(int64_t)(n + e) * D] = x;
                        if (tid == 0) {
                            A.stat[((int64_t)slot * 2) * A.ncap + n + e] = C.ref[n + e];
                            A.stat[((int64_t)slot * 2 + 1) * A.ncap + n + e] = l[e];
                        }
                    } else {
                        const float y = l[e] == 0.f ? 0.f : x / l[e];
                        if (writer) *out = uint16_t(pack_bf16x2(y, 0.f));
                    }
                    out += D;
                    if (++g == A.G) {
                        g = 0;
                        out += (int64_t)(A.Hq - A.G) * D;
                    }
                }
            }
            tc_fence_before();
            soft_sync();  // ref, poison and O are read before the next unit writes them
            if (tid == 0) C.poison = 0;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (tid == 0 && C.gave_up) atomicOr(A.status, kStatusWaitTimeout);
    if (warp == 5) tmem_free(tmem, kTmemCols);
}

// Adds the partial sums of the units that were cut, in the order of the keys.
// CTA i takes its share of the columns of the unit that is cut before CTA i;
// a warp takes a column.
template <int D>
__global__ void __launch_bounds__(kJoinThreads) step_join_kernel(const StepArgs A) {
    constexpr int E = D / 32;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int me = blockIdx.x + 1, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const CutInfo ci = A.cut[me];
    if (ci.last < me) return;
    const int members = ci.last - ci.first + 1;
    const int cuts = members - 1, rank = me - ci.first - 1;
    const int n0 = int((long long)ci.ncols * rank / cuts), n1 = int((long long)ci.ncols * (rank + 1) / cuts);
    for (int n = n0 + warp; n < n1; n += kJoinThreads / 32) {
        float m = kRefMin;
        for (int k = lane; k < members; k += 32) {
            const int slot = k == 0 ? ci.slot_first : 2 * (ci.first + k);
            m = fmaxf(m, A.stat[(int64_t)slot * 2 * A.ncap + n]);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        float acc[E], l = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = 0.f;
        for (int k0 = 0; k0 < members; k0 += 32) {
            float wk = 0.f, lk = 0.f;
            if (k0 + lane < members) {
                const int k = k0 + lane, slot = k == 0 ? ci.slot_first : 2 * (ci.first + k);
                wk = exp2_approx(A.stat[(int64_t)slot * 2 * A.ncap + n] - m);
                lk = A.stat[((int64_t)slot * 2 + 1) * A.ncap + n];
            }
            const int here = min(32, members - k0);
#pragma unroll 8
            for (int k = 0; k < here; ++k) {
                const float f = __shfl_sync(0xffffffffu, wk, k);
                l += f * __shfl_sync(0xffffffffu, lk, k);
                const int slot = k0 + k == 0 ? ci.slot_first : 2 * (ci.first + k0 + k);
                const float *p = A.part + ((int64_t)slot * A.ncap + n) * D + lane * E;
#pragma unroll
                for (int e = 0; e < E; ++e) acc[e] += f * p[e];
            }
        }
        const int c = ci.c0 + n, j = c / A.G, g = c - j * A.G;
        uint32_t *out = reinterpret_cast<uint32_t *>(A.out + ((int64_t)(ci.row0 + j) * A.Hq + ci.head0 + g) * D + lane * E);
        const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
        for (int e = 0; e < E; e += 2) out[e / 2] = pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
    }
}

int step_columns(int Hq, int Hkv, int q_max) {
    const long long cols = (long long)q_max * (Hq / Hkv);
    return int(std::min<long long>((cols + 15) / 16 * 16, kMaxCols));
}

constexpr size_t kHeaderBytes = 256 + (sizeof(CutInfo) * kAttnMaxCtas + 255) / 256 * 256;

template <int D>
cudaError_t launch(StepArgs A, const CUtensorMap &km, const CUtensorMap &vm, int ctas, cudaStream_t s) {
    const size_t slot = size_t(D) * 2 * kTile;
    const size_t fixed = 2048 + size_t((A.ncap + 63) / 64) * kTile * 128 + size_t(A.ncap) * D * 2;
    const size_t room = 232448 - sizeof(Ctrl) - 256 - fixed;
    A.slots = int(std::min<size_t>(room / slot, kMaxSlots));
    const size_t smem = fixed + A.slots * slot;
    cudaError_t e = cudaFuncSetAttribute(step_attention_kernel<D>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
    if (e != cudaSuccess) return e;
    step_attention_kernel<D><<<ctas, kThreadsStep, smem, s>>>(A, km, vm);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if (ctas == 1) return cudaSuccess;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(ctas - 1);
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = s;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, step_join_kernel<D>, A);
}

int gcd(int a, int b) { return b ? gcd(b, a % b) : a; }

}  // namespace

size_t attn_workspace_bytes(int Hq, int Hkv, int D, int q_max) {
    if (q_max > DSPARK_MAX_STEP_ROWS) return kHeaderBytes;  // dspark_prompt_attention's
    const size_t cols = size_t(step_columns(Hq, Hkv, q_max));
    return kHeaderBytes + align256(2 * kAttnMaxCtas * cols * D * sizeof(float)) +
           align256(2 * kAttnMaxCtas * 2 * cols * sizeof(float));
}

static bool step_gather_rows(const dspark_attn &a, int64_t *row, int64_t *page_rows, int64_t *head_rows,
                      int64_t *head_x) {
    *row = a.page_size > 1 ? a.slot_stride : a.page_stride;
    if (a.page_stride % *row) return false;
    *page_rows = a.page_stride / *row;
    *head_rows = *head_x = 0;
    if (a.Hkv > 1) {
        if (a.head_stride % *row == 0) *head_rows = a.head_stride / *row;
        else if ((a.Hkv - 1) * a.head_stride + a.D <= *row) *head_x = a.head_stride;
        else return false;
    }
    const int64_t last = (a.num_pages - 1) * *page_rows + (a.Hkv - 1) * *head_rows + a.page_size;
    return *row >= a.D && last <= INT32_MAX;
}

bool step_strides_ok(const dspark_attn &a) {
    int64_t row, page_rows, head_rows, head_x;
    return gcd(a.page_size, kTile) >= 8 || step_gather_rows(a, &row, &page_rows, &head_rows, &head_x);
}

cudaError_t launch_step_attention(const dspark_attn &a, int sms, uint64_t wait_ns, cudaStream_t s) {
    StepArgs A{};
    A.B = a.B; A.rows = a.rows; A.q_max = a.q_max; A.Hq = a.Hq; A.Hkv = a.Hkv; A.G = a.Hq / a.Hkv;
    A.page_size = a.page_size; A.num_pages = a.num_pages; A.max_pages = a.max_pages;
    A.window = a.window;
    A.ncap = step_columns(a.Hq, a.Hkv, a.q_max);
    A.scale2 = float(double(a.scale) * 1.4426950408889634);
    A.page_stride = a.page_stride; A.slot_stride = a.slot_stride; A.head_stride = a.head_stride;
    A.q = static_cast<const uint16_t *>(a.q_rot);
    A.v_cache = static_cast<const uint16_t *>(a.v_cache);
    A.row_off = a.row_off; A.seq_lens = a.seq_lens; A.block_table = a.block_table;
    A.out = static_cast<uint16_t *>(a.out);
    char *ws = static_cast<char *>(a.workspace);
    A.status = reinterpret_cast<int32_t *>(ws);
    A.cut = reinterpret_cast<CutInfo *>(ws + 256);
    A.part = reinterpret_cast<float *>(ws + kHeaderBytes);
    A.stat = reinterpret_cast<float *>(ws + kHeaderBytes +
                                       align256(2 * kAttnMaxCtas * size_t(A.ncap) * a.D * sizeof(float)));
    A.wait_ns = wait_ns;

    // A page of 8 k positions is copied in boxes of whole pages or parts of
    // them; other pages key by key (four keys a copy).
    CUtensorMap maps[2];
    const int box = gcd(a.page_size, kTile);
    const void *bases[2] = {a.k_cache, a.v_cache};
    if (box >= 8) {
        A.box = box;
        const uint64_t dims[4] = {uint64_t(a.D), uint64_t(a.page_size), uint64_t(a.Hkv), uint64_t(a.num_pages)};
        const uint64_t st[3] = {uint64_t(a.slot_stride) * 2, uint64_t(a.head_stride) * 2, uint64_t(a.page_stride) * 2};
        const uint32_t bx[4] = {64, uint32_t(box), 1, 1};
        for (int i = 0; i < 2; ++i) {
            const cudaError_t e = encode_map(&maps[i], bases[i], 4, dims, st, bx);
            if (e != cudaSuccess) return e;
        }
    } else {
        int64_t row, page_rows, head_rows, head_x;
        if (!step_gather_rows(a, &row, &page_rows, &head_rows, &head_x)) return cudaErrorInvalidValue;
        A.page_rows = int(page_rows);
        A.head_rows = int(head_rows);
        A.head_x = int(head_x);
        const uint64_t dims[2] = {uint64_t((head_x ? (a.Hkv - 1) * head_x : 0) + a.D),
                                  uint64_t((a.num_pages - 1) * page_rows + (a.Hkv - 1) * head_rows + a.page_size)};
        const uint64_t st[1] = {uint64_t(row) * 2};
        const uint32_t bx[2] = {64, 1};
        for (int i = 0; i < 2; ++i) {
            const cudaError_t e = encode_map(&maps[i], bases[i], 2, dims, st, bx);
            if (e != cudaSuccess) return e;
        }
    }
    const int ctas = std::min(sms, kAttnMaxCtas);
    return a.D == 128 ? launch<128>(A, maps[0], maps[1], ctas, s) : launch<64>(A, maps[0], maps[1], ctas, s);
}

}  // namespace dspark
