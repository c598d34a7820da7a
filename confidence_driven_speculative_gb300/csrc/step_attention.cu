// step_attention.cu -- the step's rows over the paged cache.
//
// Mathematics.  One request and one cached head give a block of
// cols = rows * G query vectors (G query heads share the cached head) over the
// request's keys.  The keys are walked in tiles of 128 with a running
// reference m and, per column, o = sum p v and l = sum p of the weights
// p = 2^(scale * log2(e) * (q.k - m)); the output is o / l.
//
// Layout.  A step has few columns (4 to a few tens) and many keys, so the
// products are taken transposed: the 128 keys of a tile are the M side of the
// tensor core, the columns the N side, padded only to a multiple of 16:
//     S^T [128 keys x N]  = K [128 x D] Q^T          (K and Q K-major)
//     O^T [D x N]        += V^T [D x 128] P^T        (V and P MN-major)
//     L   [D x N]        += 1 [D x 128] P^T          (sum of the rounded weights)
// S, O and L live in TMEM.  A softmax thread owns one key and, of a tile's
// columns, every fourth group of 16: four groups of 128 threads share a tile
// (with two groups, in an earlier version: 71 us against 66 for 32 requests of 17
// rows).
//
// The reference lies 2^16 of a weight above the first tile's maximum and moves
// only when some score passes it (with 2^8: window 85.4 us against 83.8).  So no
// weight passes 1, and O overflows only where the values' own sum does; a column's
// largest weight is 2^-16 or about that, which fp32 sums and bfloat16 hold with an
// unchanged relative step.  An ordinary tile needs no reduction over keys, only
// the threads' vote that nothing passed.  Weights are rounded to bfloat16 for the
// tensor core, by a relative 2^-8 at most, and L sums the rounded ones, so
// that the errors of numerator and denominator partly cancel.
//
// Bound: bytes of the cache.  One persistent CTA per SM (four softmax groups
// want its registers) keeps a ring of K and V tiles, 128 keys each, filled by TMA.
// The K producer, the V producer and a third that shares both look up pages a
// tile ahead.  A page of 8 k positions goes in boxes of whole pages or parts of
// them.  Other pages are gathered four keys a copy: 31 clocks per 512 bytes
// whichever warp issues them, at most 70 % of a copy's rate; copies by the
// lanes themselves were slower (in an earlier version 123 us against 89 for the
// windowed case below).
//
// Split.  The tiles of all (request, cached head, block of rows) units form
// one list, cut evenly over the CTAs; a unit counts for two tiles more than it
// has, what its start and end cost (when that came in, a CTA's time went from 42
// to 85 us to 49 to 61).  The cut points come from a scan of the lengths in every CTA, on
// the device.  A unit that is cut leaves partial (o, m, l) in the workspace,
// in fp32, and the CTA that writes its last part adds them in the order of the
// keys: the result does not depend on timing.
//
// Measured, 8 cached heads of 128, against the cache's bytes at a copy's 6.79
// TB/s: 256 requests of 16 to 4095 keys with 1 to 7 rows of 32 heads 311 to
// 319 us (floor 297); 2 of 131 000 keys with 9 rows of 64 heads 171 (158); 32
// of 16 to 4095 keys with 17 rows 62.5 (42); one row over 4096 keys 13.3 (2.5);
// 64 requests with a window of 1024 over single-position pages 84.5 (39).
// Long caches run at the memory's rate.  Otherwise a unit's end costs what two
// to three tiles do (the wait for its last product, the outputs, the fences of
// its parts), and one request alone is a chain of latencies: launch, cut, tile,
// join.
#include <algorithm>
#include <type_traits>

#include "attn.cuh"
#include "dspark_internal.cuh"
#include "tcgen05.cuh"

namespace dspark {
namespace {

constexpr int kTile = 128;      // keys of a tile
constexpr int kMaxCols = 160;   // columns of a unit: S, O and L take 3 x 160 of 512 TMEM columns
constexpr int kTwoS = 128;      // up to so many, S is held twice
constexpr uint32_t kPGroup = kTile * 32;  // P: 16 columns of 128 keys, rows of 32 bytes
constexpr int kMaxSlots = 12;   // ring slots (one K or one V tile each)
constexpr int kWords = 16;      // ring of the tiles' bad-key words
constexpr int kGroups = 4;          // softmax groups of 128 threads: each takes every fourth 16 columns
constexpr int kSoftThreads = kGroups * kTile;
constexpr int kWarpK = 16, kWarpV = 17, kWarpBoth = 18, kWarpMma = 19;
constexpr int kThreadsStep = 640;
constexpr uint32_t kTmemCols = 512;
constexpr float kRefMin = -3.402823466e38f;  // reference of a column without a score yet: no score is lower
constexpr float kHeadroom = 16.0f; // log2: the reference over the maximum that sets it
constexpr int kWarpScan = 128;         // up to so many requests, every warp finds the cut by itself
constexpr int kUnitCost = 2;           // what a unit costs beside its tiles, in tiles
constexpr size_t kSmemBytes = 232448;  // shared memory of a CTA

struct StepArgs {
    int B, rows, q_max, Hq, Hkv, G;
    int page_size, num_pages, max_pages, window;
    uint32_t page_mul, page_shift;  // position / page_size = position * mul >> shift
    int box;                   // keys of a TMA box (divides the page and the tile); 0: gather
    int ncap;                  // columns of a unit at most, a multiple of 16
    int rows_cap;              // rows of a unit at most
    int unit_cost;             // what a unit costs beside its tiles, in tiles
    int slots, k_slots;        // ring slots; the first k_slots hold K tiles, the others V tiles
    int two_s, two_p, two_q;   // S, P, Q held twice
    int page_rows, head_rows;  // gather: rows of the 2-D view per page and head
    int head_x;                // gather: entries of a row per head
    float scale2;              // scale * log2(e)
    float headroom;            // kHeadroom in scores q.k
    int64_t page_stride, slot_stride, head_stride;
    const uint16_t *v_cache;
    const int32_t *row_off, *seq_lens, *block_table;
    uint16_t *out;
    float *part;               // [2 * CTAs][ncap][D]
    float *stat;               // [2 * CTAs][2][ncap]: reference, sum
    int32_t *arrived;          // [CTAs] parts written of the unit that CTA i is the first of
    int32_t *status;
    uint64_t wait_ns;
};

// A request's block of work.
struct Req {
    int row0, n;     // packed rows
    int pos0;        // position of the first one
    int kbeg, kend;  // keys that some row sees
    int t0, nt;      // tiles
    int blocks, per; // blocks of rows, rows of one
};

__device__ __forceinline__ int page_of(const StepArgs &A, int pos) {
    return int((uint64_t(uint32_t(pos)) * A.page_mul) >> A.page_shift);
}

__device__ __forceinline__ Req load_req(const StepArgs &A, int b) {
    Req r;
    const int a0 = A.row_off[b], a1 = A.row_off[b + 1];
    r.row0 = min(max(a0, 0), A.rows);
    r.n = min(min(max(a1, r.row0), A.rows) - r.row0, A.q_max);
    // far past any table, where nothing is seen, stays in 32 bits
    r.pos0 = A.seq_lens ? min(max(A.seq_lens[b], 0), INT32_MAX - 65536) : 0;
    const int cap = A.max_pages * A.page_size;
    r.kend = min(r.pos0 + r.n, cap);
    r.kbeg = A.window > 0 ? min(max(r.pos0 - A.window + 1, 0), r.kend) : 0;
    r.t0 = r.kbeg / kTile;
    r.nt = max((r.kend + kTile - 1) / kTile - r.t0, 1);
    r.per = r.n;
    r.blocks = r.n > 0;
    if (r.n > A.rows_cap) {
        r.blocks = (r.n + A.rows_cap - 1) / A.rows_cap;
        r.per = (r.n + r.blocks - 1) / r.blocks;
        r.blocks = (r.n + r.per - 1) / r.per;
    }
    return r;
}

// One (request, cached head, block of rows), and walking to the next.
struct Unit {
    Req q;
    int b, h, blk;
    int j0, ncols;  // first row of the block, its columns

    __device__ __forceinline__ void shape(const StepArgs &A) {
        j0 = blk * q.per;
        ncols = min(q.per, q.n - j0) * A.G;
    }
    // Unit `i` of request b's list.
    __device__ __forceinline__ void start(const StepArgs &A, int b_, const Req &q_, int i) {
        b = b_;
        q = q_;
        h = i / q.blocks;
        blk = i - h * q.blocks;
        shape(A);
    }
    __device__ __forceinline__ void next(const StepArgs &A) {
        if (++blk == q.blocks) {
            blk = 0;
            if (++h == A.Hkv) {
                h = 0;
                do {
                    if (++b >= A.B) { b = A.B - 1; return; }
                    q = load_req(A, b);
                } while (q.blocks == 0);
            }
        }
        shape(A);
    }
};

// A list of `total` places cut into parts of equal length, one place more to
// the first ones: CTA i has start(i) .. start(i + 1).  No part is empty before
// the last one that is not.
struct Cuts {
    int parts, each, more;
    Cuts() = default;
    __device__ __forceinline__ Cuts(int total, int ctas) {
        parts = min(ctas, max(total, 1));
        each = total / parts;
        more = total - each * parts;
    }
    __device__ __forceinline__ int start(int i) const {
        i = min(i, parts);
        return each * i + min(i, more);
    }
    __device__ __forceinline__ int of(int place) const {
        const int longer = (each + 1) * more;
        return place < longer ? place / (each + 1) : more + (place - longer) / each;
    }
};

// A unit that was cut and whose last part this CTA wrote: it joins the parts.
struct Join {
    int row0, head0, ncols;             // its first packed row, first query head, columns
    int slot0, first_cta, members;      // the first part's slot, the CTAs that share it
};

struct Ctrl {
    uint64_t full[kMaxSlots], empty[kMaxSlots];
    uint64_t q_full[2], q_empty[2], s_full[2];
    uint64_t p_full[2], pv_done[2], drained;
    uint32_t tmem;
    int issued[2][2], q_issued;  // copies: (by K's and V's warps, by the third) of K and V tiles; units' queries
    int gave_up, joins;
    int poison;  // the CTA's last unit, counted from 1, that lost values (a tag: nobody has to clear it)
    Join join[2];
    int warp_cost[kThreadsStep / 32], warp_units[kThreadsStep / 32];
    int tiles_before[2];  // tiles of the list before this CTA's and up to its last
    int start_b, start_unit, start_tile;
    alignas(16) int row[2][kTile];        // producers (the third shares K's): pages of the boxes, or rows of the keys
    alignas(16) uint32_t bad[2][kWords][4];  // (by K warp) keys of a tile whose page is no memory
    alignas(16) float ref[kMaxCols];
    alignas(16) float fac[kMaxCols];
};

__device__ __forceinline__ void soft_sync() { asm volatile("barrier.cta.sync 1, 512;" ::: "memory"); }
__device__ __forceinline__ bool soft_any(bool x) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 q, %1, 0;\n\t"
        "barrier.cta.red.or.pred p, 1, 512, q;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r) : "r"(uint32_t(x)) : "memory");
    return r != 0;
}

// Is phase `parity` of `bar` over?  One answer for the whole warp.
__device__ __forceinline__ bool warp_test(uint64_t *bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_test_wait(bar, parity));
}

// The columns [lo, hi) of the unit that see the key at `kpos`.
__device__ __forceinline__ void visible_columns(const StepArgs &A, const Unit &u, int kpos, bool bad,
                                                int &lo, int &hi) {
    lo = min(max(kpos - u.q.pos0 - u.j0, 0) * A.G, u.ncols);
    hi = u.ncols;
    if (A.window > 0) {
        const long long j = (long long)kpos - u.q.pos0 - u.j0 + A.window;  // rows below see it
        hi = int(min(max(min(j, (long long)u.q.n) * A.G, 0ll), (long long)u.ncols));
    }
    if (bad || kpos < u.q.kbeg || kpos >= u.q.kend) hi = lo;
}

// 16 columns of a tile, on their way from TMEM: weights 2^((s - ref) * scale2), rounded, to P; returns
// the largest exponent.  Columns whose bit of `seen` is clear weigh nothing.
template <bool kMasked>
__device__ __forceinline__ float weigh16(float (&s)[16], const float *ref, float scale2,
                                         uint32_t seen, uint32_t at, int swz) {
    float r[16];
#pragma unroll
    for (int e = 0; e < 16; e += 4)
        *reinterpret_cast<float4 *>(r + e) = *reinterpret_cast<const float4 *>(ref + e);
    tmem_wait_ld(s);
    uint32_t p[8];
    float top = 0.f;
#pragma unroll
    for (int e = 0; e < 16; e += 2) {
        // The difference comes first.  It is exact for scores near the reference, however far both lie from
        // 0; a fused s * scale2 - scaled reference is off by half a step of that reference, by more than
        // fp32's range from scores of 2^32 on (and 1 % faster: static 62.2 us against 62.8).
        float x = (s[e] - r[e]) * scale2, y = (s[e + 1] - r[e + 1]) * scale2;
        if (kMasked) {
            if (!((seen >> e) & 1)) x = -INFINITY;
            if (!((seen >> (e + 1)) & 1)) y = -INFINITY;
        }
        top = fmaxf(top, fmaxf(x, y));
        p[e / 2] = pack_bf16x2(exp2_approx(x), exp2_approx(y));
    }
    st_shared16(at + (swz << 4), p[0], p[1], p[2], p[3]);
    st_shared16(at + ((swz ^ 1) << 4), p[4], p[5], p[6], p[7]);
    return top;
}

// Bits of the columns n .. n + 15 that lie in [lo, hi).
__device__ __forceinline__ uint32_t seen16(int n, int lo, int hi) {
    const int a = min(max(lo - n, 0), 16), b = min(max(hi - n, 0), 16);
    return ((1u << b) - 1u) & ~((1u << a) - 1u);
}

// Adds the parts of a unit that was cut, in the order of the keys, on all warps of
// the CTA that wrote its part last.  A warp takes kCols
// columns at a time and asks for 4 / kCols parts of each before it knows
// their weights.  kCols > 1: all parts are there at once (members <= 4 / kCols).
template <int D, int kCols>
__device__ __forceinline__ void join_columns(const StepArgs &A, const Join &J, int warp, int lane) {
    constexpr int E = D / 32, kParts = 4 / kCols;
    using Vec = typename std::conditional<E == 4, float4, float2>::type;
    const int ncols = J.ncols, members = J.members;
    uint16_t *const out0 = A.out + ((int64_t)J.row0 * A.Hq + J.head0) * D;
    auto slot_of = [&](int k) { return k == 0 ? J.slot0 : 2 * (J.first_cta + k); };
    const int my_k = lane % kParts, my_c = lane / kParts;  // lanes 0..3: one part of one column
    for (int n0 = warp * kCols; n0 < ncols; n0 += kThreadsStep / 32 * kCols) {
        float m = kRefMin, acc[kCols][E], l[kCols];
#pragma unroll
        for (int c = 0; c < kCols; ++c) {
            l[c] = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) acc[c][e] = 0.f;
        }
        for (int k0 = 0; k0 < members; k0 += kParts) {
            Vec x[kCols][kParts];
#pragma unroll
            for (int c = 0; c < kCols; ++c)
#pragma unroll
                for (int k = 0; k < kParts; ++k)
                    if (k0 + k < members && n0 + c < ncols)
                        x[c][k] = __ldcg(reinterpret_cast<const Vec *>(
                            A.part + ((int64_t)slot_of(k0 + k) * A.ncap + n0 + c) * D + lane * E));
            float ref = kRefMin, sum = 0.f;
            if (my_c < kCols && k0 + my_k < members && n0 + my_c < ncols) {
                const float *st = A.stat + (int64_t)slot_of(k0 + my_k) * 2 * A.ncap + n0 + my_c;
                ref = __ldcg(st);
                sum = __ldcg(st + A.ncap);
            }
            float top = ref;
#pragma unroll
            for (int o = kParts / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            const float m_new = fmaxf(m, top);  // the lane's column's
            const float w = exp2_approx((ref - m_new) * A.scale2), f_old = exp2_approx((m - m_new) * A.scale2);
            m = m_new;
#pragma unroll
            for (int c = 0; c < kCols; ++c) {
                const float f = __shfl_sync(0xffffffffu, f_old, c * kParts);
                l[c] *= f;
#pragma unroll
                for (int e = 0; e < E; ++e) acc[c][e] *= f;
#pragma unroll
                for (int k = 0; k < kParts; ++k) {
                    const float wk = __shfl_sync(0xffffffffu, w, c * kParts + k);
                    const float lk = __shfl_sync(0xffffffffu, sum, c * kParts + k);
                    if (k0 + k < members && n0 + c < ncols) {
                        l[c] = fmaf(wk, lk, l[c]);
                        const float *v = reinterpret_cast<const float *>(&x[c][k]);
#pragma unroll
                        for (int e = 0; e < E; ++e) acc[c][e] = fmaf(wk, v[e], acc[c][e]);
                    }
                }
            }
        }
#pragma unroll
        for (int c = 0; c < kCols; ++c) {
            const int n = n0 + c;
            if (n >= ncols) break;
            uint32_t *out = reinterpret_cast<uint32_t *>(out0 + (int64_t)(n / A.G) * A.Hq * D + (n % A.G) * D + lane * E);
            const float inv = l[c] == 0.f ? 0.f : 1.f / l[c];
#pragma unroll
            for (int e = 0; e < E; e += 2) out[e / 2] = pack_bf16x2(acc[c][e] * inv, acc[c][e + 1] * inv);
        }
    }
}

// kBox: pages go in TMA boxes; else gathered key by key.  (One kernel for
// both: more code for every warp to fetch, 10 % slower at long caches.)
template <int D, bool kBox>
__global__ void __launch_bounds__(kThreadsStep, 1)
step_attention_kernel(const __grid_constant__ StepArgs A, const __grid_constant__ CUtensorMap q_map,
                      const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map) {
    constexpr int kHalves = D / 64;
    constexpr uint32_t kHalfBytes = kTile * 128;
    constexpr uint32_t kSlotBytes = kHalves * kHalfBytes;
    extern __shared__ uint8_t dyn[];
    __shared__ Ctrl C;
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = tid & 31;

    // Shared memory: ring, P and Q (once or twice), ones.
    const uint32_t ring = (smem_addr(dyn) + 1023) & ~1023u;
    const uint32_t p_smem = ring + A.slots * kSlotBytes;
    const uint32_t p_bytes = A.ncap / 16 * kPGroup;
    const uint32_t q_smem = p_smem + (1 + A.two_p) * p_bytes;
    const uint32_t q_half = A.ncap * 128, q_bytes = kHalves * q_half;
    const uint32_t ones = q_smem + (1 + A.two_q) * q_bytes;
    // TMEM: S (once or twice), O, L.
    const uint32_t col_o = A.ncap * (1 + A.two_s), col_l = col_o + A.ncap;

    // ---- set-up: barriers, TMEM, the constant operand, the CTA's tiles -----
    if (warp == kWarpMma) tmem_alloc(&C.tmem, kTmemCols);
    if (tid < kMaxSlots) {
        mbar_init(&C.full[tid], 2);
        mbar_init(&C.empty[tid], 1);
    } else if (tid >= 32 && tid < 34) {
        const int s = tid - 32;
        mbar_init(&C.q_full[s], 1);
        mbar_init(&C.q_empty[s], 1);
        mbar_init(&C.s_full[s], 2);
        mbar_init(&C.p_full[s], 1);
        mbar_init(&C.pv_done[s], 1);
    } else if (tid == 64) {
        mbar_init(&C.drained, 1);
        C.gave_up = C.poison = C.joins = 0;
        C.issued[0][0] = C.issued[0][1] = C.issued[1][0] = C.issued[1][1] = C.q_issued = 0;
        C.start_b = C.start_unit = C.start_tile = 0;
        C.tiles_before[0] = C.tiles_before[1] = 0;
    } else if (tid == 96) {
        prefetch_map(&q_map);
        prefetch_map(&k_map);
        prefetch_map(&v_map);
    } else if (tid >= 128 && tid < 192) {
        st_shared16(ones + (tid - 128) * 16, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u);
    }
    fence_barrier_init();

    // Nothing before this line reads or writes memory that another kernel may
    // touch: the launch may overlap the end of the kernel before it.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // The list of all units' tiles, each unit with unit_cost further places in
    // front for what it costs beside its tiles, is cut evenly.
    const int U = A.unit_cost, me = blockIdx.x;
    auto cost_of = [&](const Req &r) { return r.blocks * A.Hkv * (r.nt + U); };
    Cuts cuts;
    int start, end, tiles, t, start_b, start_unit;
    Req start_req;
    if (A.B <= kWarpScan) {
        // Few requests: every warp finds out by itself, a lane for each
        // kWarpScan / 32 of them.
        constexpr int kEach = kWarpScan / 32;
        Req r[kEach];
        int my_cost = 0, my_units = 0;
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            const int b = lane * kEach + k;
            if (b < A.B) r[k] = load_req(A, b);
            else r[k] = Req{};
            my_cost += cost_of(r[k]);
            my_units += r[k].blocks * A.Hkv;
        }
        int cost = my_cost, units = my_units;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, cost, o), y = __shfl_up_sync(0xffffffffu, units, o);
            if (lane >= o) {
                cost += x;
                units += y;
            }
        }
        const int total = __shfl_sync(0xffffffffu, cost, 31), all_units = __shfl_sync(0xffffffffu, units, 31);
        cuts = Cuts(total, gridDim.x);
        start = cuts.start(me);
        end = cuts.start(me + 1);
        int before[2] = {0, total - U * all_units};
#pragma unroll
        for (int side = 0; side < 2; ++side) {
            const int x = side ? end : start;
            const uint32_t who = __ballot_sync(0xffffffffu, x >= cost - my_cost && x < cost);
            if (!who) continue;  // the list's end
            const int src = __ffs(who) - 1;
            int at = cost - my_cost, first_unit = units - my_units, k = 0;
#pragma unroll
            for (int j = 0; j < kEach - 1; ++j) {
                if (k == j && x >= at + cost_of(r[j])) {
                    at += cost_of(r[j]);
                    first_unit += r[j].blocks * A.Hkv;
                    k = j + 1;
                }
            }
            Req q = r[0];
#pragma unroll
            for (int j = 1; j < kEach; ++j)
                if (k == j) q = r[j];
            const int i = (x - at) / (q.nt + U), tile = max(x - at - i * (q.nt + U) - U, 0);
            before[side] = __shfl_sync(0xffffffffu, at - U * first_unit + i * q.nt + tile, src);
            if (side == 0) {
                start_b = __shfl_sync(0xffffffffu, lane * kEach + k, src);
                start_unit = __shfl_sync(0xffffffffu, i, src);
                t = __shfl_sync(0xffffffffu, tile, src);
                start_req.row0 = __shfl_sync(0xffffffffu, q.row0, src);
                start_req.n = __shfl_sync(0xffffffffu, q.n, src);
                start_req.pos0 = __shfl_sync(0xffffffffu, q.pos0, src);
                start_req.kbeg = __shfl_sync(0xffffffffu, q.kbeg, src);
                start_req.kend = __shfl_sync(0xffffffffu, q.kend, src);
                start_req.t0 = __shfl_sync(0xffffffffu, q.t0, src);
                start_req.nt = __shfl_sync(0xffffffffu, q.nt, src);
                start_req.blocks = __shfl_sync(0xffffffffu, q.blocks, src);
                start_req.per = __shfl_sync(0xffffffffu, q.per, src);
            }
        }
        tiles = start < end ? before[1] - before[0] : 0;
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
    } else {
        const int per = (A.B + kThreadsStep - 1) / kThreadsStep;
        const int b_lo = min(tid * per, A.B), b_hi = min(b_lo + per, A.B);
        int my_cost = 0, my_units = 0;
        for (int b = b_lo; b < b_hi; ++b) {
            const Req r = load_req(A, b);
            my_units += r.blocks * A.Hkv;
            my_cost += cost_of(r);
        }
        int cost = my_cost, units = my_units;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, cost, o), y = __shfl_up_sync(0xffffffffu, units, o);
            if (lane >= o) {
                cost += x;
                units += y;
            }
        }
        if (lane == 31) {
            C.warp_cost[warp] = cost;
            C.warp_units[warp] = units;
        }
        __syncthreads();
        cost -= my_cost;
        units -= my_units;
        int total = 0, all_units = 0;
        for (int w = 0; w < kThreadsStep / 32; ++w) {
            if (w < warp) {
                cost += C.warp_cost[w];
                units += C.warp_units[w];
            }
            total += C.warp_cost[w];
            all_units += C.warp_units[w];
        }
        cuts = Cuts(total, gridDim.x);
        start = cuts.start(me);
        end = cuts.start(me + 1);
        // the threads whose requests hold `start` and `end` say where
        for (int side = 0; side < 2; ++side) {
            const int x = side ? end : start;
            if (x < cost || x >= cost + my_cost) continue;
            int at = cost, first_unit = units;
            for (int b = b_lo; b < b_hi; ++b) {
                const Req r = load_req(A, b);
                const int here = cost_of(r);
                if (x < at + here) {
                    const int i = (x - at) / (r.nt + U), tile = max(x - at - i * (r.nt + U) - U, 0);
                    C.tiles_before[side] = at - U * first_unit + i * r.nt + tile;
                    if (side == 0) {
                        C.start_b = b;
                        C.start_unit = i;
                        C.start_tile = tile;
                    }
                    break;
                }
                at += here;
                first_unit += r.blocks * A.Hkv;
            }
        }
        if (tid == 0 && end == total) C.tiles_before[1] = total - U * all_units;
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        tiles = start < end ? C.tiles_before[1] - C.tiles_before[0] : 0;
        t = C.start_tile;
        start_b = C.start_b;
        start_unit = C.start_unit;
        if (tiles > 0) start_req = load_req(A, start_b);
    }
    const uint32_t tmem = C.tmem;
    volatile int *gave_up = &C.gave_up;
    Unit u;
    if (tiles > 0) u.start(A, start_b, start_req, start_unit);  // at its tile t

    if (tiles > 0 && warp >= kWarpK && warp < kWarpMma) {
        // ---- producers ----------------------------------------------------------
        // One warp copies the first two thirds of a K tile's TMA boxes, and
        // the queries, one those of a V tile, and one the rest of both.  A
        // lane looks up the pages of one box (or of four keys: gather) one
        // tile ahead; one elected lane issues the copies.
        const int part = warp == kWarpBoth;
        const int kv_lo = warp == kWarpV, kv_hi = warp == kWarpK ? 1 : 2;
        const int span = kBox ? A.box : 4, boxes = kTile / span, most = (2 * boxes + 2) / 3;
        const int my_box = part * most + lane;  // this lane's
        const bool my_turn = lane < most && my_box < boxes;
        struct Ids { int page[4]; };
        auto look_up = [&](const Unit &x, int tile, Ids &ids) {
            const int key0 = (x.q.t0 + tile) * kTile + my_box * span;
            const int32_t *table = A.block_table + (int64_t)x.b * A.max_pages;
            const bool wanted = my_turn && key0 < x.q.kend && key0 + span > x.q.kbeg;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                ids.page[i] = -1;
                if ((i == 0 || !kBox) && wanted) {
                    const int pi = page_of(A, key0 + i);
                    if (pi < A.max_pages) ids.page[i] = table[pi];
                }
            }
        };
        Ids ids;
        look_up(u, t, ids);
        Ring r[2], rq;  // K and V have rings of their own
        const int ring_slots[2] = {A.k_slots, A.slots - A.k_slots}, ring_slot0[2] = {0, A.k_slots};
        bool first = true, ok = true;
        int units = 0, issued[2] = {0, 0};
        for (int i = 0; i < tiles; ++i) {
            Unit x = u;
            int tx = t + 1;
            if (tx == u.q.nt && i + 1 < tiles) {
                x.next(A);
                tx = 0;
            }
            Ids ahead;
            if (i + 1 < tiles) look_up(x, tx, ahead);

            const int tile0 = (u.q.t0 + t) * kTile, key0 = tile0 + my_box * span;
            const bool here = my_turn && key0 < u.q.kend && key0 + span > u.q.kbeg;
            uint32_t bad_bits = 0;  // of the lane's keys (gather) or of the whole box
            int row[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const bool good = ids.page[j] >= 0 && ids.page[j] < A.num_pages;
                if (!good) bad_bits |= 1u << j;
                const int page = good ? ids.page[j] : 0;  // masked; any memory will do
                row[j] = kBox ? page
                               : page * A.page_rows + u.h * A.head_rows + key0 + j -
                                     page_of(A, key0 + j) * A.page_size;
            }
            const bool lane_bad = here && (kBox ? (bad_bits & 1) : bad_bits != 0);
            uint32_t words[4] = {0, 0, 0, 0};
            if (__any_sync(0xffffffffu, lane_bad)) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t m = 0;
                    if (lane_bad) {
                        if (kBox) {
                            const int lo = max(my_box * span - 32 * q, 0), hi = min(my_box * span + span - 32 * q, 32);
                            if (lo < hi) m = (hi - lo == 32 ? 0xffffffffu : ((1u << (hi - lo)) - 1u)) << lo;
                        } else if (my_box / 8 == q) {
                            m = bad_bits << (4 * (my_box % 8));
                        }
                    }
                    words[q] = __reduce_or_sync(0xffffffffu, m);
                }
            }
            // the boxes to copy: a run of lanes
            const uint32_t run = __ballot_sync(0xffffffffu, here);
            const int box_lo = part * most + __ffs(run) - 1, box_n = __popc(run);
            const uint32_t bytes = box_n * uint32_t(span) * D * 2;
            int *const rows = C.row[kv_lo];
            __syncwarp();
            if (my_turn) {
                if (kBox) rows[my_box] = row[0];
                else *reinterpret_cast<int4 *>(rows + 4 * my_box) = make_int4(row[0], row[1], row[2], row[3]);
            }
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
                if (kv < kv_lo || kv >= kv_hi || !ok) continue;
                const int slot = ring_slot0[kv] + r[kv].slot;
                if (i >= ring_slots[kv]) ok = wait_or_give_up(&C.empty[slot], r[kv].phase ^ 1, A.wait_ns, gave_up);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) continue;
                if (kv == 0 && lane == 0)
                    *reinterpret_cast<uint4 *>(C.bad[part][i % kWords]) =
                        make_uint4(words[0], words[1], words[2], words[3]);
                __syncwarp();
                if (elect_one()) {
                    const CUtensorMap *map = kv ? &v_map : &k_map;
                    uint64_t *full = &C.full[slot];
                    mbar_arrive_expect_tx(full, bytes);
                    uint32_t dst = ring + slot * kSlotBytes + box_lo * span * 128;
                    if (kBox) {
                        const int first_key = tile0 + box_lo * span;
                        int in_page = first_key - page_of(A, first_key) * A.page_size;
#pragma unroll 4
                        for (int j = box_lo; j < box_lo + box_n; ++j) {
                            const int page = rows[j];
                            tma_load_4d(dst, map, full, 0, in_page, u.h, page);
                            if (kHalves == 2) tma_load_4d(dst + kHalfBytes, map, full, 64, in_page, u.h, page);
                            dst += span * 128;
                            in_page += span;
                            if (in_page == A.page_size) in_page = 0;
                        }
                    } else {
                        const int x0 = u.h * A.head_x;
#pragma unroll 4
                        for (int j = box_lo; j < box_lo + box_n; ++j) {
                            const int4 k = *reinterpret_cast<const int4 *>(rows + 4 * j);
                            tma_gather4(dst, map, full, x0, k.x, k.y, k.z, k.w);
                            if (kHalves == 2) tma_gather4(dst + kHalfBytes, map, full, x0 + 64, k.x, k.y, k.z, k.w);
                            dst += span * 128;
                        }
                    }
                }
                __syncwarp();
                ++issued[kv];
                r[kv].next(ring_slots[kv]);
            }
            if (!ok) break;
            if (first && warp == kWarpK) {
                // The unit's queries: one box per row, its G heads side by side.
                if (units > A.two_q) ok = wait_or_give_up(&C.q_empty[rq.slot], rq.phase ^ 1, A.wait_ns, gave_up);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                if (elect_one()) {
                    mbar_arrive_expect_tx(&C.q_full[rq.slot], uint32_t(u.ncols) * D * 2);
                    uint32_t dst = q_smem + rq.slot * q_bytes;
                    const int row0 = u.q.row0 + u.j0, nrows = u.ncols / A.G;
                    for (int j = 0; j < nrows; ++j) {
                        tma_load_3d(dst, &q_map, &C.q_full[rq.slot], 0, u.h * A.G, row0 + j);
                        if (kHalves == 2) tma_load_3d(dst + q_half, &q_map, &C.q_full[rq.slot], 64, u.h * A.G, row0 + j);
                        dst += A.G * 128;
                    }
                }
                __syncwarp();
                rq.next(1 + A.two_q);
                ++units;
            }
            first = tx == 0;
            u = x;
            t = tx;
            ids = ahead;
        }
        if (lane == 0) {  // for the CTA's end, should a wait have given up
            if (warp != kWarpV) C.issued[part][0] = issued[0];
            if (warp != kWarpK) C.issued[part][1] = issued[1];
            if (warp == kWarpK) C.q_issued = units;
        }
    } else if (tiles > 0 && warp == kWarpMma) {
        // ---- MMA issuer: S of the next tile and O, L of this one, whichever's
        // operands are there ----------------------------------------------------
        const uint64_t kd0 = smem_desc(ring, 16, 1024), qd0 = smem_desc(q_smem, 16, 1024);
        // D = 64: the second group of 64 rows repeats the first
        const uint64_t vd0 = smem_desc(ring + A.k_slots * kSlotBytes, kHalves == 2 ? kHalfBytes : 0, 1024);
        const uint64_t pd0 = smem_desc32(p_smem, kPGroup, 256), ones_d = smem_desc(ones, 0, 0);
        Unit us = u, uo = u;         // units of the next S and of the next O
        int ts = t, to = t;
        Ring rk, rv, rq;
        const int v_slots = A.slots - A.k_slots;
        bool first_s = true, first_o = true;
        int si = 0, oi = 0;          // S and O tiles issued
        uint32_t id_s = 0, id_o = 0, id_l = 0;
        uint64_t since = 0;
        uint32_t polls = 0;
        while (oi < tiles) {
            if (si < tiles && si <= oi + A.two_s && (!first_s || warp_test(&C.q_full[rq.slot], rq.phase)) &&
                warp_test(&C.full[rk.slot], rk.phase)) {
                if (first_s) id_s = mma_idesc(128, (us.ncols + 15) & ~15, false, false);
                const int buf = A.two_s ? si & 1 : 0;
                const bool last = ts + 1 == us.q.nt || si + 1 == tiles;
                tc_fence_after();
                if (elect_one()) {
                    mbar_arrive(&C.s_full[buf]);  // passes the producer's words on
                    const uint64_t kd = kd0 + uint32_t(rk.slot) * (kSlotBytes >> 4);
                    const uint64_t qd = qd0 + uint32_t(rq.slot) * (q_bytes >> 4);
#pragma unroll
                    for (int d = 0; d < D / 16; ++d)
                        mma_ss(tmem + buf * A.ncap, kd + (((d / 4) * kHalfBytes + (d % 4) * 32) >> 4),
                               qd + (((d / 4) * q_half + (d % 4) * 32) >> 4), id_s, d > 0);
                    mma_commit(&C.s_full[buf]);
                    mma_commit(&C.empty[rk.slot]);
                    if (last) mma_commit(&C.q_empty[rq.slot]);
                }
                __syncwarp();
                rk.next(A.k_slots);
                first_s = last;
                if (last) {
                    rq.next(1 + A.two_q);
                    if (si + 1 < tiles) us.next(A);
                    ts = 0;
                } else {
                    ++ts;
                }
                ++si;
                polls = 0;
                continue;
            }
            const int pb = A.two_p ? oi & 1 : 0;
            if (oi < si && warp_test(&C.p_full[pb], (A.two_p ? oi >> 1 : oi) & 1) && warp_test(&C.full[A.k_slots + rv.slot], rv.phase)) {
                if (first_o) {
                    const int N = (uo.ncols + 15) & ~15;
                    id_o = mma_idesc(128, N, true, true);
                    id_l = mma_idesc(128, N, false, true);
                }
                tc_fence_after();
                if (elect_one()) {
                    const uint64_t vd = vd0 + uint32_t(rv.slot) * (kSlotBytes >> 4);
                    const uint64_t pd = pd0 + uint32_t(pb) * (p_bytes >> 4);
#pragma unroll
                    for (int k = 0; k < kTile / 16; ++k) {
                        mma_ss(tmem + col_o, vd + k * (2048 >> 4), pd + k * (512 >> 4), id_o, !(first_o && k == 0));
                        mma_ss(tmem + col_l, ones_d, pd + k * (512 >> 4), id_l, !(first_o && k == 0));
                    }
                    mma_commit(&C.pv_done[pb]);
                    mma_commit(&C.empty[A.k_slots + rv.slot]);
                }
                __syncwarp();
                rv.next(v_slots);
                first_o = ++to == uo.q.nt;
                if (first_o) {
                    if (oi + 1 < tiles) uo.next(A);
                    to = 0;
                }
                ++oi;
                polls = 0;
                continue;
            }
            if ((++polls & 255u) != 0) continue;
            const uint64_t now = global_timer_ns();
            if (polls == 256) since = now;
            if (__any_sync(0xffffffffu, *gave_up || now - since > A.wait_ns)) {
                *gave_up = 1;
                break;
            }
        }
    } else if (tiles > 0) {
        // ---- softmax: thread = key of the tile -----------------------------------
        // Once a wait has given up, the others return at once and the loop
        // runs to its end on whatever there is; the status tells.
        const int key = tid & 127, grp = tid >> 7;
        const uint32_t lane_tm = tmem + (uint32_t((warp & 3) * 32) << 16);
        const int swz = key & 7, p_swz = (key >> 2) & 1;
        Ring rv;
        const int v_slots = A.slots - A.k_slots;
        int i = 0;  // tile of the CTA
        if (warp == 0) {
            poll_or_give_up(&C.s_full[0], 0, A.wait_ns, gave_up);
            __syncwarp();
        }
        for (int unit = 1; i < tiles; ++unit) {
            const int N = (u.ncols + 15) & ~15, t_first = t;
            const int here = min(u.q.nt - t, tiles - i);
            // tiles that every column sees in full: [whole_lo, whole_hi)
            const int whole_hi = min(u.q.kend, u.q.pos0 + u.j0 + 1) / kTile;
            const int last_beg = A.window > 0 ? max(u.q.pos0 + u.j0 + u.ncols / A.G - A.window, u.q.kbeg) : u.q.kbeg;
            const int whole_lo = (last_beg + kTile - 1) / kTile;
            for (int k = 0; k < here; ++k, ++t, ++i) {
                const bool first = k == 0;
                const int buf = A.two_s ? i & 1 : 0;
                const uint32_t s_tm = lane_tm + buf * A.ncap;
                wait_or_give_up(&C.s_full[buf], (A.two_s ? i >> 1 : i) & 1, A.wait_ns, gave_up);
                tc_fence_after();
                const int tile = u.q.t0 + t;
                uint4 bw = *reinterpret_cast<const uint4 *>(C.bad[0][i % kWords]);
                {
                    const uint4 b1 = *reinterpret_cast<const uint4 *>(C.bad[1][i % kWords]);
                    bw = make_uint4(bw.x | b1.x, bw.y | b1.y, bw.z | b1.z, bw.w | b1.w);
                }
                const bool whole = (bw.x | bw.y | bw.z | bw.w) == 0 && tile >= whole_lo && tile < whole_hi;
                int lo = 0, hi = N;
                if (!whole) {
                    const int q = warp & 3;
                    const uint32_t word = q == 0 ? bw.x : q == 1 ? bw.y : q == 2 ? bw.z : bw.w;
                    visible_columns(A, u, tile * kTile + key, (word >> lane) & 1, lo, hi);
                }
                bool move = first;
                const int pb = A.two_p ? i & 1 : 0;
                const uint32_t p_row = p_smem + pb * p_bytes + key * 32;
                if (i > A.two_p)  // P's last reader
                    wait_or_give_up(&C.pv_done[pb], ((A.two_p ? i >> 1 : i) - 1) & 1, A.wait_ns, gave_up);
                if (__builtin_expect(!whole, 0) && (lo > 0 || hi < u.ncols)) {
                    // Masked keys must not reach O through 0 * infinity: a
                    // value row that no column sees is cleared, and one that
                    // some see loses its NaN and infinities, which are added
                    // at the unit's end to the columns that do see them.
                    wait_or_give_up(&C.full[A.k_slots + rv.slot], rv.phase, A.wait_ns, gave_up);
                    const uint32_t vb = ring + (A.k_slots + rv.slot) * kSlotBytes + key * 128;
#pragma unroll 1
                    for (int ch = grp; ch < 8 * kHalves; ch += kGroups) {
                        const uint32_t at = vb + (ch / 8) * kHalfBytes + (((ch % 8) ^ swz) << 4);
                        if (lo >= hi) {
                            st_shared16(at, 0, 0, 0, 0);
                            continue;
                        }
                        const uint4 x = ld_shared16(at);
                        if (__builtin_expect(nonfinite_any(x), 0)) {
                            st_shared16(at, x.x & ~nonfinite_mask(x.x), x.y & ~nonfinite_mask(x.y),
                                        x.z & ~nonfinite_mask(x.z), x.w & ~nonfinite_mask(x.w));
                            C.poison = unit;
                        }
                    }
                }
                rv.next(v_slots);
                __syncwarp();

                // Weights of the tile against the reference.  A unit's first
                // tile sets the reference before, a tile that passes it
                // moves it and starts again (once: then none does).
                for (int turn = 0; turn < 2; ++turn) {
                    if (__builtin_expect(move, 0)) {
                        if (!first && A.two_p)
                            wait_or_give_up(&C.pv_done[pb ^ 1], ((i - 1) >> 1) & 1, A.wait_ns, gave_up);
                        __syncwarp();
                        tc_fence_after();
                        // the warps' maxima wait in P, which is about to be written
                        float *const colmax = reinterpret_cast<float *>(dyn + (p_smem + pb * p_bytes - smem_addr(dyn)));
                        for (int n = 16 * grp; n < N; n += 16 * kGroups) {
                            float s[16];
                            tmem_ld16(s, s_tm + n);
                            const uint32_t seen = seen16(n, lo, hi);
                            tmem_wait_ld(s);
                            float keep = -INFINITY;
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                float x = ((seen >> e) & 1) ? s[e] : -INFINITY;
                                asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(x) : "f"(x));
                                if (lane == e) keep = x;
                            }
                            if (lane < 16) colmax[(warp & 3) * A.ncap + n + lane] = keep;
                        }
                        soft_sync();
                        for (int n = tid; n < N; n += kSoftThreads) {
                            const float old = first ? kRefMin : C.ref[n];
                            const float *const cm = colmax + n;
                            const float top = fmaxf(fmaxf(cm[0], cm[A.ncap]), fmaxf(cm[2 * A.ncap], cm[3 * A.ncap]));
                            const float now = fmaxf(top + A.headroom, old);
                            // the columns past the last weigh nothing
                            C.ref[n] = n < u.ncols ? now : INFINITY;
                            C.fac[n] = exp2_approx((old - now) * A.scale2);
                        }
                        soft_sync();
                        if (!first) {
                            for (int n = 16 * grp; n < N; n += 16 * kGroups) {
                                float o[16], l[16];
                                tmem_ld16(o, lane_tm + col_o + n);
                                tmem_ld16(l, lane_tm + col_l + n);
                                tmem_wait_ld(o);
                                tmem_use16(l);
#pragma unroll
                                for (int e = 0; e < 16; ++e) {
                                    o[e] *= C.fac[n + e];
                                    l[e] *= C.fac[n + e];
                                }
                                tmem_st16(lane_tm + col_o + n, o);
                                tmem_st16(lane_tm + col_l + n, l);
                            }
                            tmem_wait_st();
                        }
                    }
                    float top = 0.f;
                    for (int n = 16 * grp; n < N; n += 16 * kGroups) {
                        float s[16];
                        tmem_ld16(s, s_tm + n);
                        const uint32_t at = p_row + (n / 16) * kPGroup;
                        top = fmaxf(top, whole ? weigh16<false>(s, C.ref + n, A.scale2, 0, at, p_swz)
                                               : weigh16<true>(s, C.ref + n, A.scale2, seen16(n, lo, hi), at, p_swz));
                    }
                    fence_async_shared();
                    tc_fence_before();
                    move = soft_any(top > 0.f);
                    if (__builtin_expect(!move, 1)) break;
                }
                if (tid == 0) mbar_arrive(&C.p_full[pb]);
            }

            // ---- the unit's end in this CTA --------------------------------------
            wait_or_give_up(&C.pv_done[A.two_p ? (i - 1) & 1 : 0], (A.two_p ? (i - 1) >> 1 : i - 1) & 1,
                            A.wait_ns, gave_up);
            __syncwarp();
            tc_fence_after();
            const bool split = t_first > 0 || t < u.q.nt;
            const int d = key % D;
            const bool writer = key < D;
            // Who shares a cut unit, and the slots of their parts: a CTA's
            // first unit uses the first of its two slots.
            int first_cta = 0, members = 1, slot0 = 0, slot = 0;
            if (split) {
                const int tile0 = t_first > 0 ? start - t_first : end - t;  // the first tile's place
                first_cta = cuts.of(tile0);
                members = cuts.of(tile0 + u.q.nt - 1) - first_cta + 1;
                slot0 = 2 * first_cta + (cuts.start(first_cta) >= tile0 - U ? 0 : 1);
                slot = me == first_cta ? slot0 : 2 * me;
            }
            uint16_t *const out0 = A.out + ((int64_t)(u.q.row0 + u.j0) * A.Hq + u.h * A.G) * D;
            float *const part0 = A.part + (int64_t)slot * A.ncap * D + d;
            const int wrap = (A.Hq - A.G) * D;
            for (int n = 16 * grp; n < N; n += 16 * kGroups) {
                float o[16], l[16];
                tmem_ld16(o, lane_tm + col_o + n);
                tmem_ld16(l, lane_tm + col_l + n);
                tmem_wait_ld(o);
                tmem_use16(l);
                const int m = min(16, u.ncols - n);
                if (split) {
                    float *part = part0 + (int64_t)n * D;
                    float sum = 0.f;
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        if (e < m && writer) part[e * D] = o[e];
                        if (lane == e) sum = l[e];
                    }
                    if (lane < m && (warp & 3) == 0) {
                        A.stat[((int64_t)slot * 2) * A.ncap + n + lane] = C.ref[n + lane];
                        A.stat[((int64_t)slot * 2 + 1) * A.ncap + n + lane] = sum;
                    }
                } else {
                    int g = n % A.G;
                    uint16_t *out = out0 + (int64_t)(n / A.G) * A.Hq * D + g * D + d;
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const float y = l[e] == 0.f ? 0.f : __fdividef(o[e], l[e]);
                        if (e < m && writer) *out = uint16_t(pack_bf16x2(y, 0.f));
                        out += D;
                        if (++g == A.G) {
                            g = 0;
                            out += wrap;
                        }
                    }
                }
            }
            const bool poisoned = C.poison == unit;
            if (poisoned) soft_sync();  // the other groups' outputs are written
            if (__builtin_expect(poisoned, 0) && writer && grp == 0) {
                // What was taken out of V: for the keys of this CTA's
                // tiles that some columns see and others do not.
                const int k0 = max((u.q.t0 + t_first) * kTile, u.q.kbeg);
                const int k1 = min((u.q.t0 + t) * kTile, u.q.kend);
#pragma unroll 1
                for (int k = k0; k < k1; ++k) {
                    int vlo, vhi;
                    visible_columns(A, u, k, false, vlo, vhi);
                    if (vlo >= vhi || (vlo == 0 && vhi == u.ncols)) continue;
                    const int page = A.block_table[(int64_t)u.b * A.max_pages + k / A.page_size];
                    if (page < 0 || page >= A.num_pages) continue;
                    const float v = bf16_lo(A.v_cache[page * A.page_stride + (k % A.page_size) * A.slot_stride +
                                                      u.h * A.head_stride + d]);
                    if (isfinite(v)) continue;
#pragma unroll 1
                    for (int n = vlo; n < vhi; ++n) {
                        if (split) {
                            part0[(int64_t)n * D] += v;
                        } else {
                            uint16_t *y = out0 + (int64_t)(n / A.G) * A.Hq * D + (n % A.G) * D + d;
                            *y = uint16_t(pack_bf16x2(bf16_lo(*y) + v, 0.f));
                        }
                    }
                }
            }
            tc_fence_before();
            soft_sync();  // ref, poison and O are read before the next unit writes them
            if (tid == 0) {
                if (split) __threadfence();  // all the CTA's writes of the part: they came before the barrier
                if (split && atomicAdd(&A.arrived[first_cta], 1) == members - 1) {
                    A.arrived[first_cta] = 0;  // as the next call wants it
                    C.join[C.joins++] = Join{u.q.row0 + u.j0, u.h * A.G, u.ncols, slot0, first_cta, members};
                }
            }
            if (i < tiles) {
                u.next(A);
                t = 0;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (__builtin_expect(C.gave_up, 0)) {
        // No warp issues any more.  What is in flight lands before the CTA ends: the products, each slot's
        // latest copy, the queries.  A phase that a warp left open ends the wait at its limit; by then
        // all has landed.
        if (warp == kWarpMma) {
            if (elect_one()) mma_commit(&C.drained);
            __syncwarp();
            mbar_wait_bounded(&C.drained, 0, kDrainTimeoutNs);
        } else if (warp == kWarpK) {
            bool landed = true;
            for (int kv = 0; kv < 2; ++kv) {
                const int slots = kv ? A.slots - A.k_slots : A.k_slots, n = max(C.issued[0][kv], C.issued[1][kv]);
                for (int k = max(n - slots, 0); landed && k < n; ++k)
                    landed = mbar_wait_bounded(&C.full[(kv ? A.k_slots : 0) + k % slots], (k / slots) & 1, kDrainTimeoutNs);
            }
            for (int k = max(C.q_issued - 1 - A.two_q, 0); landed && k < C.q_issued; ++k)
                landed = mbar_wait_bounded(&C.q_full[A.two_q ? k & 1 : 0], (A.two_q ? k >> 1 : k) & 1, kDrainTimeoutNs);
        }
        if (tid == 0) atomicOr(A.status, kStatusWaitTimeout);
        __syncthreads();
    }
    if (warp == kWarpMma) tmem_free(tmem, kTmemCols);
    // The joins come last, when every warp has time and the loops above keep
    // their registers.
    for (int k = 0; k < C.joins; ++k) {
        __threadfence();
        const Join J = C.join[k];
        if (J.members <= 2) join_columns<D, 2>(A, J, warp, lane);
        else join_columns<D, 1>(A, J, warp, lane);
    }
}

// Rows of a unit at most: those whose columns fit.
int step_rows(int Hq, int Hkv, int q_max) { return std::min(q_max, kMaxCols / (Hq / Hkv)); }
int step_columns(int Hq, int Hkv, int q_max) {
    return (step_rows(Hq, Hkv, q_max) * (Hq / Hkv) + 15) / 16 * 16;
}

constexpr size_t kHeaderBytes = 256 + (sizeof(int32_t) * kAttnMaxCtas + 255) / 256 * 256;

template <int D, bool kBox>
cudaError_t launch(StepArgs A, const CUtensorMap (&maps)[3], int ctas, cudaStream_t s) {
    // What is held twice, against ring slots.  A tile of V waits for its
    // tile's softmax, so three V slots carry more than a second P or Q; Q is
    // needed twice only at a unit's border.  The first of these that leaves
    // five slots, else four, is taken.
    A.two_s = A.ncap <= kTwoS;
    const size_t slot = size_t(D) * 2 * kTile;
    const size_t p = size_t(A.ncap / 16) * kPGroup, q = size_t(A.ncap) * D * 2;
    const size_t room = kSmemBytes - sizeof(Ctrl) - 2048;
    size_t fixed = 0;
    for (int want = 5; want >= 4; --want) {
        for (int twice = 2; twice >= want - 4; --twice) {
            A.two_p = A.two_s && twice >= 1;
            A.two_q = twice == 2;
            fixed = p * (1 + A.two_p) + q * (1 + A.two_q);
            if (fixed + want * slot <= room) break;
        }
        if (fixed + want * slot <= room) break;
    }
    A.slots = int(std::min<size_t>((room - fixed) / slot, kMaxSlots));
    A.k_slots = A.slots / 2;
    const size_t smem = 2048 + fixed + A.slots * slot;
    // The limit is the process's: the same for every shape, so that calls of other shapes, from other
    // threads or between a graph's capture and its instantiation, leave it alone.
    cudaError_t e = cudaFuncSetAttribute(step_attention_kernel<D, kBox>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         int(kSmemBytes - sizeof(Ctrl)));
    if (e != cudaSuccess) return e;
    return launch_overlapped(step_attention_kernel<D, kBox>, ctas, kThreadsStep, smem, s, A, maps[0], maps[1], maps[2]);
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

bool step_list_fits(const dspark_attn &a) {
    const long long blocks = (a.q_max + step_rows(a.Hq, a.Hkv, a.q_max) - 1) / step_rows(a.Hq, a.Hkv, a.q_max) + 1;
    const long long places = (long long)a.max_pages * a.page_size / kTile + 2 + kUnitCost;
    return places * blocks * a.Hkv <= INT32_MAX / a.B;
}

cudaError_t launch_step_attention(const dspark_attn &a, int sms, uint64_t wait_ns, cudaStream_t s) {
    StepArgs A{};
    A.B = a.B; A.rows = a.rows; A.q_max = a.q_max; A.Hq = a.Hq; A.Hkv = a.Hkv; A.G = a.Hq / a.Hkv;
    A.page_size = a.page_size; A.num_pages = a.num_pages; A.max_pages = a.max_pages;
    A.window = a.window;
    A.page_shift = 31;  // exact below 2^31: page_mul = ceil(2^shift / page_size) < 2^32
    while ((1u << (A.page_shift - 31)) < unsigned(a.page_size)) ++A.page_shift;
    A.page_mul = uint32_t(((1ull << A.page_shift) + a.page_size - 1) / a.page_size);
    A.ncap = step_columns(a.Hq, a.Hkv, a.q_max);
    A.rows_cap = step_rows(a.Hq, a.Hkv, a.q_max);
    A.scale2 = float(double(a.scale) * 1.4426950408889634);
    A.headroom = std::min(kHeadroom / A.scale2, 1e38f);
    A.page_stride = a.page_stride; A.slot_stride = a.slot_stride; A.head_stride = a.head_stride;
    A.v_cache = static_cast<const uint16_t *>(a.v_cache);
    A.row_off = a.row_off; A.seq_lens = a.seq_lens; A.block_table = a.block_table;
    A.out = static_cast<uint16_t *>(a.out);
    char *ws = static_cast<char *>(a.workspace);
    A.status = reinterpret_cast<int32_t *>(ws);
    A.arrived = reinterpret_cast<int32_t *>(ws + 256);
    A.part = reinterpret_cast<float *>(ws + kHeaderBytes);
    A.stat = reinterpret_cast<float *>(ws + kHeaderBytes +
                                       align256(2 * kAttnMaxCtas * size_t(A.ncap) * a.D * sizeof(float)));
    A.unit_cost = kUnitCost;
    A.wait_ns = wait_ns;

    // A page of 8 k positions is copied in boxes of whole pages or parts of
    // them; other pages key by key (four keys a copy).
    CUtensorMap maps[3];
    {
        const uint64_t dims[3] = {uint64_t(a.D), uint64_t(a.Hq), uint64_t(a.rows)};
        const uint64_t st[2] = {uint64_t(a.D) * 2, uint64_t(a.D) * a.Hq * 2};
        const uint32_t bx[3] = {64, uint32_t(A.G), 1};
        const cudaError_t e = encode_map(&maps[0], a.q_rot, 3, dims, st, bx);
        if (e != cudaSuccess) return e;
    }
    const int box = gcd(a.page_size, kTile);
    const void *bases[2] = {a.k_cache, a.v_cache};
    if (box >= 8) {
        A.box = box;
        const uint64_t dims[4] = {uint64_t(a.D), uint64_t(a.page_size), uint64_t(a.Hkv), uint64_t(a.num_pages)};
        const uint64_t st[3] = {uint64_t(a.slot_stride) * 2, uint64_t(a.head_stride) * 2, uint64_t(a.page_stride) * 2};
        const uint32_t bx[4] = {64, uint32_t(box), 1, 1};
        for (int i = 0; i < 2; ++i) {
            const cudaError_t e = encode_map(&maps[1 + i], bases[i], 4, dims, st, bx);
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
            const cudaError_t e = encode_map(&maps[1 + i], bases[i], 2, dims, st, bx);
            if (e != cudaSuccess) return e;
        }
    }
    const int ctas = std::min(sms, kAttnMaxCtas);
    if (A.box) return a.D == 128 ? launch<128, true>(A, maps, ctas, s) : launch<64, true>(A, maps, ctas, s);
    return a.D == 128 ? launch<128, false>(A, maps, ctas, s) : launch<64, false>(A, maps, ctas, s);
}

}  // namespace dspark
