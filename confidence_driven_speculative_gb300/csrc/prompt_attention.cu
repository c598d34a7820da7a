// prompt_attention.cu -- whole prompts, causal, packed one after the other.
//
// Mathematics.  For a block of rows of one query head: S = Q K^T, the weights
// P = 2^(scale log2(e) S - m) against a running reference m per row, l the
// sum of P, O += P V; the output is O / l.  The reference is the first tile's
// maximum; a later tile moves it, and rescales O and l, only where its
// maximum passes the reference by 2^32 (the weights stay in the range of fp32
// and bfloat16 keeps its relative step), which is next to never.
//
// Bound: the tensor cores.  A unit is 256 rows of one head in two blocks of
// 128, walked over tiles of 128 keys.  S and O of both blocks fill TMEM
// (4 x 128 columns); P overwrites its S in TMEM and is the A operand of
// P V.  While one block's softmax runs, the tensor cores work on the other
// block: O_0 += P_0 V, S_0 of the next tile, O_1 += P_1 V, S_1 of the next tile.
// A softmax thread owns a row, so maxima and sums stay in its registers.
//
// Units are handed out by a counter, the longest of a prompt first, so the
// CTAs end together; a unit's result does not depend on who computes it.
#include <algorithm>

#include "attn.cuh"
#include "dspark_internal.cuh"
#include "tcgen05.cuh"

namespace dspark {
namespace {

constexpr int kTile = 128;        // rows of a block, keys of a tile
constexpr int kThreadsP = 384;
constexpr int kScan = 128;        // threads that sum up the prompts' units
constexpr int kWarpMmaP = 8, kWarpLoad = 9, kWarpClean = 10;  // softmax 0..7; two cleaners
constexpr int kCleaners = 64;
constexpr int kSlotsMax = 10;
constexpr int kSched = 4;         // units on their way to the warps
constexpr int kSchedReaders = 11; // warps that read them
constexpr float kRefMin = -1e30f;
constexpr float kRefSlack = 32.0f;
constexpr size_t kSmemBytes = 232448;

struct PromptArgs {
    int B, rows, q_max, Hq, Hkv, G, window;
    int slots, k_slots;
    float scale2;
    int64_t v_stride;
    const uint16_t *v;
    const int32_t *row_off;
    uint16_t *out;
    int32_t *counter;  // next unit, CTAs that are done
    int32_t *status;
    uint64_t wait_ns;
};

struct Unit {
    int row0, n;   // the prompt's first packed row, its rows
    int q0, h;     // first row of the unit in the prompt, query head; h < 0: no more units
};

// Tiles of keys that block a (rows q .. q + 127) of a unit walks.
struct Span { int lo, hi; };
__device__ __forceinline__ Span span_of(const PromptArgs &A, const Unit &u, int a) {
    const int q = u.q0 + a * kTile;
    if (q >= u.n) return {0, 0};
    Span s;
    s.lo = A.window > 0 ? max(q - A.window + 1, 0) / kTile : 0;
    s.hi = (min(q + kTile, u.n) + kTile - 1) / kTile;
    return s;
}
// Does some row of block a not see some key of tile t?
__device__ __forceinline__ bool partial(const PromptArgs &A, const Unit &u, int a, int t) {
    const int q = u.q0 + a * kTile;
    return (t + 1) * kTile - 1 > q || (A.window > 0 && t * kTile <= min(q + kTile, u.n) - 1 - A.window);
}

struct Ctrl {
    uint64_t full[kSlotsMax], empty[kSlotsMax], clean[kSlotsMax];
    uint64_t q_full[2], q_empty[2], s_full[2], o_full[2];
    uint64_t p_full[2][2];    // by block and half of the keys
    uint64_t sched_full[kSched], sched_empty[kSched], drained;
    Unit unit[kSched];
    int poisoned[8];          // by unit number % 8: the last unit + 1 that lost values
    int pairs[kScan + 1];     // exclusive sums of the units (per head) of each thread's prompts
    int warp_sum[kScan / 32];
    uint32_t tmem;
    int gave_up;
};

// Reads the next unit off the ring.
struct SchedReader {
    Ring r;
    __device__ __forceinline__ Unit next(Ctrl &C, const PromptArgs &A, volatile int *gave_up, int lane) {
        Unit u{0, 0, 0, -1};
        bool ok = wait_or_give_up(&C.sched_full[r.slot], r.phase, A.wait_ns, gave_up);
        ok = __all_sync(0xffffffffu, ok);
        if (ok) u = C.unit[r.slot];
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(&C.sched_empty[r.slot]);
        r.next(kSched);
        return u;
    }
};

template <int D>
__global__ void __launch_bounds__(kThreadsP, 1)
prompt_attention_kernel(const __grid_constant__ PromptArgs A, const __grid_constant__ CUtensorMap q_map,
                        const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map) {
    constexpr int kHalves = D / 64;
    constexpr uint32_t kHalfBytes = kTile * 128;
    constexpr uint32_t kSlotBytes = kHalves * kHalfBytes;
    constexpr uint32_t kColO = 2 * kTile;  // S_0, S_1, O_0, O_1
    extern __shared__ uint8_t dyn[];
    __shared__ Ctrl C;
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
    const uint32_t q_smem = (smem_addr(dyn) + 1023) & ~1023u;
    const uint32_t ring = q_smem + 2 * kSlotBytes;
    const int v_slots = A.slots - A.k_slots;
    const uint32_t v_ring = ring + A.k_slots * kSlotBytes;
    const uint32_t stage = ring + A.slots * kSlotBytes;  // 4 KB for each softmax warp
    volatile int *gave_up = &C.gave_up;

    if (tid == 0) {
        for (int s = 0; s < A.slots; ++s) {
            mbar_init(&C.full[s], 1);
            mbar_init(&C.empty[s], 1);
            mbar_init(&C.clean[s], 2);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&C.q_full[a], 1);
            mbar_init(&C.q_empty[a], 1);
            mbar_init(&C.s_full[a], 1);
            mbar_init(&C.p_full[a][0], 4);
            mbar_init(&C.p_full[a][1], 4);
            mbar_init(&C.o_full[a], 2);
        }
        for (int s = 0; s < kSched; ++s) {
            mbar_init(&C.sched_full[s], 1);
            mbar_init(&C.sched_empty[s], kSchedReaders);
        }
        mbar_init(&C.drained, 1);
        for (int i = 0; i < 8; ++i) C.poisoned[i] = 0;
        C.gave_up = 0;
        fence_barrier_init();
    }
    if (warp == kWarpMmaP) tmem_alloc(&C.tmem, 512);
    if (warp == kWarpLoad && lane == 0) {
        prefetch_map(&q_map);
        prefetch_map(&k_map);
        prefetch_map(&v_map);
    }
    // Units of each thread's prompts.
    const int per = (A.B + kScan - 1) / kScan;
    auto prompt = [&](int b, int &row0) {
        row0 = min(max(A.row_off[b], 0), A.rows);
        return min(min(max(A.row_off[b + 1], row0), A.rows) - row0, A.q_max);
    };
    int mine = 0;
    for (int b = min(tid * per, A.B); tid < kScan && b < min(tid * per + per, A.B); ++b) {
        int row0;
        mine += (prompt(b, row0) + 2 * kTile - 1) / (2 * kTile);
    }
    int sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += x;
    }
    if (lane == 31 && tid < kScan) C.warp_sum[warp] = sum;
    __syncthreads();
    if (tid < kScan) {
        for (int w = 0; w < warp; ++w) sum += C.warp_sum[w];
        C.pairs[tid] = sum - mine;
        if (tid == kScan - 1) C.pairs[kScan] = sum;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = C.tmem;

    if (warp == kWarpLoad) {
        // ---- units, and their queries, keys and values -----------------------
        const int total = C.pairs[kScan] * A.Hq;  // at most 2^17 * 2^8
        Ring rs, rk, rv;
        uint32_t q_uses[2] = {0, 0};
        int issued[2] = {0, 0}, published = 0;
        bool ok = true;
        // The next unit off the counter, published to the other warps.
        auto claim = [&] {
            Unit u{0, 0, 0, -1};
            int idx = 0;
            if (lane == 0) idx = atomicAdd(A.counter, 1);
            idx = __shfl_sync(0xffffffffu, idx, 0);
            if (idx < total) {
                const int pair = idx / A.Hq;
                u.h = idx - pair * A.Hq;
                int lo = 0, hi = kScan;  // the thread whose prompts hold it
                while (hi - lo > 1) {
                    const int mid = (lo + hi) / 2;
                    if (C.pairs[mid] <= pair) lo = mid; else hi = mid;
                }
                int left = pair - C.pairs[lo];
                for (int b = lo * per; b < A.B; ++b) {
                    u.n = prompt(b, u.row0);
                    const int units = (u.n + 2 * kTile - 1) / (2 * kTile);
                    if (left < units) {
                        u.q0 = (units - 1 - left) * 2 * kTile;  // the longest first
                        break;
                    }
                    left -= units;
                }
            }
            if (published >= kSched)
                ok = wait_or_give_up(&C.sched_empty[rs.slot], rs.phase ^ 1, A.wait_ns, gave_up);
            ok = __all_sync(0xffffffffu, ok);
            if (ok && lane == 0) {
                C.unit[rs.slot] = u;
                mbar_arrive(&C.sched_full[rs.slot]);
            }
            __syncwarp();
            rs.next(kSched);
            ++published;
            return u;
        };
        Unit ahead = claim();
        while (ok && ahead.h >= 0) {
            const Unit u = ahead;
            ahead = claim();
            if (!ok) break;
            const Span s0 = span_of(A, u, 0), s1 = span_of(A, u, 1);
            const int t_lo = s0.lo, t_hi = max(s0.hi, s1.hi), kvh = u.h / A.G;
            for (int a = 0; a < 2 && ok; ++a) {
                if (a == 1 && s1.hi == 0) break;
                if (q_uses[a] > 0) ok = wait_or_give_up(&C.q_empty[a], (q_uses[a] - 1) & 1, A.wait_ns, gave_up);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                if (elect_one()) {
                    mbar_arrive_expect_tx(&C.q_full[a], kSlotBytes);
                    for (int hf = 0; hf < kHalves; ++hf)
                        tma_load_3d(q_smem + a * kSlotBytes + hf * kHalfBytes, &q_map, &C.q_full[a], hf * 64, u.h,
                                    u.row0 + u.q0 + a * kTile);
                }
                __syncwarp();
                ++q_uses[a];
            }
            for (int t = t_lo; t < t_hi && ok; ++t) {
#pragma unroll
                for (int kv = 0; kv < 2; ++kv) {
                    Ring &r = kv ? rv : rk;
                    const int slots = kv ? v_slots : A.k_slots, slot = (kv ? A.k_slots : 0) + r.slot;
                    if (issued[kv] >= slots) ok = wait_or_give_up(&C.empty[slot], r.phase ^ 1, A.wait_ns, gave_up);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    if (elect_one()) {
                        mbar_arrive_expect_tx(&C.full[slot], kSlotBytes);
                        for (int hf = 0; hf < kHalves; ++hf)
                            tma_load_3d(ring + slot * kSlotBytes + hf * kHalfBytes, kv ? &v_map : &k_map, &C.full[slot],
                                        hf * 64, kvh, u.row0 + t * kTile);
                    }
                    __syncwarp();
                    r.next(slots);
                    ++issued[kv];
                }
            }
        }
        if (C.gave_up) {
            // Let the copies in flight land before the CTA ends.
            for (int kv = 0; kv < 2; ++kv) {
                const int slots = kv ? v_slots : A.k_slots;
                for (int k = max(issued[kv] - slots, 0); k < issued[kv]; ++k)
                    mbar_wait_bounded(&C.full[(kv ? A.k_slots : 0) + k % slots], (k / slots) & 1, kDrainTimeoutNs);
            }
            for (int a = 0; a < 2; ++a)
                if (q_uses[a]) mbar_wait_bounded(&C.q_full[a], (q_uses[a] - 1) & 1, kDrainTimeoutNs);
        }
        if (lane == 0) {
            // The last CTA leaves the counter as the next call wants it.
            __threadfence();
            if (atomicAdd(A.counter + 1, 1) == int(gridDim.x) - 1) {
                A.counter[0] = 0;
                A.counter[1] = 0;
            }
        }
    } else if (warp == kWarpMmaP) {
        // ---- MMA issuer -----------------------------------------------------
        const uint64_t qd = smem_desc(q_smem, 16, 1024), kd0 = smem_desc(ring, 16, 1024);
        const uint64_t vd0 = smem_desc(v_ring, kHalfBytes, 1024);
        constexpr uint32_t id_s = mma_idesc(128, kTile, false, false), id_o = mma_idesc(128, D, false, true);
        SchedReader sched;
        Ring rk, rv;
        uint32_t q_uses[2] = {0, 0}, p_uses[2] = {0, 0};
        bool ok = true;
        auto warp_test = [&](uint64_t *bar, uint32_t phase) {
            return __all_sync(0xffffffffu, mbar_test_wait(bar, phase));
        };
        auto wait = [&](uint64_t *bar, uint32_t phase) {
            ok = ok && wait_or_give_up(bar, phase, A.wait_ns, gave_up);
            ok = __all_sync(0xffffffffu, ok);
        };
        struct Work { Unit u; Span sp[2]; int lo, hi; };
        auto fetch = [&] {
            Work w;
            w.u = sched.next(C, A, gave_up, lane);
            w.sp[0] = w.u.h < 0 ? Span{0, 0} : span_of(A, w.u, 0);
            w.sp[1] = w.u.h < 0 ? Span{0, 0} : span_of(A, w.u, 1);
            w.lo = w.sp[0].lo;
            w.hi = max(w.sp[0].hi, w.sp[1].hi);
            return w;
        };
        // S of block a and tile t, whose K is in slot rk
        auto issue_s = [&](const Work &w, int a, int t) {
            if (t < w.sp[a].lo || t >= w.sp[a].hi) return;
            if (t == w.sp[a].lo) {
                wait(&C.q_full[a], q_uses[a] & 1);
                ++q_uses[a];
            }
            wait(&C.full[rk.slot], rk.phase);
            if (!ok) return;
            tc_fence_after();
            if (elect_one()) {
                const uint64_t kd = kd0 + uint32_t(rk.slot) * (kSlotBytes >> 4);
#pragma unroll
                for (int d = 0; d < D / 16; ++d) {
                    const uint32_t at = ((d / 4) * kHalfBytes + (d % 4) * 32) >> 4;
                    mma_ss(tmem + a * kTile, qd + a * (kSlotBytes >> 4) + at, kd + at, id_s, d > 0);
                }
                mma_commit(&C.s_full[a]);
                if (t == w.sp[a].hi - 1) mma_commit(&C.q_empty[a]);
            }
            __syncwarp();
        };
        auto free_k = [&] {
            if (elect_one()) mma_commit(&C.empty[rk.slot]);
            __syncwarp();
            rk.next(A.k_slots);
        };
        Work w = fetch();
        for (int a = 0; a < 2 && ok; ++a) issue_s(w, a, w.lo);
        if (w.hi > 0 && ok) free_k();
        while (ok && w.hi > 0) {
            Work nx = w;
            for (int t = w.lo; t < w.hi && ok; ++t) {
                // S of the step after this one goes between the two blocks'
                // products; at a unit's end that is the next unit's.
                const bool last = t + 1 == w.hi;
                if (last) nx = fetch();
                const int tn = last ? nx.lo : t + 1;
                const bool more = tn < nx.hi;
                bool s0_late = false;
#pragma unroll
                for (int a = 0; a < 2; ++a) {
                    if (t >= w.sp[a].lo && t < w.sp[a].hi) {
                        wait(&C.clean[A.k_slots + rv.slot], rv.phase);
                        const uint64_t vd = vd0 + uint32_t(rv.slot) * (kSlotBytes >> 4);
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            wait(&C.p_full[a][half], p_uses[a] & 1);
                            if (!ok) break;
                            tc_fence_after();
                            if (elect_one()) {
#pragma unroll
                                for (int k = 4 * half; k < 4 * half + 4; ++k)
                                    mma_ts(tmem + kColO + a * D, tmem + a * kTile + k * 8, vd + k * (2048 >> 4), id_o,
                                           !(t == w.sp[a].lo && k == 0));
                                if (half == 1 && t == w.sp[a].hi - 1) {
                                    mbar_arrive(&C.o_full[a]);  // passes the cleaners' word on
                                    mma_commit(&C.o_full[a]);
                                }
                            }
                            __syncwarp();
                        }
                        ++p_uses[a];
                    }
                    if (!ok) break;
                    if (!more) continue;
                    if (a == 0 && last && !(warp_test(&C.q_full[0], q_uses[0] & 1) && warp_test(&C.full[rk.slot], rk.phase)))
                        s0_late = true;  // not there yet: block 1's product goes first
                    else
                        issue_s(nx, a, tn);
                }
                if (!ok) break;
                if (s0_late) issue_s(nx, 0, tn);
                if (elect_one()) mma_commit(&C.empty[A.k_slots + rv.slot]);
                __syncwarp();
                rv.next(v_slots);
                if (more && ok) free_k();
            }
            w = nx;
        }
        if (C.gave_up) {
            if (elect_one()) mma_commit(&C.drained);
            __syncwarp();
            mbar_wait_bounded(&C.drained, 0, kDrainTimeoutNs);
        }
    } else if (warp >= kWarpClean) {
        // ---- cleaners: masked keys must not reach O through 0 * infinity.  A
        // value tile that some row does not see in full loses its NaN and
        // infinities; the epilogue adds them to the rows that see them. -----
        SchedReader sched;
        Ring rv;
        const int id = tid - kWarpClean * 32;
        bool ok = true;
        for (int unit = 0; ok; ++unit) {
            const Unit u = sched.next(C, A, gave_up, lane);
            if (u.h < 0) break;
            const Span s0 = span_of(A, u, 0), s1 = span_of(A, u, 1);
            for (int t = s0.lo; t < max(s0.hi, s1.hi); ++t) {
                const int slot = A.k_slots + rv.slot;
                ok = wait_or_give_up(&C.full[slot], rv.phase, A.wait_ns, gave_up);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                if ((t >= s0.lo && t < s0.hi && partial(A, u, 0, t)) ||
                    (t >= s1.lo && t < s1.hi && partial(A, u, 1, t))) {
                    const uint32_t at0 = v_ring + rv.slot * kSlotBytes + id * 16;
                    bool lost = false;
#pragma unroll 4
                    for (uint32_t c = 0; c < kSlotBytes; c += kCleaners * 16) {
                        const uint4 x = ld_shared16(at0 + c);
                        const uint32_t mx = nonfinite_mask(x.x), my = nonfinite_mask(x.y),
                                       mz = nonfinite_mask(x.z), mw = nonfinite_mask(x.w);
                        if (mx | my | mz | mw) {
                            st_shared16(at0 + c, x.x & ~mx, x.y & ~my, x.z & ~mz, x.w & ~mw);
                            lost = true;
                        }
                    }
                    if (lost) C.poisoned[unit % 8] = unit + 1;
                    fence_async_shared();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&C.clean[slot]);
                rv.next(v_slots);
            }
        }
    } else {
        // ---- softmax and output: thread = row of block a -----------------------
        const int a = warp >> 2, row = tid & 127;
        const uint32_t lane_tm = tmem + (uint32_t((warp & 3) * 32) << 16);
        const uint32_t s_tm = lane_tm + a * kTile, o_tm = lane_tm + kColO + a * D;
        SchedReader sched;
        uint32_t s_uses = 0, o_uses = 0;
        bool ok = true;
        for (int unit = 0; ok; ++unit) {
            const Unit u = sched.next(C, A, gave_up, lane);
            if (u.h < 0) break;
            const Span sp = span_of(A, u, a);
            if (sp.hi == 0) continue;
            const int q = u.q0 + a * kTile + row;  // the thread's row; past the prompt: computed, not stored
            float ref = 0.f;
            float2 l2 = make_float2(0.f, 0.f);
            for (int t = sp.lo; t < sp.hi; ++t) {
                ok = wait_or_give_up(&C.s_full[a], s_uses & 1, A.wait_ns, gave_up);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                ++s_uses;
                tc_fence_after();
                float s[kTile];
#pragma unroll
                for (int c = 0; c < kTile; c += 32) tmem_ld32(s + c, s_tm + c);
                asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
                for (int c = 0; c < kTile; c += 32) tmem_use32(s + c);
                if (partial(A, u, a, t)) {
                    // The row sees keys (lo, hi] of the tile.  By 32 keys, what
                    // the warp's rows all see stays as it is.
                    const int hi = q - t * kTile, lo = A.window > 0 ? hi - A.window : -1;
                    const int hi0 = hi - lane, lo31 = lo + 31 - lane;  // its first row's, its last row's
#pragma unroll
                    for (int c = 0; c < kTile; c += 32) {
                        if (c + 31 > hi0) {
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (c + e > hi) s[c + e] = -INFINITY;
                        }
                        if (A.window > 0 && c <= lo31) {
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (c + e <= lo) s[c + e] = -INFINITY;
                        }
                    }
                }
                float m0 = max3(s[0], s[1], s[2]), m1 = max3(s[3], s[4], s[5]);
#pragma unroll
                for (int e = 6; e < kTile - 2; e += 4) {
                    m0 = max3(m0, s[e], s[e + 1]);
                    m1 = max3(m1, s[e + 2], s[e + 3]);
                }
                const float m = max3(m0, m1, fmaxf(s[kTile - 2], s[kTile - 1])) * A.scale2;
                if (t == sp.lo) {
                    ref = fmaxf(m, kRefMin);
                } else if (__any_sync(0xffffffffu, m > ref + kRefSlack)) {
                    const float now = m > ref + kRefSlack ? m : ref;
                    const float f = exp2_approx(ref - now);
                    ref = now;
                    l2.x *= f;
                    l2.y *= f;
#pragma unroll
                    for (int c = 0; c < D; c += 16) {
                        float o[16];
                        tmem_ld16(o, o_tm + c);
                        tmem_wait_ld(o);
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[e] *= f;
                        tmem_st16(o_tm + c, o);
                    }
                }
                const float2 sc = make_float2(A.scale2, A.scale2), nr = make_float2(-ref, -ref);
#pragma unroll
                for (int c = 0; c < kTile; c += 32) {
                    uint32_t p[16];
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        float2 x = fma2(make_float2(s[c + e], s[c + e + 1]), sc, nr);
                        x.x = exp2_approx(x.x);
                        x.y = exp2_approx(x.y);
                        l2 = add2(l2, x);
                        p[e / 2] = pack_bf16x2(x.x, x.y);
                    }
                    tmem_st16u(s_tm + c / 2, p);
                    if (c % 64 == 32) {  // half of the keys: their product may begin
                        tmem_wait_st();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&C.p_full[a][c / 64]);
                    }
                }
            }
            if (!ok) break;
            ok = wait_or_give_up(&C.o_full[a], o_uses & 1, A.wait_ns, gave_up);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            ++o_uses;
            tc_fence_after();
            const float l = l2.x + l2.y, inv = l == 0.f ? 0.f : 1.f / l;
            uint16_t *const out = A.out + ((int64_t)(u.row0 + q) * A.Hq + u.h) * D;
            // 64 entries of the warp's 32 rows at a time go through shared
            // memory, so that eight lanes write a row's 128 bytes.
            const uint32_t mine = stage + warp * 4096;
#pragma unroll
            for (int c = 0; c < D; c += 64) {
#pragma unroll
                for (int half = 0; half < 64; half += 32) {
                    float o[32];
                    tmem_ld32(o, o_tm + c + half);
                    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
                    tmem_use32(o);
#pragma unroll
                    for (int e = 0; e < 32; e += 8)
                        st_shared16(mine + lane * 128 + ((((half + e) / 8) ^ (lane & 7)) << 4),
                                    pack_bf16x2(o[e] * inv, o[e + 1] * inv), pack_bf16x2(o[e + 2] * inv, o[e + 3] * inv),
                                    pack_bf16x2(o[e + 4] * inv, o[e + 5] * inv), pack_bf16x2(o[e + 6] * inv, o[e + 7] * inv));
                }
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 32; i += 4) {
                    const int r = i + lane / 8, ch = lane % 8;
                    if (q - lane + r < u.n)
                        *reinterpret_cast<uint4 *>(out + (int64_t)(r - lane) * A.Hq * D + c + ch * 8) =
                            ld_shared16(mine + r * 128 + ((ch ^ (r & 7)) << 4));
                }
                __syncwarp();
            }
            tc_fence_before();
            __syncwarp();  // the row was written by other lanes
            if (C.poisoned[unit % 8] == unit + 1 && q < u.n) {
                // what the cleaners took out of the values that this row sees
                for (int t = sp.lo; t < sp.hi; ++t) {
                    const bool mixed = partial(A, u, a, t) ||
                                       (span_of(A, u, a ^ 1).hi > t && span_of(A, u, a ^ 1).lo <= t && partial(A, u, a ^ 1, t));
                    if (!mixed) continue;
                    for (int k = t * kTile; k < min((t + 1) * kTile, q + 1); ++k) {
                        if (A.window > 0 && k <= q - A.window) continue;
                        const uint16_t *v = A.v + (int64_t)(u.row0 + k) * A.v_stride + (u.h / A.G) * D;
                        for (int d = 0; d < D; ++d) {
                            const float x = bf16_lo(v[d]);
                            if (!isfinite(x)) out[d] = uint16_t(pack_bf16x2(bf16_lo(out[d]) + x, 0.f));
                        }
                    }
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (tid == 0 && C.gave_up) atomicOr(A.status, kStatusWaitTimeout);
    if (warp == kWarpMmaP) tmem_free(tmem, 512);
}

template <int D>
cudaError_t launch(PromptArgs A, const CUtensorMap (&maps)[3], int ctas, cudaStream_t s) {
    const size_t slot = size_t(D) * 2 * kTile;
    constexpr size_t stage = 8 * 4096;
    A.slots = int(std::min<size_t>((kSmemBytes - sizeof(Ctrl) - 1024 - stage - 2 * slot) / slot, kSlotsMax));
    A.k_slots = A.slots / 2;
    const size_t smem = 1024 + (2 + A.slots) * slot + stage;
    const cudaError_t e = cudaFuncSetAttribute(prompt_attention_kernel<D>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
    if (e != cudaSuccess) return e;
    prompt_attention_kernel<D><<<ctas, kThreadsP, smem, s>>>(A, maps[0], maps[1], maps[2]);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prompt_attention(const dspark_attn &a, int sms, uint64_t wait_ns, cudaStream_t s) {
    PromptArgs A{};
    A.B = a.B; A.rows = a.rows; A.q_max = a.q_max; A.Hq = a.Hq; A.Hkv = a.Hkv; A.G = a.Hq / a.Hkv;
    A.window = a.window;
    A.scale2 = float(double(a.scale) * 1.4426950408889634);
    A.v_stride = a.v_stride;
    A.v = static_cast<const uint16_t *>(a.v);
    A.row_off = a.row_off;
    A.out = static_cast<uint16_t *>(a.out);
    A.status = static_cast<int32_t *>(a.workspace);
    A.counter = static_cast<int32_t *>(a.workspace) + 1;
    A.wait_ns = wait_ns;
    CUtensorMap maps[3];
    const void *base[3] = {a.q_rot, a.k_rot, a.v};
    const int heads[3] = {a.Hq, a.Hkv, a.Hkv};
    const int64_t stride[3] = {(int64_t)a.Hq * a.D, (int64_t)a.Hkv * a.D, a.v_stride};
    for (int i = 0; i < 3; ++i) {
        const uint64_t dims[3] = {uint64_t(a.D), uint64_t(heads[i]), uint64_t(a.rows)};
        const uint64_t st[2] = {uint64_t(a.D) * 2, uint64_t(stride[i]) * 2};
        const uint32_t box[3] = {64, 1, kTile};
        const cudaError_t e = encode_map(&maps[i], base[i], 3, dims, st, box);
        if (e != cudaSuccess) return e;
    }
    const int ctas = std::min(sms, kAttnMaxCtas);
    return a.D == 128 ? launch<128>(A, maps, ctas, s) : launch<64>(A, maps, ctas, s);
}

}  // namespace dspark
