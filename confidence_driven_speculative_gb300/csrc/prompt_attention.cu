// prompt_attention.cu -- whole prompts, causal, packed one after the other.
//
// Mathematics.  For a block of rows of one query head: S = Q K^T, the weights
// P = 2^(scale log2(e) S - m) against a running reference m per row, l the
// sum of P, O += P V; the output is O / l.  The reference lies 16 above the first
// tile's maximum; a later tile moves it, and rescales O and l, only where a score
// passes it, which is next to never (with 8 in place of 16: long 358 us against
// 353).  So no weight passes 1, and O overflows only where the values' own sum
// does; a row's largest weight is 2^-16 or about that, which fp32 sums and
// bfloat16 hold with an unchanged relative step.
//
// The weights are rounded to bfloat16 for the tensor core, by a relative 2^-8
// at most; l sums the rounded ones, in registers, so that the errors of numerator
// and denominator partly cancel: 0.0020 of the output's norm against 0.0023 with
// the unrounded ones, where the output's own rounding is 0.0017 (and values that are
// all alike come out as they are).  Additions that take a bfloat16 operand
// cost next to nothing for that; widening the weights first does (packed 238 us
// against 234, after P has gone out 241).
//
// Bound: the tensor cores.  A unit is 256 rows of one head in two blocks of
// 128, walked over tiles of 128 keys.  S and O of both blocks fill TMEM
// (4 x 128 columns); P overwrites its S in TMEM and is the A operand of
// P V.  While one block's softmax runs, the tensor cores work on the other
// block: O_0 += P_0 V with S_0 of the next tile, then O_1 += P_1 V with S_1.
// Two threads share a row, 64 keys each: one thread a row had twice the chain
// of exponentials between two products (in an earlier version 359 us against 346
// for the long prompt below).
//
// Units are handed out by a counter, the longest of a prompt first, so the
// CTAs end together; a unit's result does not depend on who computes it.
//
// Measured, D = 128: one prompt of 8192 rows and 32 heads 346 to 350 us in loops
// of seconds, under the power limit, 1.58 PFLOP/s where a library product keeps up
// 1.72; in a burst of 15 ms at 2070 MHz 316 us, 1.74 against 1.91.  24 prompts of
// 20 to 2000 rows and 40 heads 233 to 236 us (228 in a burst), 113 at the library's
// rate.  A step's products are 2048 clocks by the tensor cores' nominal rate and
// 2770 at the library's; a step takes about 2900.  The softmax hides behind that:
// without the halves' vote (240 clocks of a block's chain) an earlier version took
// 319 us against 321 in a burst.  A unit's border costs some 4000 clocks more (last
// product, outputs, diagonal masks), and short prompts have few steps to a unit.
#include <algorithm>
#include <cmath>

#include "attn.cuh"
#include "dspark_internal.cuh"
#include "tcgen05.cuh"

namespace dspark {
namespace {

constexpr int kTile = 128;        // rows of a block, keys of a tile
constexpr int kThreadsP = 640;
constexpr int kScan = 128;        // threads that sum up the prompts' units
constexpr int kWarpMma = 0, kWarpLoad = 1, kWarpReady = 2, kWarpSoft = 4;  // 3: idle; softmax 4..19
constexpr int kSlotsMax = 10;
constexpr int kSched = 4;         // units on their way to the warps
constexpr int kSchedReaders = 18; // warps that read them
constexpr float kRefMin = -3.402823466e38f;  // reference of a row without a score yet: no score is lower
constexpr float kHeadroom = 16.0f;  // log2: the reference over the maximum that sets it
// log2: from here on a reference is far.  A weight is 2^(s * scale - reference), fused, so half a step of the
// rounded reference is an error of the exponent, the same for all of a row: 2^4 below this limit, more than
// fp32's range from 2^32 on.  A far row is scaled by a power of two instead: its products are exact.  That
// changes no weight that counts: fp32 scores of that size are equal or lie 2^4 apart at least.  (Rounding the
// products instead, in all rows: packed 231 us against 236, long 349 against 358.)
constexpr float kFar = 536870912.0f;
constexpr size_t kSmemBytes = 232448;

struct PromptArgs {
    int B, rows, q_max, Hq, Hkv, G, window;
    int slots, k_slots;
    int wide_out;      // out is 32-byte aligned
    float scale2;      // scale * log2(e)
    float far_scale;   // the power of two at or above it
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
template <bool kWindow>
__device__ __forceinline__ Span span_of(const PromptArgs &A, const Unit &u, int a) {
    const int q = u.q0 + a * kTile;
    if (q >= u.n) return {0, 0};
    Span s;
    s.lo = kWindow ? max(q - A.window + 1, 0) / kTile : 0;
    s.hi = (min(q + kTile, u.n) + kTile - 1) / kTile;
    return s;
}
// Does some row of block a not see some key of tile t?
template <bool kWindow>
__device__ __forceinline__ bool partial(const PromptArgs &A, const Unit &u, int a, int t) {
    const int q = u.q0 + a * kTile;
    return (t + 1) * kTile - 1 > q || (kWindow && t * kTile <= min(q + kTile, u.n) - 1 - A.window);
}

struct Ctrl {
    uint64_t full[kSlotsMax], empty[kSlotsMax];
    uint64_t q_full[2], q_empty[2], s_full[2], o_full[2];
    uint64_t p_full[2];       // P is written, and V of its tile and K of the next one are there
    uint64_t sched_full[kSched], sched_empty[kSched], drained;
    Unit unit[kSched];
    int poisoned[8];          // by unit number % 8: the last unit + 1 that lost values
    int pairs[kScan + 1];     // exclusive sums of the units (per head) of each thread's prompts
    int warp_sum[kScan / 32];
    float swap[2][2][2][kTile];  // between the two threads of a row (maxima, sums): by block and half
    uint32_t tmem;
    int issued[2], q_issued[2];  // copies of K and V tiles, of the blocks' queries
    int gave_up;
};

// 16 bfloat16 of one row: a whole sector where the alignment allows.
__device__ __forceinline__ void st_global32(uint16_t *p, const uint32_t (&y)[8], bool wide) {
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                     ::"l"(p), "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3]), "r"(y[4]), "r"(y[5]), "r"(y[6]), "r"(y[7])
                     : "memory");
    } else {
        reinterpret_cast<uint4 *>(p)[0] = make_uint4(y[0], y[1], y[2], y[3]);
        reinterpret_cast<uint4 *>(p)[1] = make_uint4(y[4], y[5], y[6], y[7]);
    }
}

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

// kWindow: is there one?  Code that an unwindowed call does not run is code that
// its warps need not fetch past.
template <int D, bool kWindow>
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
    volatile int *gave_up = &C.gave_up;

    if (tid == 0) {
        for (int s = 0; s < A.slots; ++s) {
            mbar_init(&C.full[s], 1);
            mbar_init(&C.empty[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&C.q_full[a], 1);
            mbar_init(&C.q_empty[a], 1);
            mbar_init(&C.s_full[a], 1);
            mbar_init(&C.p_full[a], 9);
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
    if (warp == kWarpMma) tmem_alloc(&C.tmem, 512);
    if (warp == kWarpLoad && lane == 0) {
        prefetch_map(&q_map);
        prefetch_map(&k_map);
        prefetch_map(&v_map);
    }
    // Nothing before this line reads or writes memory that another kernel may
    // touch: the launch may overlap the end of the kernel before it.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
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
            const Span s0 = span_of<kWindow>(A, u, 0), s1 = span_of<kWindow>(A, u, 1);
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
        if (lane == 0) {
            for (int a = 0; a < 2; ++a) {  // for the CTA's end, should a wait have given up
                C.issued[a] = issued[a];
                C.q_issued[a] = int(q_uses[a]);
            }
            // The last CTA leaves the counter as the next call wants it.
            __threadfence();
            if (atomicAdd(A.counter + 1, 1) == int(gridDim.x) - 1) {
                A.counter[0] = 0;
                A.counter[1] = 0;
            }
        }
    } else if (warp == kWarpMma) {
        // ---- MMA issuer -----------------------------------------------------
        const uint64_t qd = smem_desc(q_smem, 16, 1024), kd0 = smem_desc(ring, 16, 1024);
        const uint64_t vd0 = smem_desc(v_ring, kHalfBytes, 1024);
        constexpr uint32_t id_s = mma_idesc(128, kTile, false, false), id_o = mma_idesc(128, D, false, true);
        SchedReader sched;
        Ring rk, rv;
        uint32_t q_phase[2] = {0, 0}, p_phase[2] = {0, 0};
        bool ok = true;
        auto wait = [&](uint64_t *bar, uint32_t phase) {
            ok = ok && wait_or_give_up(bar, phase, A.wait_ns, gave_up);
            ok = __all_sync(0xffffffffu, ok);
        };
        // A unit's tiles.  They come from lane 0 by shuffles, which the
        // compiler knows to be the same in all lanes.
        struct Work { Span sp[2]; int lo, hi; };
        auto fetch = [&] {
            Work w;
            const Unit u = sched.next(C, A, gave_up, lane);
#pragma unroll
            for (int a = 0; a < 2; ++a) {
                w.sp[a] = u.h < 0 ? Span{0, 0} : span_of<kWindow>(A, u, a);
                w.sp[a].lo = __shfl_sync(0xffffffffu, w.sp[a].lo, 0);
                w.sp[a].hi = __shfl_sync(0xffffffffu, w.sp[a].hi, 0);
            }
            w.lo = w.sp[0].lo;
            w.hi = max(w.sp[0].hi, w.sp[1].hi);
            return w;
        };
        auto has = [](const Span &s, int t) { return t >= s.lo && t < s.hi; };
        // S of block a and the tile whose K is in slot rk; by one lane
        auto issue_s = [&](int a, bool last) {
            const uint64_t kd = kd0 + uint32_t(rk.slot) * (kSlotBytes >> 4);
#pragma unroll
            for (int d = 0; d < D / 16; ++d) {
                const uint32_t at = ((d / 4) * kHalfBytes + (d % 4) * 32) >> 4;
                mma_ss(tmem + a * kTile, qd + a * (kSlotBytes >> 4) + at, kd + at, id_s, d > 0);
            }
            mma_commit(&C.s_full[a]);
            if (last) mma_commit(&C.q_empty[a]);
        };
        Work w = fetch();
        if (w.hi > 0) {
            wait(&C.full[rk.slot], rk.phase);
            for (int a = 0; a < 2; ++a) {
                if (!has(w.sp[a], w.lo)) continue;
                wait(&C.q_full[a], q_phase[a]);
                q_phase[a] ^= 1;
                tc_fence_after();
                if (elect_one()) issue_s(a, w.sp[a].hi == w.lo + 1);
                __syncwarp();
            }
            if (elect_one()) mma_commit(&C.empty[rk.slot]);
            __syncwarp();
            rk.next(A.k_slots);
        }
        // O += P V of block a's tile, whose V is in slot rv; by one lane
        auto issue_o = [&](int a, bool first) {
            const uint64_t vd = vd0 + uint32_t(rv.slot) * (kSlotBytes >> 4);
#pragma unroll
            for (int k = 0; k < kTile / 16; ++k)
                mma_ts(tmem + kColO + a * D, tmem + a * kTile + k * 8, vd + k * (2048 >> 4), id_o, !(first && k == 0));
        };
        while (ok && w.hi > 0) {
            Work nx = w;
            // O += P V of a step and S of the next one go out together for a
            // block: 16 products behind one wait, since the tensor cores queue
            // hardly any and idle while this warp waits and tests.
            for (int t = w.lo; t < w.hi && ok; ++t) {
                if (t > w.sp[0].lo && t > w.sp[1].lo && t + 1 < w.sp[0].hi && t + 1 < w.sp[1].hi) {
                    // both blocks, neither at an end: as little as can be
#pragma unroll
                    for (int a = 0; a < 2; ++a) {
                        wait(&C.p_full[a], p_phase[a]);
                        p_phase[a] ^= 1;
                        tc_fence_after();
                        if (elect_one()) {
                            issue_o(a, false);
                            issue_s(a, t + 2 == w.sp[a].hi);
                            if (a == 1) {
                                mma_commit(&C.empty[A.k_slots + rv.slot]);
                                mma_commit(&C.empty[rk.slot]);
                            }
                        }
                        __syncwarp();
                    }
                    rv.next(v_slots);
                    rk.next(A.k_slots);
                    continue;
                }
                const bool last = t + 1 == w.hi;
                if (last) nx = fetch();  // S of the next step is the next unit's
                const int tn = last ? nx.lo : t + 1;
                const bool more = tn < nx.hi;
#pragma unroll
                for (int a = 0; a < 2; ++a) {
                    const bool pv = has(w.sp[a], t), s = more && has(nx.sp[a], tn);
                    if (s && tn == nx.sp[a].lo) {
                        wait(&C.q_full[a], q_phase[a]);
                        q_phase[a] ^= 1;
                    }
                    if (pv) {
                        wait(&C.p_full[a], p_phase[a]);
                        p_phase[a] ^= 1;
                    } else if (s) {
                        wait(&C.full[rk.slot], rk.phase);
                    }
                    if (!ok) break;
                    tc_fence_after();
                    if (elect_one()) {
                        if (pv) {
                            issue_o(a, t == w.sp[a].lo);
                            if (t == w.sp[a].hi - 1) {
                                mbar_arrive(&C.o_full[a]);  // passes on what was lost of V
                                mma_commit(&C.o_full[a]);
                            }
                        }
                        if (s) issue_s(a, tn == nx.sp[a].hi - 1);
                        if (a == 1) {
                            mma_commit(&C.empty[A.k_slots + rv.slot]);
                            if (more) mma_commit(&C.empty[rk.slot]);
                        }
                    }
                    __syncwarp();
                }
                rv.next(v_slots);
                if (more) rk.next(A.k_slots);
            }
            w = nx;
        }
    } else if (warp == kWarpReady) {
        // ---- the last of P's arrivals: V of its tile and K of the next are there,
        // so that the MMA issuer has one barrier to test and not three ----------
        SchedReader sched;
        Ring rk, rv;
        uint32_t uses[2] = {0, 0};
        bool ok = true;
        Unit u = sched.next(C, A, gave_up, lane);
        // The first K, which the MMA issuer waits for itself: a wait for a slot's next use is good only once
        // the use before has landed.
        if (u.h >= 0) ok = poll_or_give_up(&C.full[rk.slot], rk.phase, A.wait_ns, gave_up);
        rk.next(A.k_slots);
        ok = __all_sync(0xffffffffu, ok);
        while (ok && u.h >= 0) {
            const Span sp[2] = {span_of<kWindow>(A, u, 0), span_of<kWindow>(A, u, 1)};
            const int t_hi = max(sp[0].hi, sp[1].hi);
            Unit nx = u;
            for (int t = sp[0].lo; t < t_hi && ok; ++t) {
                ok = wait_or_give_up(&C.full[A.k_slots + rv.slot], rv.phase, A.wait_ns, gave_up);
                if (t + 1 == t_hi) nx = sched.next(C, A, gave_up, lane);
                if (nx.h >= 0) {
                    ok = ok && wait_or_give_up(&C.full[rk.slot], rk.phase, A.wait_ns, gave_up);
                    rk.next(A.k_slots);
                }
#pragma unroll
                for (int a = 0; a < 2; ++a) {
                    if (t < sp[a].lo || t >= sp[a].hi) continue;
                    // not before the tile before is through
                    if (uses[a] > 0)
                        ok = ok && wait_or_give_up(&C.p_full[a], (uses[a] - 1) & 1, A.wait_ns, gave_up);
                    ++uses[a];
                    ok = __all_sync(0xffffffffu, ok);
                    if (ok && lane == 0) mbar_arrive(&C.p_full[a]);
                }
                ok = __all_sync(0xffffffffu, ok);
                rv.next(v_slots);
            }
            u = nx;
        }
    } else if (warp >= kWarpSoft) {
        // ---- softmax and output --------------------------------------------------
        // Two threads share a row of block a: thread `half` takes 64 keys of
        // each tile, and 64 (32) entries of O.  The halves' warps meet twice
        // where they must: both have read S before either writes P over it,
        // and both know of a reference that moves.
        const int sw = warp - kWarpSoft, a = sw >> 3, half = (sw >> 2) & 1, row = (warp & 3) * 32 + lane;
        constexpr int kKeys = kTile / 2, kEntries = D / 2;
        const uint32_t lane_tm = tmem + (uint32_t((warp & 3) * 32) << 16);
        const uint32_t s_tm = lane_tm + a * kTile, o_tm = lane_tm + kColO + a * D + half * kEntries;
        const uint32_t pair_bar = 1 + a * 4 + (warp & 3);
        auto pair_any = [&](bool x) {
            uint32_t r;
            asm volatile(
                "{\n\t.reg .pred p, q;\n\t"
                "setp.ne.u32 q, %2, 0;\n\t"
                "barrier.cta.red.or.pred p, %1, 64, q;\n\t"
                "selp.u32 %0, 1, 0, p;\n\t}"
                : "=r"(r) : "r"(pair_bar), "r"(uint32_t(x)) : "memory");
            return r != 0;
        };
        auto pair_sync = [&] { asm volatile("barrier.cta.sync %0, 64;" ::"r"(pair_bar) : "memory"); };
        // The other thread's x.  A pair_any lies between two uses of a kind.
        auto exchange = [&](int kind, float x) {
            C.swap[kind][a][half][row] = x;
            pair_sync();
            return C.swap[kind][a][half ^ 1][row];
        };
        SchedReader sched;
        Ring rv;  // of the block's next tile
        uint32_t s_uses = 0, o_uses = 0;
        for (int unit = 0;; ++unit) {
            const Unit u = sched.next(C, A, gave_up, lane);
            if (pair_any(u.h < 0)) break;
            const Span sp = span_of<kWindow>(A, u, a), other = span_of<kWindow>(A, u, a ^ 1);
            const int t_lo = a ? other.lo : sp.lo, t_hi = max(sp.hi, other.hi);
            for (int t = t_lo; t < (sp.hi == 0 ? t_hi : sp.lo); ++t) rv.next(v_slots);
            if (sp.hi == 0) continue;
            const int q = u.q0 + a * kTile + row;  // the row; past the prompt: computed, not stored
            float ref = 0.f, scale2 = A.scale2;  // the row's; far_scale where its scores are far
            float2 l2 = make_float2(0.f, 0.f);
            // Once a wait has given up, the others return at once and the
            // loops run to their ends on whatever there is; the status tells.
            for (int t = sp.lo; t < sp.hi; ++t) {
                const bool cut = partial<kWindow>(A, u, a, t);
                // Masked keys must not reach O through 0 * infinity: a value
                // tile that some row does not see in full loses its NaN and
                // infinities; the rows that see them get them back at the
                // unit's end.  Of a tile that both blocks walk, block 0 does it
                // for both: its P comes before either block's products with
                // that tile, so both read it clean, and both outputs come after
                // the mark.  The tile's scores are still being made.
                bool clean = cut;
                if (kWindow && t >= other.lo && t < other.hi) clean = a == 0 && (cut || partial<kWindow>(A, u, 1, t));
                if (clean) {
                    // The wait for V is good only once the slot's use before has landed: a parity tells two
                    // phases apart, not three.  The block's waits so far say so (a tile's scores are issued
                    // after the products of the tile two before) but in two places that a window makes: block
                    // 1's first tile, since it skips units without a wait, and block 0's second one where V
                    // has two slots.  There the tile's own scores say it.
                    if (kWindow && (a ? t == sp.lo : t == sp.lo + 1 && v_slots < 3))
                        wait_or_give_up(&C.s_full[a], s_uses & 1, A.wait_ns, gave_up);
                    wait_or_give_up(&C.full[A.k_slots + rv.slot], rv.phase, A.wait_ns, gave_up);
                    __syncwarp();
                    const uint32_t at0 = v_ring + rv.slot * kSlotBytes + (half * kTile + row) * 16;
                    bool odd = false;
#pragma unroll
                    for (uint32_t c = 0; c < kSlotBytes; c += 2 * kTile * 16) odd |= nonfinite_any(ld_shared16(at0 + c));
                    if (__builtin_expect(odd, 0)) {
#pragma unroll 1
                        for (uint32_t c = 0; c < kSlotBytes; c += 2 * kTile * 16) {
                            const uint4 x = ld_shared16(at0 + c);
                            st_shared16(at0 + c, x.x & ~nonfinite_mask(x.x), x.y & ~nonfinite_mask(x.y),
                                        x.z & ~nonfinite_mask(x.z), x.w & ~nonfinite_mask(x.w));
                        }
                        C.poisoned[unit % 8] = unit + 1;
                        fence_async_shared();
                    }
                }
                wait_or_give_up(&C.s_full[a], s_uses & 1, A.wait_ns, gave_up);
                __syncwarp();
                ++s_uses;
                tc_fence_after();
                float s[kKeys];
#pragma unroll
                for (int c = 0; c < kKeys; c += 32) tmem_ld32(s + c, s_tm + half * kKeys + c);
                asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
                for (int c = 0; c < kKeys; c += 32) tmem_use32(s + c);
                if (cut) {
                    // The row sees keys (lo, hi] of the half tile.
                    const int hi = q - t * kTile - half * kKeys, lo = kWindow ? hi - A.window : -1;
#pragma unroll
                    for (int c = 0; c < kKeys; c += 32) {
                        uint32_t seen = hi < c ? 0u : 0xffffffffu >> max(31 + c - hi, 0);
                        if (kWindow) seen &= lo < c ? 0xffffffffu : lo >= c + 31 ? 0u : 0xfffffffeu << (lo - c);
                        if (__all_sync(0xffffffffu, seen == 0xffffffffu)) continue;
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (!(seen >> e & 1)) s[c + e] = -INFINITY;
                    }
                }
                float m0 = max3(s[0], s[1], s[2]), m1 = max3(s[3], s[4], s[5]);
#pragma unroll
                for (int e = 6; e < kKeys - 2; e += 4) {
                    m0 = max3(m0, s[e], s[e + 1]);
                    m1 = max3(m1, s[e + 2], s[e + 3]);
                }
                const float m = max3(m0, m1, fmaxf(s[kKeys - 2], s[kKeys - 1]));
                const bool first = t == sp.lo;
                if (__builtin_expect(pair_any(first || m * scale2 > ref), 0)) {
                    const float top = fmaxf(m, exchange(0, m)), near = top * A.scale2 + kHeadroom;
                    const float to_scale = fabsf(near) > kFar ? A.far_scale : A.scale2;
                    const float to = fmaxf(top * to_scale + kHeadroom, kRefMin);
                    if (first) {
                        ref = to;
                        scale2 = to_scale;
                    } else {
                        // From near to far the difference is one of near values; from far to
                        // near it is beyond any exponent, and f is 0.
                        const bool moves = top * scale2 > ref;
                        const float f = moves ? exp2_approx(ref - (to_scale == scale2 ? to : near)) : 1.f;
                        if (moves) {
                            ref = to;
                            scale2 = to_scale;
                        }
                        l2.x *= f;
                        l2.y *= f;
#pragma unroll 1
                        for (int c = 0; c < kEntries; c += 16) {
                            float o[16];
                            tmem_ld16(o, o_tm + c);
                            tmem_wait_ld(o);
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] *= f;
                            tmem_st16(o_tm + c, o);
                        }
                        tmem_wait_st();
                        tc_fence_before();
                        pair_sync();  // all of O is rescaled before either half's P is used
                    }
                }
                const float2 sc = make_float2(scale2, scale2), nr = make_float2(-ref, -ref);
                float2 sums[2] = {l2, make_float2(0.f, 0.f)};
#pragma unroll
                for (int c = 0; c < kKeys; c += 32) {
                    uint32_t p[16];
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        const float2 x = fma2(make_float2(s[c + e], s[c + e + 1]), sc, nr);
                        p[e / 2] = pack_bf16x2(exp2_approx(x.x), exp2_approx(x.y));
                        add_bf16x2(sums[(e / 2) & 1], p[e / 2]);
                    }
                    tmem_st16u(s_tm + (half * kKeys + c) / 2, p);
                }
                rv.next(v_slots);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&C.p_full[a]);
                l2 = add2(sums[0], sums[1]);
            }
            for (int t = sp.hi; t < t_hi; ++t) rv.next(v_slots);
            const float mine = l2.x + l2.y, l = mine + exchange(1, mine), inv = l == 0.f ? 0.f : 1.f / l;
            wait_or_give_up(&C.o_full[a], o_uses & 1, A.wait_ns, gave_up);
            __syncwarp();
            ++o_uses;
            tc_fence_after();
            uint16_t *const out = A.out + ((int64_t)(u.row0 + q) * A.Hq + u.h) * D + half * kEntries;
#pragma unroll 1
            for (int c = 0; c < kEntries; c += 32) {
                float o[32];
                tmem_ld32(o, o_tm + c);
                asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
                tmem_use32(o);
                if (q < u.n) {
#pragma unroll
                    for (int e = 0; e < 32; e += 16) {
                        uint32_t y[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) y[i] = pack_bf16x2(o[e + 2 * i] * inv, o[e + 2 * i + 1] * inv);
                        st_global32(out + c + e, y, A.wide_out);
                    }
                }
            }
            tc_fence_before();
            if (__builtin_expect(C.poisoned[unit % 8] == unit + 1, 0) && q < u.n) {
                // what was taken out of the values that this row sees
                for (int t = sp.lo; t < sp.hi; ++t) {
                    if (!partial<kWindow>(A, u, a, t) && !(t >= other.lo && t < other.hi && partial<kWindow>(A, u, a ^ 1, t))) continue;
                    for (int k = t * kTile; k < min((t + 1) * kTile, q + 1); ++k) {
                        if (kWindow && k <= q - A.window) continue;
                        const uint16_t *v = A.v + (int64_t)(u.row0 + k) * A.v_stride + (u.h / A.G) * D + half * kEntries;
#pragma unroll 1
                        for (int d = 0; d < kEntries; ++d) {
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
    if (__builtin_expect(C.gave_up, 0)) {
        // No warp issues any more.  What is in flight lands before the CTA ends: the products, each slot's
        // latest copy, the queries.
        if (warp == kWarpMma) {
            if (elect_one()) mma_commit(&C.drained);
            __syncwarp();
            mbar_wait_bounded(&C.drained, 0, kDrainTimeoutNs);
        } else if (warp == kWarpLoad) {
            bool landed = true;
            for (int kv = 0; kv < 2; ++kv) {
                const int slots = kv ? A.slots - A.k_slots : A.k_slots, n = C.issued[kv];
                for (int k = max(n - slots, 0); landed && k < n; ++k)
                    landed = mbar_wait_bounded(&C.full[(kv ? A.k_slots : 0) + k % slots], (k / slots) & 1, kDrainTimeoutNs);
            }
            for (int a = 0; a < 2; ++a)
                if (landed && C.q_issued[a]) landed = mbar_wait_bounded(&C.q_full[a], (C.q_issued[a] - 1) & 1, kDrainTimeoutNs);
        }
        if (tid == 0) atomicOr(A.status, kStatusWaitTimeout);
        __syncthreads();
    }
    if (warp == kWarpMma) tmem_free(tmem, 512);
}

template <int D, bool kWindow>
cudaError_t launch(PromptArgs A, const CUtensorMap (&maps)[3], int ctas, cudaStream_t s) {
    const size_t slot = size_t(D) * 2 * kTile;
    A.slots = int(std::min<size_t>((kSmemBytes - sizeof(Ctrl) - 1024 - 2 * slot) / slot, kSlotsMax));
    A.k_slots = A.slots / 2;
    static_assert((kSmemBytes - sizeof(Ctrl) - 1024) / (D * 2 * kTile) >= 2 + 4, "two slots each of K and V");
    const size_t smem = 1024 + (2 + A.slots) * slot;
    const cudaError_t e = cudaFuncSetAttribute(prompt_attention_kernel<D, kWindow>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
    if (e != cudaSuccess) return e;
    return launch_overlapped(prompt_attention_kernel<D, kWindow>, ctas, kThreadsP, smem, s, A, maps[0], maps[1], maps[2]);
}

}  // namespace

cudaError_t launch_prompt_attention(const dspark_attn &a, int sms, uint64_t wait_ns, cudaStream_t s) {
    PromptArgs A{};
    A.B = a.B; A.rows = a.rows; A.q_max = a.q_max; A.Hq = a.Hq; A.Hkv = a.Hkv; A.G = a.Hq / a.Hkv;
    A.window = a.window;
    A.scale2 = float(double(a.scale) * 1.4426950408889634);
    int exponent;
    A.far_scale = std::frexp(A.scale2, &exponent) == 0.5f ? A.scale2 : std::ldexp(1.0f, exponent);
    A.v_stride = a.v_stride;
    A.v = static_cast<const uint16_t *>(a.v);
    A.row_off = a.row_off;
    A.out = static_cast<uint16_t *>(a.out);
    A.wide_out = reinterpret_cast<uintptr_t>(a.out) % 32 == 0;
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
    if (a.window > 0)
        return a.D == 128 ? launch<128, true>(A, maps, ctas, s) : launch<64, true>(A, maps, ctas, s);
    return a.D == 128 ? launch<128, false>(A, maps, ctas, s) : launch<64, false>(A, maps, ctas, s);
}

}  // namespace dspark
