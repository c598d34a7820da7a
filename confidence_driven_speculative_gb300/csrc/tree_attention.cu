// tree_attention.cu -- dspark_step_attention_tree: the rows of drafted trees
// over the paged cache.
//
// Mathematics.  As in step_attention.cuh; here the query vectors are the M side
// of the tensor core.  One request and one cached head give rows * G vectors
// (G query heads share the cached head); a block holds up to 128 of them, a
// unit one block or two.  S = Q K^T over tiles of 128 keys, weights
// P = 2^(scale log2(e) (S - m)) against a running reference m per vector that lies
// 2^16 above the first tile's maximum and moves only when a score passes it,
// l = sum P, O += P V; the output is O / l.
//
// Two streams of S, P and O fill TMEM.  The tensor cores work on one while
// the other's softmax runs; P overwrites its S and is the A operand of P V.
// A job is one block over one tile, and jobs go to the streams in turn.  Where a
// unit has two blocks, each stream keeps one, and they share the tiles; where it
// has one, the streams take every other tile of the same queries, and the
// two sums are joined at the end.  Either way both streams are busy.
//
// What a row sees of a tile is a word of 64 bits to each thread (two share a row):
// the cached keys by its window, its own request's entries by the bits of row_seen.
// Tiles that every row sees, all but the last one or two, need none.
//
// Bound: bytes of the cache; a tile's 64 KB take an SM's share of the memory
// 1.46 us, two jobs about 1.4.  The split of the list of tiles over the CTAs is
// step_attention.cuh's.  A unit that was cut leaves its parts in the workspace; a
// second kernel adds them, a warp for each column, spread over all SMs: with
// one request the parts are megabytes, and one SM reads a tenth of one per microsecond.
//
// Measured, 32 heads over 8 cached ones of 128: 32 requests of 16 to 4095 keys with
// trees of 17 to 48 rows over pages of 16 positions 72 us (cache, queries and outputs
// at a copy's 6.78 TB/s 44); one request of 4095 keys with 60 rows 18.5 (2.7): a
// chain of launch, cut, first tiles, a part's last product, its way through the
// workspace and the second kernel.  With keys on the M side, as for the few
// columns of a chain, the same calls took 142 and 34.
#include "step_attention.cuh"

namespace dspark {
namespace {

constexpr int kThreadsT = 640;
constexpr int kWarpTMma = 0, kWarpTK = 1, kWarpTV = 2, kWarpTReady = 3, kWarpTSoft = 4;  // softmax 4..19
constexpr int kSlotsT = 10;      // ring slots at most
constexpr int kParts = 4;        // parts on their way to the warps
constexpr int kPartReaders = 19; // warps that read them
constexpr int kBad = 8;          // ring of the tiles' bad-key words
// Places of the list: of a tile of one block, of one of two, and what a unit costs beside its tiles.
constexpr int kTileOne = 2, kTileTwo = 3, kUnitPlaces = 10;
// Up to so many tiles a CTA all units have one block: the two blocks of a request then go to different CTAs, which
// read the same keys but have half as many columns to write out and to add up.  Trees of 60 rows, 8 cached heads,
// one block and two: 1 request of 4095 keys (1.7 tiles a CTA) 18.5 us and 22.2, 8 of 1000 (3.8) 27.2 and 29.4,
// 4 of 4095 (6.9) 34.9 and 36.0, 1 of 16 000 (6.6) 31.4 and 29.5, 12 of 2000 (10.4) 49.5 and 44.0.  (Near the border
// the requests' number decides as well, by a few percent either way.)
constexpr int kFewTiles = 6;

// A unit that was cut, for the second kernel.
struct Cut {
    int row0, head0, ncols, members;  // members 0: none
};

struct TreeArgs : StepArgs {
    const int32_t *packed_pos;  // with a window
    const uint64_t *row_seen;
    int rb;       // rows of a block
    int v_slots;
    int wide_out;  // out is 32-byte aligned
    Cut *cuts;    // [CTAs], by the CTA that the unit begins in
};

// A tree's row: what it sees, and where its window ends (its position).
struct TreeRow {
    uint64_t seen;
    int pos;
    __device__ __forceinline__ TreeRow(const TreeArgs &A, const Req &q, int j, bool there) : seen(0), pos(q.pos0) {
        if (!there) return;
        // (asked for here, and not where it is used first)
        asm volatile("ld.global.b64 %0, [%1];" : "=l"(seen) : "l"(A.row_seen + q.row0 + j));
        if (A.window > 0) pos = max(A.packed_pos[q.row0 + j], q.pos0);
    }
    // Which of the 32 keys from k0 on it sees.
    __device__ __forceinline__ uint32_t word(const TreeArgs &A, const Req &q, int k0) const {
        auto below = [&](int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; };
        uint32_t cached = below(q.pos0 - k0);
        if (A.window > 0) cached &= ~below(pos - A.window + 1 - k0) | below(A.sinks - k0);
        const int at = k0 - q.pos0;  // the own entry that k0 is
        const uint32_t own = at >= 64 || at <= -32 ? 0u : at >= 0 ? uint32_t(seen >> at) : uint32_t(seen) << -at;
        return (cached | own) & below(q.kend - k0);
    }
};

// The same request in units of up to `rows` rows.
__device__ __forceinline__ Req in_units_of(Req r, int rows) {
    if (r.per > rows) {
        // for up to 64: the quotient lies 1 / (2 b) at least from a whole number
        auto ceil_div = [](int a, int b) { return int(__fdividef(float(a + b) - 0.5f, float(b))); };
        r.blocks = ceil_div(r.n, rows);
        r.per = ceil_div(r.n, r.blocks);
        r.blocks = ceil_div(r.n, r.per);
    }
    return r;
}

// What a CTA does of one unit.
struct Part {
    int n;                   // tiles; 0: no more parts
    int blocks, jobs, job0;  // blocks of queries; n * blocks; the CTA's jobs before
    int t_beg, q_use;        // first tile; the CTA's query blocks before
    int slot;                // of the workspace, where the unit was cut; else -1
    int b, h, row0, nrows;   // request, cached head, first packed row, rows
    int whole_lo, whole_hi;  // tiles that every row sees in full, beside the sinks'
    Req q;
};

struct TCtrl {
    uint64_t full[kSlotsT], empty[kSlotsT];
    uint64_t q_full[2], q_empty[2], s_full[2], p_full[2], o_full[2];
    uint64_t part_full[kParts], part_empty[kParts], drained;
    Part part[kParts];
    alignas(16) uint32_t bad[kBad][4];
    float swap[2][2][kTile];        // between threads of a row: by stream and half
    int poisoned[8];                // by part % 8: the last part + 1 that lost values
    int spread[8];                  // and of those in a tile that all rows see, but for a page that is none
    uint32_t tmem;
    int issued[2], q_issued;
    int gave_up;
};

template <int a>
using Stream = std::integral_constant<int, a>;

// Reads the next part off the ring; `then` copies what the warp wants of it.
struct PartReader {
    Ring r;
    template <typename F>
    __device__ __forceinline__ bool next(TCtrl &C, const TreeArgs &A, volatile int *gave_up, int lane, F then) {
        bool ok = wait_or_give_up(&C.part_full[r.slot], r.phase, A.wait_ns, gave_up);
        ok = __all_sync(0xffffffffu, ok);
        if (ok) {
            then(C.part[r.slot]);
            __syncwarp();
            if (lane == 0) mbar_arrive(&C.part_empty[r.slot]);
            r.next(kParts);
        }
        return ok;
    }
};

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, w;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "mul.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// The copies of one tile of K or V: a lane per box (or four keys: gather).
template <int D, bool kBox>
struct Tiles {
    int span, boxes;
    uint64_t policy;  // the cache's lines make way for the parts of cut units, which are read again
    struct Ids { int page[4]; };
    __device__ __forceinline__ Tiles(const TreeArgs &A) : span(kBox ? A.box : 4), boxes(kTile / span), policy(evict_first()) {}

    __device__ __forceinline__ void look_up(const TreeArgs &A, int b, const Req &q, int t, int lane, Ids &ids) const {
        const int key0 = tile_at<kSinks>(q, t) * kTile + lane * span;
        const int32_t *table = A.block_table + (int64_t)b * A.max_pages;
        const bool wanted = lane < boxes && wants<kSinks>(A, q, t, key0, span);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            ids.page[i] = -1;
            if ((i == 0 || !kBox) && wanted) {
                const int pi = page_of(A, key0 + i);
                if (pi < A.max_pages) ids.page[i] = table[pi];
            }
        }
    }
    // Issues them to `dst`; the keys that have no memory in `bad` (where it is not NULL).
    __device__ __forceinline__ void copy(const TreeArgs &A, const CUtensorMap *map, int h, const Req &q, int t, int lane,
                                         const Ids &ids, uint32_t dst, uint64_t *full, uint32_t *bad) const {
        constexpr int kHalves = D / 64;
        constexpr uint32_t kHalfBytes = kTile * 128;
        const int tile0 = tile_at<kSinks>(q, t) * kTile, key0 = tile0 + lane * span;
        const bool here = lane < boxes && wants<kSinks>(A, q, t, key0, span);
        uint32_t bad_bits = 0;
        int row[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bool good = ids.page[j] >= 0 && ids.page[j] < A.num_pages;
            if (!good) bad_bits |= 1u << j;
            const int page = good ? ids.page[j] : 0;  // masked; any memory will do
            row[j] = kBox ? page : page * A.page_rows + h * A.head_rows + key0 + j - page_of(A, key0 + j) * A.page_size;
        }
        if (bad) {
            const bool lane_bad = here && (kBox ? (bad_bits & 1) : bad_bits != 0);
            uint32_t words[4] = {0, 0, 0, 0};
            if (__any_sync(0xffffffffu, lane_bad)) {
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    uint32_t m = 0;
                    if (lane_bad) {
                        if (kBox) {
                            const int lo = max(lane * span - 32 * w, 0), hi = min(lane * span + span - 32 * w, 32);
                            if (lo < hi) m = (hi - lo == 32 ? 0xffffffffu : ((1u << (hi - lo)) - 1u)) << lo;
                        } else if (lane / 8 == w) {
                            m = bad_bits << (4 * (lane % 8));
                        }
                    }
                    words[w] = __reduce_or_sync(0xffffffffu, m);
                }
            }
            if (lane == 0) *reinterpret_cast<uint4 *>(bad) = make_uint4(words[0], words[1], words[2], words[3]);
        }
        // the boxes to copy: a run of lanes
        const uint32_t run = __ballot_sync(0xffffffffu, here);
        const int box_lo = __ffs(run) - 1, box_n = __popc(run);
        __syncwarp();
        const bool leader = elect_one();
        if (leader) mbar_arrive_expect_tx(full, box_n * uint32_t(span) * D * 2);
        dst += box_lo * span * 128;
        if (kBox) {
            const int first_key = tile0 + box_lo * span;
            int in_page = first_key - page_of(A, first_key) * A.page_size;
            for (int j = box_lo; j < box_lo + box_n; ++j) {
                const int page = __shfl_sync(0xffffffffu, row[0], j);
                if (leader) {
                    tma_load_4d(dst, map, full, 0, in_page, h, page, policy);
                    if (kHalves == 2) tma_load_4d(dst + kHalfBytes, map, full, 64, in_page, h, page, policy);
                }
                dst += span * 128;
                in_page += span;
                if (in_page == A.page_size) in_page = 0;
            }
        } else {
            const int x0 = h * A.head_x;
            for (int j = box_lo; j < box_lo + box_n; ++j) {
                int k[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) k[i] = __shfl_sync(0xffffffffu, row[i], j);
                if (leader) {
                    tma_gather4(dst, map, full, x0, k[0], k[1], k[2], k[3], policy);
                    if (kHalves == 2) tma_gather4(dst + kHalfBytes, map, full, x0 + 64, k[0], k[1], k[2], k[3], policy);
                }
                dst += span * 128;
            }
        }
        __syncwarp();
    }
};

template <int D, bool kBox>
__global__ void __launch_bounds__(kThreadsT, 1)
tree_attention_kernel(const __grid_constant__ TreeArgs A, const __grid_constant__ CUtensorMap q_map,
                      const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map) {
    constexpr int kHalves = D / 64;
    constexpr uint32_t kHalfBytes = kTile * 128;
    constexpr uint32_t kSlotBytes = kHalves * kHalfBytes;
    constexpr uint32_t kColO = 2 * kTile;  // S_0, S_1, O_0, O_1
    extern __shared__ __align__(1024) uint8_t dyn[];
    // Queries (two blocks), ring, control.
    const uint32_t q_smem = smem_addr(dyn);
    const uint32_t ring = q_smem + 2 * kSlotBytes, v_ring = ring + A.k_slots * kSlotBytes;
    const uint32_t ctrl = ring + A.slots * kSlotBytes;
    TCtrl &C = *reinterpret_cast<TCtrl *>(dyn + (ctrl - smem_addr(dyn)));
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
    volatile int *gave_up = &C.gave_up;

    // ---- set-up -------------------------------------------------------------
    if (tid == 0) {
        for (int s = 0; s < A.slots; ++s) {
            mbar_init(&C.full[s], 1);
            mbar_init(&C.empty[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&C.q_full[a], 1);
            mbar_init(&C.q_empty[a], 1);
            mbar_init(&C.s_full[a], 2);
            mbar_init(&C.p_full[a], 9);
            mbar_init(&C.o_full[a], 2);
        }
        for (int s = 0; s < kParts; ++s) {
            mbar_init(&C.part_full[s], 1);
            mbar_init(&C.part_empty[s], kPartReaders);
        }
        mbar_init(&C.drained, 1);
        for (int i = 0; i < 8; ++i) C.poisoned[i] = C.spread[i] = 0;
        C.gave_up = C.issued[0] = C.issued[1] = C.q_issued = 0;
        fence_barrier_init();
    }
    if (warp == kWarpTMma) tmem_alloc(&C.tmem, kTmemCols);
    if (warp == kWarpTK && lane == 0) {
        prefetch_map(&q_map);
        prefetch_map(&k_map);
        prefetch_map(&v_map);
    }
    // The vectors past a block's last row are zeros, which no copy touches.
    for (int x = A.rb * A.G * 8 + tid; x < kTile * 8; x += kThreadsT)
        for (int s = 0; s < 2 * kHalves; ++s) st_shared16(q_smem + s * kHalfBytes + x * 16, 0, 0, 0, 0);
    fence_async_shared();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // Nothing before this line reads or writes memory that another kernel may
    // touch: the launch may overlap the end of the kernel before it.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const uint32_t tmem = C.tmem;

    if (warp == kWarpTK) {
        // ---- the CTA's parts, their queries and keys ---------------------------
        constexpr int U = kUnitPlaces;
        const int me = blockIdx.x, per = (A.B + 31) / 32, b_lo = min(lane * per, A.B), b_hi = min(b_lo + per, A.B);
        auto places_of = [&](const Req &r) { return r.per > A.rb ? kTileTwo : kTileOne; };  // of a tile
        auto cost_of = [&](const Req &r) { return r.blocks * A.Hkv * (r.nt * places_of(r) + U); };
        // Units of two blocks or of one: see kFewTiles.
        int two = 0, tiles_two = 0;
        uint32_t one = 0;  // (may pass 32 bits where it is not used)
        // (unrolled, the loop costs its fetch: 0.4 us for few requests, and a lane's requests share a sector)
#pragma unroll 1
        for (int b = b_lo; b < b_hi; ++b) {
            const Req r = load_req<kSinks>(A, b);
            two += cost_of(r);
            one += uint32_t(cost_of(in_units_of(r, A.rb)));
            tiles_two += r.blocks * A.Hkv * r.nt;
        }
        const bool few = __reduce_add_sync(0xffffffffu, tiles_two) <= kFewTiles * int(gridDim.x);
        const int rows_cap = few ? A.rb : A.rows_cap, mine = few ? int(one) : two;
        int sum = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += x;
        }
        const int total = __shfl_sync(0xffffffffu, sum, 31);
        // (no CTA's share is shorter than a tile, so that a cut unit has a tile in each CTA from its first to its last)
        const Cuts cuts(total, min(int(gridDim.x), max(total / kTileTwo, 1)));
        const int start = cuts.start(me), end = cuts.start(me + 1);
        const uint32_t who = __ballot_sync(0xffffffffu, start >= sum - mine && start < sum);
        int b = A.B, place = sum - mine;  // the request that holds `start`, and where it begins
        if (who) {
            const int src = __ffs(who) - 1;
            if (lane == src)
                for (b = b_lo; b < b_hi; ++b) {
                    const int c = cost_of(in_units_of(load_req<kSinks>(A, b), rows_cap));
                    if (start < place + c) break;
                    place += c;
                }
            b = __shfl_sync(0xffffffffu, b, src);
            place = __shfl_sync(0xffffffffu, place, src);
        }
        if (lane == 0) A.cuts[me].members = 0;
        const Tiles<D, kBox> tiles(A);
        Ring rs, rk;
        int published = 0, issued = 0, q_use = 0, jobs = 0;
        bool ok = true;
        for (; b < A.B && place < end && ok; ++b) {
            const Req q = in_units_of(load_req<kSinks>(A, b), rows_cap);
            const int w = places_of(q), each = q.nt * w + U, units = q.blocks * A.Hkv;
            int i = max(start - place, 0) / each;
            for (; i < units && place + i * each < end && ok; ++i) {
                const int tile0 = place + i * each + U;  // the place of the unit's first tile
                Part p;
                p.t_beg = (max(start - tile0, 0) + w - 1) / w;
                p.n = min((max(end - tile0, 0) + w - 1) / w, q.nt) - p.t_beg;
                if (p.n <= 0) continue;  // only its cost lies here
                p.b = b;
                p.h = i / q.blocks;
                const int j0 = (i - p.h * q.blocks) * q.per;
                p.row0 = q.row0 + j0;
                p.nrows = min(q.per, q.n - j0);
                p.q = q;
                p.blocks = p.nrows > A.rb ? 2 : 1;
                p.jobs = p.n * p.blocks;
                p.job0 = jobs;
                p.q_use = q_use;
                p.slot = -1;
                if (p.n < q.nt) {
                    // A unit that begins here and goes on is the CTA's last, one that goes on here its first.
                    p.slot = 2 * me + (p.t_beg == 0);
                    if (p.t_beg == 0 && lane == 0)
                        A.cuts[me] = Cut{p.row0, p.h * A.G, p.nrows * A.G, cuts.of(tile0 + (q.nt - 1) * w) - me + 1};
                }
                int last_pos = q.pos0;
                if (A.window > 0) {
                    for (int j = lane; j < p.nrows; j += 32) last_pos = max(last_pos, A.packed_pos[p.row0 + j]);
                    last_pos = __reduce_max_sync(0xffffffffu, last_pos);
                }
                p.whole_hi = min(q.kend, q.pos0) / kTile;
                p.whole_lo = ((A.window > 0 ? max(last_pos - A.window + 1, q.kbeg) : q.kbeg) + kTile - 1) / kTile;
                jobs += p.jobs;
                if (published >= kParts) ok = wait_or_give_up(&C.part_empty[rs.slot], rs.phase ^ 1, A.wait_ns, gave_up);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                if (lane == 0) {
                    C.part[rs.slot] = p;
                    mbar_arrive(&C.part_full[rs.slot]);
                }
                __syncwarp();
                rs.next(kParts);
                ++published;
                typename Tiles<D, kBox>::Ids ids, ahead;
                tiles.look_up(A, b, q, p.t_beg, lane, ids);
                for (int t = 0; t < p.n && ok; ++t) {
                    if (t + 1 < p.n) tiles.look_up(A, b, q, p.t_beg + t + 1, lane, ahead);
                    if (issued >= A.k_slots) ok = wait_or_give_up(&C.empty[rk.slot], rk.phase ^ 1, A.wait_ns, gave_up);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    tiles.copy(A, &k_map, p.h, q, p.t_beg + t, lane, ids, ring + rk.slot * kSlotBytes, &C.full[rk.slot],
                               C.bad[issued % kBad]);
                    rk.next(A.k_slots);
                    ++issued;
                    ids = ahead;
                    // the queries behind the first keys: they wait until the part before has no use for theirs
                    for (int x = 0; t == 0 && x < p.blocks && ok; ++x, ++q_use) {
                        const int s = q_use & 1;
                        if (q_use >= 2) ok = wait_or_give_up(&C.q_empty[s], ((q_use >> 1) - 1) & 1, A.wait_ns, gave_up);
                        ok = __all_sync(0xffffffffu, ok);
                        if (!ok) break;
                        if (elect_one()) {
                            mbar_arrive_expect_tx(&C.q_full[s], uint32_t(A.rb * A.G) * D * 2);
                            for (int hf = 0; hf < kHalves; ++hf)
                                tma_load_3d(q_smem + s * kSlotBytes + hf * kHalfBytes, &q_map, &C.q_full[s], hf * 64, p.h * A.G,
                                            p.row0 + x * A.rb);
                        }
                        __syncwarp();
                    }
                }
            }
            place += units * each;
        }
        // no more
        if (ok && published >= kParts) ok = wait_or_give_up(&C.part_empty[rs.slot], rs.phase ^ 1, A.wait_ns, gave_up);
        ok = __all_sync(0xffffffffu, ok);
        if (lane == 0) {
            if (ok) {
                C.part[rs.slot].n = 0;
                mbar_arrive(&C.part_full[rs.slot]);
            }
            C.issued[0] = issued;  // for the CTA's end, should a wait have given up
            C.q_issued = q_use;
        }
    } else if (warp == kWarpTV) {
        // ---- values ----------------------------------------------------------------
        const Tiles<D, kBox> tiles(A);
        PartReader parts;
        Ring rv;
        int issued = 0;
        for (bool ok = true; ok;) {
            int n = 0, b = 0, h = 0, t0 = 0;
            Req q{};
            ok = parts.next(C, A, gave_up, lane, [&](const Part &p) {
                n = p.n;
                b = p.b;
                h = p.h;
                t0 = p.t_beg;
                q = p.q;
            });
            if (!ok || n == 0) break;
            typename Tiles<D, kBox>::Ids ids, ahead;
            tiles.look_up(A, b, q, t0, lane, ids);
            for (int t = 0; t < n && ok; ++t) {
                if (t + 1 < n) tiles.look_up(A, b, q, t0 + t + 1, lane, ahead);
                const int slot = A.k_slots + rv.slot;
                if (issued >= A.v_slots) ok = wait_or_give_up(&C.empty[slot], rv.phase ^ 1, A.wait_ns, gave_up);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tiles.copy(A, &v_map, h, q, t0 + t, lane, ids, ring + slot * kSlotBytes, &C.full[slot], nullptr);
                rv.next(A.v_slots);
                ++issued;
                ids = ahead;
            }
        }
        if (lane == 0) C.issued[1] = issued;
    } else if (warp == kWarpTMma) {
        // ---- MMA issuer: O of a job, then S of the stream's next one -----------------
        // A part's first two S come when all products of the part before are on their way: whoever
        // computes its outputs waits for those, and not for the next part's queries and keys.
        const uint64_t qd0 = smem_desc(q_smem, 16, 1024), kd0 = smem_desc(ring, 16, 1024);
        const uint64_t vd0 = smem_desc(v_ring, kHalfBytes, 1024);
        constexpr uint32_t id_s = mma_idesc(128, kTile, false, false), id_o = mma_idesc(128, D, false, true);
        PartReader parts;
        Ring rk, rv;
        uint32_t p_phase[2] = {0, 0};
        bool ok = true;
        int n = 0, blocks = 1, job0 = 0, q_use = 0;  // the part: its jobs, ..., its first query block
        auto wait = [&](uint64_t *bar, uint32_t phase) {
            ok = ok && wait_or_give_up(bar, phase, A.wait_ns, gave_up);
            ok = __all_sync(0xffffffffu, ok);
        };
        // S of job k, on stream a.
        auto issue_s = [&](auto stream, int k) {
            constexpr int a = decltype(stream)::value;
            const int x = blocks == 2 ? k & 1 : 0, u = q_use + x;  // the query block
            const bool tile_done = blocks == 1 || x == 1;
            tc_fence_after();
            if (elect_one()) {
                mbar_arrive(&C.s_full[a]);  // passes the producer's words on
                const uint64_t qd = qd0 + uint32_t(u & 1) * (kSlotBytes >> 4);
                const uint64_t kd = kd0 + uint32_t(rk.slot) * (kSlotBytes >> 4);
#pragma unroll
                for (int d = 0; d < D / 16; ++d) {
                    const uint32_t at = ((d / 4) * kHalfBytes + (d % 4) * 32) >> 4;
                    mma_ss(tmem + a * kTile, qd + at, kd + at, id_s, d > 0);
                }
                mma_commit(&C.s_full[a]);
                if (tile_done) mma_commit(&C.empty[rk.slot]);
                if (k + blocks >= n) mma_commit(&C.q_empty[u & 1]);
            }
            __syncwarp();
            if (tile_done) rk.next(A.k_slots);
        };
        // One of a part's first two jobs: its queries and keys are waited for here.
        auto first_s = [&](auto stream, int k) {
            const int u = q_use + (blocks == 2 ? k & 1 : 0);
            if (k < blocks) wait(&C.q_full[u & 1], (u >> 1) & 1);
            wait(&C.full[rk.slot], rk.phase);
            if (ok) issue_s(stream, k);
        };
        // O of job k on stream a, and S of job k + 2.
        auto step = [&](auto stream, int k) {
            constexpr int a = decltype(stream)::value;
            wait(&C.p_full[a], p_phase[a]);
            if (!ok) return;
            p_phase[a] ^= 1;
            const bool tile_done = blocks == 1 || (k & 1), more = k + 2 < n;
            tc_fence_after();
            if (elect_one()) {
                const uint64_t vd = vd0 + uint32_t(rv.slot) * (kSlotBytes >> 4);
#pragma unroll
                for (int i = 0; i < kTile / 16; ++i)
                    mma_ts(tmem + kColO + a * D, tmem + a * kTile + i * 8, vd + i * (2048 >> 4), id_o, !(k < 2 && i == 0));
                if (tile_done) mma_commit(&C.empty[A.k_slots + rv.slot]);
                if (!more) {
                    mbar_arrive(&C.o_full[a]);  // passes on what was lost of V
                    mma_commit(&C.o_full[a]);
                }
            }
            __syncwarp();
            if (tile_done) rv.next(A.v_slots);
            if (more) issue_s(stream, k + 2);
        };
        auto whole_part = [&](auto even, auto odd) {  // the streams of its even and odd jobs
            first_s(even, 0);
            if (ok && n > 1) first_s(odd, 1);
            for (int k = 0; ok && k < n; k += 2) {
                step(even, k);
                if (ok && k + 1 < n) step(odd, k + 1);
            }
        };
        while (ok) {
            ok = parts.next(C, A, gave_up, lane, [&](const Part &p) {
                n = __shfl_sync(0xffffffffu, p.jobs, 0);
                blocks = __shfl_sync(0xffffffffu, p.blocks, 0);
                job0 = __shfl_sync(0xffffffffu, p.job0, 0);
                q_use = __shfl_sync(0xffffffffu, p.q_use, 0);
                if (__shfl_sync(0xffffffffu, p.n, 0) == 0) n = 0;
            });
            if (!ok || n == 0) break;
            if (job0 & 1) whole_part(Stream<1>{}, Stream<0>{});
            else whole_part(Stream<0>{}, Stream<1>{});
        }
    } else if (warp == kWarpTReady) {
        // ---- the last of P's arrivals: V of its tile and K of the stream's next job in the part
        // are there, so that the MMA issuer has one barrier to test and not three ----------
        PartReader parts;
        Ring rk, rv;
        uint32_t uses[2] = {0, 0};
        bool ok = true;
        int keys = 0, tiles_before = 0;  // tiles whose K was waited for (each in turn: a parity tells two uses apart)
        while (ok) {
            int n = 0, blocks = 1, job0 = 0;
            ok = parts.next(C, A, gave_up, lane, [&](const Part &p) {
                n = p.n ? p.jobs : 0;
                blocks = p.blocks;
                job0 = p.job0;
            });
            if (!ok || n == 0) break;
            for (int k = 0; ok && k < n; ++k) {
                const int a = (job0 + k) & 1, want = min(k + 2, n - 1);
                for (const int last = tiles_before + (blocks == 2 ? want >> 1 : want); ok && keys <= last; ++keys) {
                    ok = keys == 0 ? poll_or_give_up(&C.full[rk.slot], rk.phase, A.wait_ns, gave_up)
                                   : wait_or_give_up(&C.full[rk.slot], rk.phase, A.wait_ns, gave_up);
                    ok = __all_sync(0xffffffffu, ok);
                    rk.next(A.k_slots);
                }
                ok = ok && wait_or_give_up(&C.full[A.k_slots + rv.slot], rv.phase, A.wait_ns, gave_up);
                if (blocks == 1 || (k & 1)) rv.next(A.v_slots);
                // not before the stream's job before is through
                if ((a ? uses[1] : uses[0]) > 0)
                    ok = ok && wait_or_give_up(&C.p_full[a], ((a ? uses[1] : uses[0]) - 1) & 1, A.wait_ns, gave_up);
                uses[0] += a == 0;
                uses[1] += a == 1;
                ok = __all_sync(0xffffffffu, ok);
                if (ok && lane == 0) mbar_arrive(&C.p_full[a]);
                __syncwarp();
            }
            tiles_before += blocks == 2 ? n / 2 : n;
        }
    } else {
        // ---- softmax and output --------------------------------------------------
        // Two threads share a vector of stream a: thread `half` takes 64 keys of
        // each tile.  The halves' warps meet twice a job: both have read S before
        // either writes P over it, and both know of a reference that moves.
        const int sw = warp - kWarpTSoft, a = sw >> 3, half = (sw >> 2) & 1, row = (warp & 3) * 32 + lane;
        constexpr int kKeys = kTile / 2;
        const uint32_t lane_tm = tmem + (uint32_t((warp & 3) * 32) << 16);
        const uint32_t s_tm = lane_tm + a * kTile, o_tm = lane_tm + kColO;
        const uint32_t pair_bar = 1 + a * 4 + (warp & 3), quad_bar = 9 + (warp & 3);
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
        auto quad_sync = [&] { asm volatile("barrier.cta.sync %0, 128;" ::"r"(quad_bar) : "memory"); };
        PartReader parts;
        int s_uses = 0, o_uses0 = 0, o_uses1 = 0;
        int tiles_before = 0;  // of the CTA's parts so far
        for (int part = 0;; ++part) {
            int n = 0, blocks = 1, jobs = 0, job0 = 0, t_beg = 0, slot = -1, h = 0, row0 = 0, nrows = 0, whole_lo = 0, whole_hi = 0, b = 0;
            Req q{};
            const bool got = parts.next(C, A, gave_up, lane, [&](const Part &p) {
                n = p.n;
                blocks = p.blocks;
                jobs = p.jobs;
                job0 = p.job0;
                t_beg = p.t_beg;
                slot = p.slot;
                b = p.b;
                h = p.h;
                row0 = p.row0;
                nrows = p.nrows;
                whole_lo = p.whole_lo;
                whole_hi = p.whole_hi;
                q = p.q;
            });
            // all warps leave together: the exchanges below need them
            uint32_t stop;
            asm volatile(
                "{\n\t.reg .pred p, q;\n\t"
                "setp.ne.u32 q, %2, 0;\n\t"
                "barrier.cta.red.or.pred p, %1, 128, q;\n\t"
                "selp.u32 %0, 1, 0, p;\n\t}"
                : "=r"(stop) : "r"(quad_bar), "r"(uint32_t(!got || n == 0)) : "memory");
            if (stop) break;
            const int k0 = (a ^ job0) & 1;              // the stream's first job of the part
            const int x = blocks == 2 ? k0 : 0;         // its block
            const int j = x * A.rb + row / A.G;         // the thread's row of the unit
            const bool valid = row < A.rb * A.G && j < nrows;
            TreeRow mine(A, q, row0 - q.row0 + j, valid);
            float ref = kRefMin;
            float2 l2 = make_float2(0.f, 0.f);
            // Once a wait has given up, the others return at once and the
            // loops run to their ends on whatever there is; the status tells.
            for (int k = k0; k < jobs; k += 2) {
                const int t = blocks == 2 ? k >> 1 : k, tile = tile_at<kSinks>(q, t_beg + t);
                wait_or_give_up(&C.s_full[a], s_uses & 1, A.wait_ns, gave_up);
                __syncwarp();
                ++s_uses;
                tc_fence_after();
                const uint4 bw = *reinterpret_cast<const uint4 *>(C.bad[(tiles_before + t) % kBad]);
                const bool edge = tile >= whole_hi || !(tile >= whole_lo || (tile + 1) * kTile <= A.sinks);
                const bool cut = edge || (bw.x | bw.y | bw.z | bw.w) != 0;
                if (__builtin_expect(cut, 0) && (blocks == 1 || k0 == 0)) {
                    // Masked keys must not reach O through 0 * infinity: the tile's values lose their NaN
                    // and infinities; the rows that see them get them back at the part's end.  Where both
                    // streams use the tile, the one with its first job does it for both: its P comes
                    // before either's products.  (S of this job says that the products of V's use of this
                    // slot before are through, so that the parity tells whether V is there.)
                    const int use = tiles_before + t, vs = use % A.v_slots;
                    wait_or_give_up(&C.full[A.k_slots + vs], (use / A.v_slots) & 1, A.wait_ns, gave_up);
                    __syncwarp();
                    const uint32_t at0 = v_ring + vs * kSlotBytes + (half * kTile + row) * 16;
                    bool odd = false;
#pragma unroll
                    for (uint32_t c = 0; c < kSlotBytes; c += 2 * kTile * 16) odd |= nonfinite_any(ld_shared16(at0 + c));
                    if (__builtin_expect(odd, 0)) {
#pragma unroll 1
                        for (uint32_t c = 0; c < kSlotBytes; c += 2 * kTile * 16) {
                            const uint4 v = ld_shared16(at0 + c);
                            if (!nonfinite_any(v)) continue;
                            st_shared16(at0 + c, v.x & ~nonfinite_mask(v.x), v.y & ~nonfinite_mask(v.y),
                                        v.z & ~nonfinite_mask(v.z), v.w & ~nonfinite_mask(v.w));
                            // what no copy has brought, or lies outside the sequence, is not missed
                            const int key = tile * kTile + int(((half * kTile + row) * 16 + c) % kHalfBytes / 128);
                            if (key < q.kend && (key >= q.kbeg || key < A.sinks)) {
                                C.poisoned[part % 8] = part + 1;
                                if (!edge) C.spread[part % 8] = part + 1;
                            }
                        }
                        fence_async_shared();
                    }
                }
                float s[kKeys];
#pragma unroll
                for (int c = 0; c < kKeys; c += 32) tmem_ld32(s + c, s_tm + half * kKeys + c);
                asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
                for (int c = 0; c < kKeys; c += 32) tmem_use32(s + c);
                if (__builtin_expect(cut, 0)) {
#pragma unroll
                    for (int c = 0; c < kKeys; c += 32) {
                        const uint32_t bad = half ? (c ? bw.w : bw.z) : (c ? bw.y : bw.x);
                        const uint32_t seen = valid ? mine.word(A, q, tile * kTile + half * kKeys + c) & ~bad : 0u;
                        if (__all_sync(0xffffffffu, seen == 0xffffffffu || !valid)) continue;
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
                const bool first = k < 2;
                if (__builtin_expect(pair_any(first || m > ref), 0)) {
                    C.swap[a][half][row] = m;
                    pair_sync();
                    const float top = fmaxf(m, C.swap[a][half ^ 1][row]);
                    const float now = fmaxf(top + A.headroom, kRefMin);
                    if (first) {
                        ref = valid ? now : INFINITY;  // vectors that are none weigh nothing
                    } else {
                        const bool moves = top > ref;
                        const float f = moves ? exp2_approx((ref - now) * A.scale2) : 1.f;
                        if (moves) ref = now;
                        l2.x *= f;
                        l2.y *= f;
                        // the stream's O is still: its last product came before this S
                        const uint32_t at = o_tm + a * D + half * (D / 2);
#pragma unroll 1
                        for (int c = 0; c < D / 2; c += 16) {
                            float o[16];
                            tmem_ld16(o, at + c);
                            tmem_wait_ld(o);
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] *= f;
                            tmem_st16(at + c, o);
                        }
                        tmem_wait_st();
                        tc_fence_before();
                    }
                    pair_sync();  // swap is read, and all of O is rescaled before either half's P is used
                }
                const float2 sc = make_float2(A.scale2, A.scale2), nr = make_float2(-ref, -ref);
                float2 sums[2] = {l2, make_float2(0.f, 0.f)};
#pragma unroll
                for (int c = 0; c < kKeys; c += 32) {
                    uint32_t p[16];
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        // the difference first: it is exact for scores near the reference, however far from 0
                        const float2 y = mul2(add2(make_float2(s[c + e], s[c + e + 1]), nr), sc);
                        p[e / 2] = pack_bf16x2(exp2_approx(y.x), exp2_approx(y.y));
                        add_bf16x2(sums[(e / 2) & 1], p[e / 2]);
                    }
                    tmem_st16u(s_tm + (half * kKeys + c) / 2, p);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&C.p_full[a]);
                l2 = add2(sums[0], sums[1]);
            }
            tiles_before += n;
            // ---- the part's end ----------------------------------------------------
            // blocks = 2: the stream's own O, a thread half of its entries.  blocks = 1: both streams' O of
            // the same vector, joined, a thread a quarter.
            float l = l2.x + l2.y, f0 = 1.f, f1 = 0.f;  // of the stream's O, or of streams 0 and 1
            quad_sync();
            C.swap[a][half][row] = l;
            quad_sync();
            const bool one = blocks == 2 || jobs == 1;  // one stream's O
            const int st0 = blocks == 2 ? a : jobs == 1 ? job0 & 1 : 0;
            const int entries = blocks == 2 ? D / 2 : D / 4, c0 = (blocks == 2 ? half : 2 * a + half) * entries;
            if (blocks == 2) {
                l += C.swap[a][half ^ 1][row];
            } else {
                const float l0 = C.swap[0][0][row] + C.swap[0][1][row], l1 = C.swap[1][0][row] + C.swap[1][1][row];
                quad_sync();
                C.swap[a][half][row] = ref;
                quad_sync();
                const float ref0 = C.swap[0][0][row], ref1 = C.swap[1][0][row];
                // a stream without a job has the lowest reference and l = 0
                ref = fmaxf(ref0, ref1);
                f0 = exp2_approx((ref0 - ref) * A.scale2);
                f1 = exp2_approx((ref1 - ref) * A.scale2);
                l = f0 * l0 + f1 * l1;
                if (one) f0 = 1.f;
            }
            if (!one || st0 == 0) {
                wait_or_give_up(&C.o_full[0], o_uses0 & 1, A.wait_ns, gave_up);
                __syncwarp();
            }
            if (!one || st0 == 1) {
                wait_or_give_up(&C.o_full[1], o_uses1 & 1, A.wait_ns, gave_up);
                __syncwarp();
            }
            o_uses0 += jobs > 1 || !(job0 & 1);
            o_uses1 += jobs > 1 || (job0 & 1);
            tc_fence_after();
            const int col = x * A.rb * A.G + row;  // of the unit's columns
            const float inv = slot >= 0 ? 1.f : l == 0.f ? 0.f : 1.f / l;
            uint16_t *const out = A.out + ((int64_t)(row0 + j) * A.Hq + h * A.G + row % A.G) * D + c0;
            // parts lie by entry and then by column: a warp's stores are whole lines
            float *const part_o = A.part + ((int64_t)max(slot, 0) * D + c0) * A.ncap + col;
            const float g0 = f0 * inv, g1 = f1 * inv;
#pragma unroll 1
            for (int c = 0; c < entries; c += 16) {
                float o[16];
                tmem_ld16(o, o_tm + st0 * D + c0 + c);
                tmem_wait_ld(o);
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] *= g0;
                if (!one) {
                    float o1[16];
                    tmem_ld16(o1, o_tm + D + c0 + c);
                    tmem_wait_ld(o1);
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[e] = fmaf(o1[e], g1, o[e]);
                }
                if (valid) {
                    if (slot >= 0) {
#pragma unroll
                        for (int e = 0; e < 16; ++e) part_o[(int64_t)(c + e) * A.ncap] = o[e];
                    } else {
                        uint32_t y[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) y[e] = pack_bf16x2(o[2 * e], o[2 * e + 1]);
                        st_global32(out + c, y, A.wide_out);
                    }
                }
            }
            if (slot >= 0 && valid && half == 0 && (blocks == 2 || a == 0)) {
                A.stat[(int64_t)slot * 2 * A.ncap + col] = ref;
                A.stat[((int64_t)slot * 2 + 1) * A.ncap + col] = l;
            }
            tc_fence_before();
            if (__builtin_expect(C.poisoned[part % 8] == part + 1, 0) && valid) {
                // what was taken out of the values that this row sees
#pragma unroll 1
                for (int t = t_beg; t < t_beg + n; ++t) {
                    const int tile = tile_at<kSinks>(q, t);
                    const bool edge = tile >= whole_hi || !(tile >= whole_lo || (tile + 1) * kTile <= A.sinks);
                    if (!edge && C.spread[part % 8] != part + 1) continue;
#pragma unroll 1
                    for (int k = tile * kTile; k < (tile + 1) * kTile && k < q.kend; ++k) {
                        if (!(mine.word(A, q, k) & 1u)) continue;
                        const int page = A.block_table[(int64_t)b * A.max_pages + k / A.page_size];
                        if (page < 0 || page >= A.num_pages) continue;
                        // (a value that was not taken out has its infinity or NaN in the sum already, and a
                        // second one changes nothing)
                        const uint16_t *v = A.v_cache + page * A.page_stride + (k % A.page_size) * A.slot_stride +
                                            h * A.head_stride + c0;
#pragma unroll 1
                        for (int d = 0; d < entries; ++d) {
                            const float y = bf16_lo(v[d]);
                            if (isfinite(y)) continue;
                            if (slot >= 0) part_o[(int64_t)d * A.ncap] += y;
                            else out[d] = uint16_t(pack_bf16x2(bf16_lo(out[d]) + y, 0.f));
                        }
                    }
                }
            }
            // O is read, by the other stream's threads too, before this stream's next P lets it be written
            quad_sync();
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (__builtin_expect(C.gave_up, 0)) {
        // No warp issues any more.  What is in flight lands before the CTA ends: the products, each slot's
        // latest copy, the queries.
        if (warp == kWarpTMma) {
            if (elect_one()) mma_commit(&C.drained);
            __syncwarp();
            mbar_wait_bounded(&C.drained, 0, kDrainTimeoutNs);
        } else if (warp == kWarpTK) {
            bool landed = true;
            for (int kv = 0; kv < 2; ++kv) {
                const int slots = kv ? A.v_slots : A.k_slots, n = C.issued[kv];
                for (int k = max(n - slots, 0); landed && k < n; ++k)
                    landed = mbar_wait_bounded(&C.full[(kv ? A.k_slots : 0) + k % slots], (k / slots) & 1, kDrainTimeoutNs);
            }
            for (int k = max(C.q_issued - 2, 0); landed && k < C.q_issued; ++k)
                landed = mbar_wait_bounded(&C.q_full[k & 1], (k >> 1) & 1, kDrainTimeoutNs);
        }
        if (tid == 0) atomicOr(A.status, kStatusWaitTimeout);
        __syncthreads();
    }
    if (warp == kWarpTMma) tmem_free(tmem, kTmemCols);
}

constexpr int kThreadsJoin = 256;

// Adds the parts of a cut unit in the order of the keys: for column n, entries d .. d + kEntries - 1.  The loads of
// kParts parts are in flight at once.
template <int D, int kEntries, int kParts>
__device__ __forceinline__ void join_entries(const TreeArgs &A, const Cut &cut, int first_cta, int n, int d) {
    static_assert(kEntries == 16 || kEntries == 4, "one store");
    float top = kRefMin, l = 0.f, acc[kEntries] = {};
    for (int k0 = 0; k0 < cut.members; k0 += kParts) {
        float ref[kParts], sum[kParts], o[kParts][kEntries];
#pragma unroll
        for (int k = 0; k < kParts; ++k) {
            ref[k] = kRefMin;
            sum[k] = 0.f;
#pragma unroll
            for (int e = 0; e < kEntries; ++e) o[k][e] = 0.f;
            if (k0 + k < cut.members) {
                // (2 * kAttnMaxCtas * 128 * 256 floats at most: 32 bits)
                const uint32_t slot = k0 + k == 0 ? 2 * first_cta + 1 : 2 * (first_cta + k0 + k);
                const float *stat = A.stat + slot * 2 * A.ncap + n, *part = A.part + (slot * D + d) * A.ncap + n;
                ref[k] = __ldcg(stat);
                sum[k] = __ldcg(stat + A.ncap);
#pragma unroll
                for (int e = 0; e < kEntries; ++e) {
                    o[k][e] = __ldcg(part);
                    part += A.ncap;
                }
            }
        }
        float now = top;
#pragma unroll
        for (int k = 0; k < kParts; ++k) now = fmaxf(now, ref[k]);
        const float f = exp2_approx((top - now) * A.scale2);
        top = now;
        l *= f;
#pragma unroll
        for (int e = 0; e < kEntries; ++e) acc[e] *= f;
#pragma unroll
        for (int k = 0; k < kParts; ++k) {
            const float w = exp2_approx((ref[k] - now) * A.scale2);
            l = fmaf(w, sum[k], l);
#pragma unroll
            for (int e = 0; e < kEntries; ++e) acc[e] = fmaf(w, o[k][e], acc[e]);
        }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    uint16_t *const out = A.out + ((int64_t)(cut.row0 + n / A.G) * A.Hq + cut.head0 + n % A.G) * D + d;
    uint32_t y[kEntries / 2];
#pragma unroll
    for (int e = 0; e < kEntries; e += 2) y[e / 2] = pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
    if constexpr (kEntries == 16) st_global32(out, y, A.wide_out);
    else *reinterpret_cast<uint2 *>(out) = make_uint2(y[0], y[1]);
}

// A warp takes 32 columns of a unit, a lane each, and some of their entries: 16 where there are up to three parts,
// 4 where there are more, so that some 50 loads are in flight either way.  (16 and 4 everywhere: 19 parts of 240 columns
// 30.7 and 22.3 us for the call, 32 requests' two or three parts 72.5 and 79.2.  2 and 8 entries for the 19 parts, in an
// earlier version where 4 took 25.1: 27.3 and 29.1; 2 entries are bound by their instructions.  A third kind, 8 entries
// of up to 6 parts: 2 requests of 4095 keys 25.2 to 23.8, but one 18.5 to 18.7 and one of 65 000 62.2 to 64.6.)
constexpr int kFewParts = 3, kEntriesFew = 16, kManyParts = 10, kEntriesMany = 4;

template <int D>
__global__ void __launch_bounds__(kThreadsJoin) join_parts_kernel(const TreeArgs A, int ctas) {
    static_assert(kAttnMaxCtas <= kThreadsJoin, "a thread for each CTA's unit");
    __shared__ int before[kThreadsJoin + 1], warp_sum[kThreadsJoin / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    Cut mine{0, 0, 0, 0};
    if (tid < ctas) mine = A.cuts[tid];
    auto each = [](int members) { return D / (members <= kFewParts ? kEntriesFew : kEntriesMany); };
    const int groups = mine.members > 1 ? (mine.ncols + 31) / 32 * each(mine.members) : 0;
    int x = groups;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) warp_sum[warp] = x;
    __syncthreads();
    for (int w = 0; w < warp; ++w) x += warp_sum[w];
    before[tid] = x - groups;
    if (tid == kThreadsJoin - 1) before[kThreadsJoin] = x;
    __syncthreads();
    const int total = before[kThreadsJoin];
    for (int i = blockIdx.x * (kThreadsJoin / 32) + warp; i < total; i += gridDim.x * (kThreadsJoin / 32)) {
        int u = 0;  // the CTA whose unit it is
#pragma unroll
        for (int o = kThreadsJoin / 2; o > 0; o >>= 1)
            if (before[u + o] <= i) u += o;
        const Cut cut = A.cuts[u];
        const int g = i - before[u], parts = each(cut.members), n = g / parts * 32 + lane, d = g % parts;
        if (n >= cut.ncols) continue;
        if (cut.members <= kFewParts) join_entries<D, kEntriesFew, kFewParts>(A, cut, u, n, d * kEntriesFew);
        else join_entries<D, kEntriesMany, kManyParts>(A, cut, u, n, d * kEntriesMany);
    }
}

template <int D, bool kBox>
cudaError_t launch_tree(TreeArgs A, const CUtensorMap (&maps)[3], int ctas, cudaStream_t s) {
    constexpr size_t slot = size_t(D) * 2 * kTile, room = (kSmemBytes - sizeof(TCtrl)) / slot;
    static_assert(D == 64 || room >= 2 + 5, "two blocks of queries, two tiles of K and three of V");
    A.slots = int(std::min<size_t>(room - 2, kSlotsT));
    A.k_slots = A.slots / 2;
    A.v_slots = A.slots - A.k_slots;
    const size_t smem = (2 + A.slots) * slot + sizeof(TCtrl);
    cudaError_t e = cudaFuncSetAttribute(tree_attention_kernel<D, kBox>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         int(smem));
    if (e != cudaSuccess) return e;
    e = launch_overlapped(tree_attention_kernel<D, kBox>, ctas, kThreadsT, smem, s, A, maps[0], maps[1], maps[2]);
    if (e != cudaSuccess) return e;
    return launch_overlapped(join_parts_kernel<D>, 4 * ctas, kThreadsJoin, 0, s, A, ctas);
}

// Rows of a block, and of a unit.
int block_rows(int Hq, int Hkv, int q_max) { return std::min(q_max, kTile / (Hq / Hkv)); }
int unit_rows(int Hq, int Hkv, int q_max) { return std::min(q_max, 2 * block_rows(Hq, Hkv, q_max)); }
// Where the workspace has the cut units, behind the parts.
size_t cuts_at(int Hq, int Hkv, int D, int q_max) {
    const size_t cols = size_t(unit_rows(Hq, Hkv, q_max)) * (Hq / Hkv);
    return kHeaderBytes + align256(2 * kAttnMaxCtas * cols * D * sizeof(float)) +
           align256(2 * kAttnMaxCtas * 2 * cols * sizeof(float));
}

}  // namespace

bool tree_list_fits(const dspark_attn &a) {
    const int rows = unit_rows(a.Hq, a.Hkv, a.q_max);
    const long long units = (a.q_max + rows - 1) / rows + 1;
    const long long places = ((long long)a.max_pages * a.page_size / kTile + 2) * kTileTwo + kUnitPlaces;
    return places * units * a.Hkv <= INT32_MAX / a.B;
}

size_t tree_attn_workspace_bytes(int Hq, int Hkv, int D, int q_max) {
    return cuts_at(Hq, Hkv, D, q_max) + sizeof(Cut) * kAttnMaxCtas;
}

cudaError_t launch_step_attention_tree(const dspark_attn &a, const uint64_t *row_seen, int sinks, int sms, uint64_t wait_ns,
                                  cudaStream_t s) {
    TreeArgs A{};
    A.row_seen = row_seen;
    A.packed_pos = a.packed_pos;
    CUtensorMap maps[3];
    A.rb = block_rows(a.Hq, a.Hkv, a.q_max);
    const int rows = unit_rows(a.Hq, a.Hkv, a.q_max);
    const cudaError_t e = step_args(a, sinks, rows, rows * (a.Hq / a.Hkv), A.rb, wait_ns, A, maps);
    if (e != cudaSuccess) return e;
    A.wide_out = reinterpret_cast<uintptr_t>(a.out) % 32 == 0;
    A.cuts = reinterpret_cast<Cut *>(static_cast<char *>(a.workspace) + cuts_at(a.Hq, a.Hkv, a.D, a.q_max));
    const int ctas = std::min(sms, kAttnMaxCtas);
    if (A.box) return a.D == 128 ? launch_tree<128, true>(A, maps, ctas, s) : launch_tree<64, true>(A, maps, ctas, s);
    return a.D == 128 ? launch_tree<128, false>(A, maps, ctas, s) : launch_tree<64, false>(A, maps, ctas, s);
}

}  // namespace dspark
