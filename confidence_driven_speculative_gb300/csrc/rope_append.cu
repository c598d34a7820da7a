// rope_append.cu -- position rotation of q and k, and append of k and v to a
// paged cache.
//
// Mathematics: pair i of a head at position p turns by p * f_i.  The
// frequency comes as an integer F_i in 2^-64 of a turn, so the phase
// p * F_i mod 2^64 is exact, and its top 32 bits (2^-32 of a turn, below
// fp32's resolution of the result) give the angle in half turns in [-1, 1)
// for sincospif.  The rotation is fp32, rounded once to bfloat16.
//
// Bound: bytes.  A row of Hq + 2 Hkv heads is read once and written once.  A
// CTA of 128 threads takes a row.  A thread keeps one pair of 16-byte chunks
// (8 rotation pairs) of a head and walks the heads with it, so its 8 sines and
// cosines are computed once per row, and the loads of up to four heads are in
// flight before the angles are needed.
//
// Measured, Hq = 32, Hkv = 8, D = 128: 20 425 rows, no padding, k_rot written
// too, 84.7 us, 6.4 TB/s, 95 % of a copy's rate; 1024 rows of 256 requests in
// 4352 slots 6.7 us; one request's 17 rows 3.8 us a call, the host's part and
// the launch.
#include "attn.cuh"
#include "dspark_internal.cuh"
#include "tcgen05.cuh"

namespace dspark {
namespace {

constexpr int kRopeThreads = 128;
constexpr int kHeadsInFlight = 4;

struct RopeArgs {
    int B, rows, Hq, Hkv, page_size, num_pages, max_pages, rot_dim;
    int64_t q_stride, k_stride, v_stride, page_stride, slot_stride, head_stride;
    const uint16_t *q, *k, *v;
    uint16_t *q_rot, *k_rot, *k_cache, *v_cache;
    const int32_t *row_req, *packed_pos, *block_table, *row_off, *seq_lens;
    const uint64_t *freq;
};

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// (a, b) chunks of 8 elements: rotate element i of a with element i of b
// (halves), or neighbours inside a and inside b (interleaved).
template <bool kInterleaved>
__device__ __forceinline__ void rotate(uint4 &a, uint4 &b, const float (&c)[8], const float (&s)[8]) {
    float x[8], y[8];
    Vec<uint16_t>::unpack(a, x);
    Vec<uint16_t>::unpack(b, y);
    uint32_t *ra = reinterpret_cast<uint32_t *>(&a), *rb = reinterpret_cast<uint32_t *>(&b);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (kInterleaved) {
            ra[i] = pack_bf16(x[2 * i] * c[i] - x[2 * i + 1] * s[i],
                              x[2 * i + 1] * c[i] + x[2 * i] * s[i]);
            rb[i] = pack_bf16(y[2 * i] * c[4 + i] - y[2 * i + 1] * s[4 + i],
                              y[2 * i + 1] * c[4 + i] + y[2 * i] * s[4 + i]);
        } else {
            const int j = 2 * i, k = 2 * i + 1;
            ra[i] = pack_bf16(x[j] * c[j] - y[j] * s[j], x[k] * c[k] - y[k] * s[k]);
            rb[i] = pack_bf16(y[j] * c[j] + x[j] * s[j], y[k] * c[k] + x[k] * s[k]);
        }
    }
}

// kTree: the entry's place is seq_lens[b] + the row's index, and not its position.
template <int D, bool kInterleaved, bool kTree>
__device__ __forceinline__ void append_row(const RopeArgs &A, int r, int b, int pos) {
    constexpr int kLanes = D / 16;  // threads of a head, two 16-byte chunks each
    constexpr int kHeads = kRopeThreads / kLanes;
    if (b < 0 || b >= A.B || pos < 0) return;
    const int c = threadIdx.x % kLanes;
    // The thread's two chunks of a head (element offsets) and its first
    // pair.  Chunk pairs past the rotated part are plain copies.
    const int rc = A.rot_dim / 16;
    const bool turns = c < rc;
    int e0 = 16 * c, e1 = 16 * c + 8;
    if (turns && !kInterleaved) { e0 = 8 * c; e1 = 8 * c + A.rot_dim / 2; }
    int place = pos;
    if (kTree) {
        // far past any table, where nothing is stored, stays in 32 bits
        place = (A.seq_lens ? min(max(A.seq_lens[b], 0), INT32_MAX - DSPARK_MAX_ROWS) : 0) + r - A.row_off[b];
        if (place < 0) return;
    }
    const int page_i = place / A.page_size;
    int page = -1;
    if (A.k && page_i < A.max_pages) page = A.block_table[(int64_t)b * A.max_pages + page_i];
    const bool stored = page >= 0 && page < A.num_pages;
    const int64_t entry = stored ? page * A.page_stride + (place % A.page_size) * A.slot_stride : 0;

    const int q_heads = A.q ? A.Hq : 0, kv_heads = A.k ? A.Hkv : 0;
    const int slots = q_heads + 2 * kv_heads;
    float cs[8], sn[8];
    bool have = false;
    for (int h0 = threadIdx.x / kLanes; h0 < slots; h0 += kHeads * kHeadsInFlight) {
        uint4 x[kHeadsInFlight], y[kHeadsInFlight];
#pragma unroll
        for (int u = 0; u < kHeadsInFlight; ++u) {
            const int h = h0 + u * kHeads;
            if (h >= slots) continue;
            const uint16_t *src =
                h < q_heads ? A.q + r * A.q_stride + (int64_t)h * D
                : h < q_heads + kv_heads ? A.k + r * A.k_stride + (int64_t)(h - q_heads) * D
                                         : A.v + r * A.v_stride + (int64_t)(h - q_heads - kv_heads) * D;
            x[u] = *reinterpret_cast<const uint4 *>(src + e0);
            y[u] = *reinterpret_cast<const uint4 *>(src + e1);
        }
        if (!have && turns) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint64_t phase = A.freq[8 * c + i] * uint64_t(uint32_t(pos));
                // top word as a signed fraction of a turn, in half turns
                sincospif(float(int32_t(phase >> 32)) * (1.0f / 2147483648.0f), &sn[i], &cs[i]);
            }
            have = true;
        }
#pragma unroll
        for (int u = 0; u < kHeadsInFlight; ++u) {
            const int h = h0 + u * kHeads;
            if (h >= slots) continue;
            const bool is_q = h < q_heads, is_k = !is_q && h < q_heads + kv_heads;
            if (turns && (is_q || is_k)) rotate<kInterleaved>(x[u], y[u], cs, sn);
            const int kvh = is_q ? 0 : is_k ? h - q_heads : h - q_heads - kv_heads;
            if (is_q || (is_k && A.k_rot)) {
                uint16_t *dst = is_q ? A.q_rot + ((int64_t)r * A.Hq + h) * D
                                     : A.k_rot + ((int64_t)r * A.Hkv + kvh) * D;
                *reinterpret_cast<uint4 *>(dst + e0) = x[u];
                *reinterpret_cast<uint4 *>(dst + e1) = y[u];
            }
            if (!is_q && stored) {
                uint16_t *dst = (is_k ? A.k_cache : A.v_cache) + entry + kvh * A.head_stride;
                *reinterpret_cast<uint4 *>(dst + e0) = x[u];
                *reinterpret_cast<uint4 *>(dst + e1) = y[u];
            }
        }
    }
}

// A CTA for each row slot.
template <int D, bool kInterleaved, bool kTree>
__global__ void __launch_bounds__(kRopeThreads) rope_append_kernel(const RopeArgs A) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    append_row<D, kInterleaved, kTree>(A, blockIdx.x, A.row_req[blockIdx.x], A.packed_pos[blockIdx.x]);
}

// The CTAs walk the row slots; the next one's place is asked for before this
// one's work.
template <int D, bool kInterleaved, bool kTree>
__global__ void __launch_bounds__(kRopeThreads) rope_append_walk_kernel(const RopeArgs A) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    int b = A.row_req[blockIdx.x], pos = A.packed_pos[blockIdx.x];
    for (int r = blockIdx.x; r < A.rows;) {
        const int next = r + gridDim.x;
        int b_next = -1, pos_next = -1;
        if (next < A.rows) {
            b_next = A.row_req[next];
            pos_next = A.packed_pos[next];
        }
        append_row<D, kInterleaved, kTree>(A, r, b, pos);
        r = next;
        b = b_next;
        pos = pos_next;
    }
}

template <int D, bool kInterleaved>
auto *rope_kernel(bool walk, bool tree) {
    return walk ? (tree ? rope_append_walk_kernel<D, kInterleaved, true> : rope_append_walk_kernel<D, kInterleaved, false>)
                : (tree ? rope_append_kernel<D, kInterleaved, true> : rope_append_kernel<D, kInterleaved, false>);
}

}  // namespace

cudaError_t launch_rope_append(const dspark_attn &a, bool tree, int sms, cudaStream_t s) {
    RopeArgs A{a.B, a.rows, a.Hq, a.Hkv, a.page_size, a.num_pages, a.max_pages, a.rot_dim,
               a.q_stride, a.k_stride, a.v_stride, a.page_stride, a.slot_stride, a.head_stride,
               static_cast<const uint16_t *>(a.q), static_cast<const uint16_t *>(a.k),
               static_cast<const uint16_t *>(a.v), static_cast<uint16_t *>(a.q_rot),
               static_cast<uint16_t *>(a.k_rot), static_cast<uint16_t *>(a.k_cache),
               static_cast<uint16_t *>(a.v_cache), a.row_req, a.packed_pos, a.block_table,
               a.row_off, a.seq_lens, a.rope_freq};
    if (!a.k) A.page_size = 1;  // not checked, not used
    // Walking pays where most slots are padding, as in a batch of steps: a CTA
    // that finds an empty slot costs a launch, a walker a load that is already
    // under way.  4352 slots with 1024 rows: 7.6 us with a CTA a slot, 6.4
    // with 14 walkers an SM.  Where the slots are full it costs a little
    // (4096 rows: 20.6 us against 21.5; 8192: 36.7 against 37.4), and more the
    // longer the walk (32768: 134 against 150), so long lists keep a CTA a slot.
    const int walkers = 14 * sms;
    const bool walk = a.rows > walkers && a.rows <= 4 * walkers;
    auto *kernel = a.D == 128 ? (a.interleaved ? rope_kernel<128, true>(walk, tree) : rope_kernel<128, false>(walk, tree))
                              : (a.interleaved ? rope_kernel<64, true>(walk, tree) : rope_kernel<64, false>(walk, tree));
    return launch_overlapped(kernel, walk ? walkers : a.rows, kRopeThreads, 0, s, A);
}

}  // namespace dspark
