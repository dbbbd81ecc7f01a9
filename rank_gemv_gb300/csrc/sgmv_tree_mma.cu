// sgmv_tree_mma.cu -- tree attention on the tensor cores, for heads of up to
// 128 columns.
//
// The rows of one sequence that share a KV head (nodes x query heads of the
// group) are cut into row tiles of RT = 8, 16, 32, 64 or 128, the tokens into
// tiles of 128.  Both products run transposed, so that the long axis (tokens,
// then head columns) fills the 128 lanes of the tensor cores however few rows
// there are:
//
//   S^T [tokens x RT] = K . Q^T          A = K tile (K-major),  B = Q rows
//   O^T [columns x RT] += V^T . P^T      A = V tile (M-major),  B = P
// (of 16 columns at least: with RT = 8 nobody reads the others)
//
// with S^T and O^T in tensor memory.  A softmax thread owns one token: it
// reads its scores, makes p = 2^(c s - ref[row]) and writes them as one row
// of P.  ref[row] is the row's running maximum, moved only when a score
// exceeds it by more than 2^kSlack (then O^T and the sums are scaled), so an
// ordinary tile needs one vote and no reduction over tokens.
//
// Decomposition: the (sequence, head, row tile) items, each of ceil(length /
// 128) token tiles and one or two more for what its end costs, form one line of
// work that is cut into equal shares, one per CTA of a grid that fills the GPU
// once.  A share that covers an item writes its output; items cut across shares
// leave unnormalised O, sums and
// references in the workspace, and a second, small kernel joins them, in share
// order.  (Joined by whichever CTA finished last, behind a fence and a counter, each join
// took 15 us: its chain of loads queued behind the stream of K and V.  Claiming the
// last quarter of the line in small shares at run time balanced the SMs' unequal
// bandwidth, but its parts and joins cost more than it won: 188, 287 and 67 us against
// 182, 275 and 61 on 32 trees, 64 heads on 8, and 128 decode rows.)
//
// Warps: 4, 4, 4, 8 or 16 for the softmax (32 rows each four); one that issues the
// MMAs, a score product ahead of the softmax; one that walks the line,
// brings Q in and says which rows see which tree nodes; two that bring K and V
// into a ring of 32 KB stages, through the block table: by TMA, or, for pages
// that are no multiple of 8 tokens, with cp.async, 16 bytes per lane.
//
// Values that a row does not see never reach it: scores are masked after
// the product, and non-finite v of tree nodes are taken out of the staged
// tile (a masked weight of 0 times infinity would be NaN) and added back for
// the rows that do see them.
#include <math.h>

#include <algorithm>
#include <climits>
#include <numeric>
#include <type_traits>

#include "sgmv_device.cuh"
#include "sgmv_internal.h"
#include "sgmv_spec.h"
#include "sgmv_tcgen05.cuh"

namespace sgmv {
namespace {

constexpr int kTok = 128;                // lanes: tokens per tile, at most
constexpr uint32_t kHalf = kTok * 128u;  // bytes of 64 columns of a tile
constexpr uint32_t kStage = 2 * kHalf;   // a K or V tile, 128 columns
constexpr int kLoaders = 64;             // loading threads
constexpr int kSegs = 4;                 // segments known ahead
constexpr float kUnset = -3e38f;         // ref of a row that has seen nothing
constexpr float kBias = 7.f;             // weights are 2^(kBias + score - ref) ...
constexpr float kSlack = 8.f;            // ... <= 2^(kBias + kSlack), finite in f16
constexpr int kMaxSms = 152;
constexpr int kSeqTable = 64;            // entries of the table that finds a tile's sequence
constexpr int kMaxParts = 64;            // parts of an item (about)

template <int RT> struct Shape {
    static constexpr int kGroups = RT > 32 ? RT / 32 : 1;  // softmax warpgroups
    static constexpr int kRows = RT / kGroups;            // rows per warpgroup
    static constexpr int kN = RT < 16 ? 16 : RT;          // columns of the products, the least there is
    static constexpr int kSoft = 128 * kGroups;           // softmax threads
    static constexpr int kThreads = kSoft + 64 + kLoaders;
    // Two CTAs per SM where they fit: one's sums and segment changes hide behind
    // the other's loads (128 decode rows 76 us
    // with one, 67 with two).
    static constexpr int kPerSm = RT <= 16 ? 2 : 1;
    static constexpr int kQ = RT > 64 || kPerSm > 1 ? 1 : 2;  // Q buffers
    static constexpr int kStages = kPerSm > 1 ? 3 : RT > 64 ? 4 : 5;
    // What an item costs beside its tiles, in tiles: with 0, 1 and 2, 32 trees over 4096
    // tokens took 202, 191 and 191 us (32 nodes, RT 32), 227, 209 and 204 (64), 155,
    // 145 and 137 (64 nodes, 32 heads on 8, RT 128; 136 with 3).
    static constexpr int kEnd = RT > 32 ? 2 : 1;
    static constexpr int kWords = RT < 32 ? 1 : RT / 32;  // words of one bit per row
    static constexpr uint32_t kQBytes = kN * 256u;
    // A token's row of P: 64 columns of 128-byte swizzle, or 16 of 32-byte swizzle
    static constexpr uint32_t kPRow = RT <= 16 ? 32 : 128;
    static constexpr uint32_t kPBytes = (RT > 64 ? 2 : 1) * kTok * kPRow;
    static constexpr uint32_t kTmem = RT <= 16 ? 64 : RT <= 32 ? 128 : RT <= 64 ? 256 : 512;
    // dynamic shared memory
    static constexpr uint32_t kOffQ = kStages * kStage;
    static constexpr uint32_t kOffP = kOffQ + kQ * kQBytes;
    static constexpr uint32_t kOffTab = kOffP + kPBytes;            // cp.async: row offsets of 2 tiles
    static constexpr uint32_t kOffSee = kOffTab + 2u * kTok * 8u;   // who sees each node, two trees
    static constexpr uint32_t kOffRow = kOffSee + 2u * SGMV_TREE_MAX_NODES * kWords * 4u;  // rows' places
    static constexpr uint32_t kBytes = kOffRow + kSegs * RT * 8u + 1024u;  // + alignment
};

struct MmaParams {
    // the caches as [page][head][token][D], boxes of `box` tokens by 64 columns
    CUtensorMap map_k, map_v;
    CUtensorMap map_q;  // q as [token][head][D], boxes of a row tile's nodes x the group x 64 columns
    int32_t q_box;    // 0: row tiles do not hold whole nodes, or q's strides do not fit a map: cp.async
    int32_t box;      // tokens per box; 0: cp.async
    int32_t tok;      // tokens per tile: 128, or the boxes that fit in 128
    sgmv_tree_attention_args a;
    float c;          // scale * log2(e)
    int32_t group;    // query heads per KV head
    int ctas;         // shares at most
    int *shares;      // shares of this call
    struct Cut *cut;  // [share]: the cut item that begins there
    float *ml;        // [share][2][RT][2]: reference and sum of parts of items
    float *part;      // [share][2][RT][128]
    int *err;
    int inject;       // diagnostic launch: the role (1 to 4) whose wait runs out
};

// An item whose parts are in the workspace; parts = 0: none.
struct Cut {
    int t0, n, h, rt, first, parts, pad0, pad1;
};

// The tiles of one item inside one share.  Begins at the item's first tile:
// slot 2 share + 1, else 2 share (the share's first).
struct Segment {
    int b, t0, n, prefix, total;     // sequence
    int h, rt;                       // KV head, row tile
    int tile, end;                   // tiles; end = 0: no more segments
    int whole;                       // the whole item
    int slot;                        // where a part goes
    int see;                         // which tree table
};

// How the line of W tiles (ends counted) is cut: share i is [i own, (i + 1) own).
struct Plan {
    int64_t W, own;
    int32_t stride;
    int64_t before[kSeqTable];       // tiles before every stride-th sequence
    int32_t t0[kSeqTable], n[kSeqTable], prefix[kSeqTable];  // of the sequences, if there are no more
};

// A sequence's part of the line.
struct Sequence {
    int b, t0, n, prefix, total, tiles, nrt, each;  // each: an item's place on the line
    uint32_t items;

    // false: bad metadata
    template <int RT> __device__ __forceinline__ bool enter(const MmaParams &P, int b_, const Plan *plan = nullptr) {
        const sgmv_tree_attention_args &a = P.a;
        b = b_;
        if (plan && a.B <= kSeqTable) {
            t0 = plan->t0[b];
            n = plan->n[b];
            prefix = plan->prefix[b];
        } else {
            t0 = a.tree_ptr[b];
            n = a.tree_ptr[b + 1] - t0;
            prefix = a.prefix_lens[b];
        }
        items = 0;
        tiles = each = 1;
        if (!(t0 >= 0 && n >= 0 && n <= SGMV_TREE_MAX_NODES && (int64_t)t0 + n <= a.T && prefix >= 0 &&
              (int64_t)prefix + n <= (int64_t)a.max_blocks * a.block_size && prefix <= INT_MAX - 2 * kTok - n))
            return false;
        if (n == 0) return true;
        total = prefix + n;
        tiles = (total + P.tok - 1) / P.tok;
        each = tiles + Shape<RT>::kEnd;
        nrt = (n * P.group + RT - 1) / RT;
        items = (uint32_t)P.a.Hkv * (uint32_t)nrt;
        return true;
    }
    __device__ __forceinline__ int64_t work() const { return (int64_t)items * each; }
};

// Bounded wait of a whole warp; false if it ran out for any lane.  Then, or when
// another role's did, `lost` is set, and every wait that would last returns false at
// once.  The roles that walk, load and multiply stop there, so that nothing is copied or
// armed out of turn; the softmax warps, which meet at barriers of their own, finish
// their segment on whatever the buffers hold and write none of it.  The end of the
// kernel waits for the copies in flight and marks the share for the join.
__device__ __forceinline__ bool await(uint64_t *bar, uint32_t parity, volatile int *lost) {
    bool there = mbar_try_wait(bar, parity);
    if (!there) {
        const uint64_t t0 = global_ns();
        for (uint32_t i = 0;; ++i) {
            if (*lost || i >= kMaxPolls || global_ns() - t0 > kWaitLimitNs) {
                *lost = 1;
                break;
            }
            if ((there = mbar_try_wait(bar, parity))) break;
        }
    }
    return __all_sync(0xffffffffu, there);
}

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// One lane of the (whole) warp, always the same.
__device__ __forceinline__ uint32_t elect() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n" : "=r"(r));
    return r;
}
// As mma_f16 and mma_commit, by the lane whose `on` is set: a predicate in
// place of a branch keeps the operands in uniform registers.
__device__ __forceinline__ void mma_on(uint32_t on, uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                       uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(on)
        : "memory");
}
__device__ __forceinline__ void commit_on(uint32_t on, uint64_t *bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}\n" ::"r"(
            smem_addr(bar)),
        "r"(on)
        : "memory");
}
// Two fp32 operations in one instruction, each rounded as alone.
__device__ __forceinline__ void fma_pair(float &x, float &y, float c, float a, float b) {
    uint64_t v, w, k;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(x), "f"(y));
    asm("mov.b64 %0, {%1, %1};" : "=l"(k) : "f"(c));
    asm("mov.b64 %0, {%1, %2};" : "=l"(w) : "f"(a), "f"(b));
    asm("fma.rn.f32x2 %0, %0, %1, %2;" : "+l"(v) : "l"(k), "l"(w));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
}
__device__ __forceinline__ void add_pair(float &x, float &y, float a, float b) {
    uint64_t v, w;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(x), "f"(y));
    asm("mov.b64 %0, {%1, %2};" : "=l"(w) : "f"(a), "f"(b));
    asm("add.rn.f32x2 %0, %0, %1;" : "+l"(v) : "l"(w));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
}
__device__ __forceinline__ void sts16(void *p, uint16_t v) {
    asm volatile("st.shared.u16 [%0], %1;" ::"r"(smem_addr(p)), "h"(v) : "memory");
}
// Barrier of the 128 threads of softmax warpgroup g; with a vote.
__device__ __forceinline__ void group_bar(int g) {
    asm volatile("barrier.cta.sync %0, 128;" ::"r"(2 + g) : "memory");
}
__device__ __forceinline__ bool group_any(int g, bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %2, 0;\n\t"
        "barrier.cta.red.or.pred q, %1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}\n"
        : "=r"(r)
        : "r"(2 + g), "r"((uint32_t)v)
        : "memory");
    return r != 0;
}
// Tensor memory, 32 lanes x N columns; the whole warp, brought together first.
template <int N> __device__ __forceinline__ void tmem_load(uint32_t addr, float (&v)[N]) {
    __syncwarp();
    if constexpr (N == 32)
        tmem_ld32(addr, v);
    else if constexpr (N == 16)
        tmem_ld16(addr, v);
    else
        tmem_ld8(addr, v);
}
template <int N> __device__ __forceinline__ void tmem_store(uint32_t addr, const float (&v)[N]) {
    __syncwarp();
    if constexpr (N == 8)
        asm volatile(
            "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(addr),
            "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])),
            "r"(__float_as_uint(v[3])), "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])),
            "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7]))
            : "memory");
#pragma unroll
    for (int i = 0; i + 16 <= N; i += 16)
        asm volatile(
            "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
            "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr + i),
            "r"(__float_as_uint(v[i])), "r"(__float_as_uint(v[i + 1])), "r"(__float_as_uint(v[i + 2])),
            "r"(__float_as_uint(v[i + 3])), "r"(__float_as_uint(v[i + 4])), "r"(__float_as_uint(v[i + 5])),
            "r"(__float_as_uint(v[i + 6])), "r"(__float_as_uint(v[i + 7])), "r"(__float_as_uint(v[i + 8])),
            "r"(__float_as_uint(v[i + 9])), "r"(__float_as_uint(v[i + 10])), "r"(__float_as_uint(v[i + 11])),
            "r"(__float_as_uint(v[i + 12])), "r"(__float_as_uint(v[i + 13])),
            "r"(__float_as_uint(v[i + 14])), "r"(__float_as_uint(v[i + 15]))
            : "memory");
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// v[i], i < N: row i's partial of every lane.  Afterwards lane l holds, in
// v[0], the whole warp's sum or maximum (NaN wins) of the row returned; a row of
// N < 32 is held by 32 / N lanes.
template <bool MAX> __device__ __forceinline__ float join2(float a, float b) {
    if (!MAX) return a + b;
    float m;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
    return m;
}
template <bool MAX, int N> __device__ __forceinline__ int warp_rows(float (&v)[N], int lane) {
    int row = 0;
    int n = N;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        if (n > 1) {
            n >>= 1;
            const bool up = lane & o;
            if (up) row += n;
#pragma unroll
            for (int i = 0; i < N / 2; ++i)
                if (i < n) {
                    const float give = up ? v[i] : v[i + n];
                    const float keep = up ? v[i + n] : v[i];
                    v[i] = join2<MAX>(keep, __shfl_xor_sync(0xffffffffu, give, o));
                }
        } else {
            v[0] = join2<MAX>(v[0], __shfl_xor_sync(0xffffffffu, v[0], o));
        }
    }
    return row;
}

// Non-finite 16-bit values: all ones in the exponent.
template <typename T> __device__ __forceinline__ bool bad16(uint32_t h) {
    constexpr uint32_t e = std::is_same<T, __half>::value ? 0x7C00u : 0x7F80u;
    return (h & e) == e;
}

// Row r of an item's row tile: its token (~token for a padding row) and query head.
__device__ __forceinline__ int2 row_place(const MmaParams &P, int t0, int h, int i) {
    const int node = i / P.group;
    int t = t0 + node;
    const int hq = h * P.group + (i - node * P.group);
    if (P.a.parents) {
        const int p = P.a.parents[t];
        if (p < -1 || p >= node) t = ~t;
    }
    return make_int2(t, hq);
}

template <typename T, int RT>
__global__ void __launch_bounds__(Shape<RT>::kThreads, Shape<RT>::kPerSm)
    sgmv_tree_mma_kernel(const __grid_constant__ MmaParams P) {
    using S = Shape<RT>;
    constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
    const sgmv_tree_attention_args &a = P.a;
    extern __shared__ __align__(1024) uint8_t dsm[];
    __shared__ __align__(8) uint64_t full[S::kStages], empty[S::kStages], q_full[S::kQ], q_empty[S::kQ];
    __shared__ __align__(8) uint64_t seg_full[kSegs], seg_empty[kSegs], aux_full[kSegs];
    __shared__ __align__(8) uint64_t p_full, pv_done, tab_ready, drained;
    __shared__ uint32_t s_tmem;
    __shared__ int s_lost, s_poison, s_longest, s_known;
    __shared__ int64_t s_sum[32];
    __shared__ Plan plan;
    __shared__ Segment s_seg[kSegs], s_cur[2];     // s_cur: the softmax warps' segment, and the next
    __shared__ int16_t s_parent[SGMV_TREE_MAX_NODES];
    __shared__ __align__(16) float s_ref[RT], s_fac[RT];  // s_ref: -ref
    __shared__ float s_red[4][RT];
    uint8_t *const sm = align1024(dsm);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    constexpr int kWarps = S::kThreads / 32, kMmaWarp = S::kSoft / 32, kWalkWarp = kMmaWarp + 1;

    if (warp == kMmaWarp) {
        if (lane == 0) {
            for (int i = 0; i < S::kStages; ++i)
                mbar_init(&full[i], P.box ? kLoaders / 32 : kLoaders), mbar_init(&empty[i], 1);
            for (int i = 0; i < S::kQ; ++i) mbar_init(&q_full[i], P.q_box ? 1 : 32), mbar_init(&q_empty[i], 1);
            for (int i = 0; i < kSegs; ++i) {
                mbar_init(&seg_full[i], 1);
                mbar_init(&seg_empty[i], 2 + kLoaders / 32);  // MMA, softmax, loaders
                mbar_init(&aux_full[i], 1);
            }
            mbar_init(&p_full, S::kSoft / 32);
            mbar_init(&pv_done, 1);
            mbar_init(&tab_ready, kLoaders);
            mbar_init(&drained, 1);
            mbar_init_fence();
            s_lost = s_longest = s_known = 0;
            s_poison = -1;
            for (int i = 0; i < kSegs; ++i) s_seg[i].tile = s_seg[i].end = 0;
        }
        __syncwarp();
        tmem_alloc(&s_tmem, S::kTmem);
    }
    for (int i = tid; i < RT; i += S::kThreads) s_ref[i] = -kUnset;
    // columns past D that the products read are zero: in Q, and in K where TMA
    // does not fill them; so are the rows past a short tile
    if (P.tok < kTok)
        for (uint32_t i = tid * 16u; i < S::kOffQ; i += S::kThreads * 16u)
            sts128(sm + i, make_uint4(0, 0, 0, 0));
    if (a.D % 64 != 0 && !(P.box && P.q_box))
        for (uint32_t i = (P.box ? S::kOffQ : 0u) + tid * 16u; i < S::kOffP; i += S::kThreads * 16u)
            sts128(sm + i, make_uint4(0, 0, 0, 0));
    fence_proxy_async();
    pdl_wait();
    pdl_trigger();

    // ---- the line of work -----------------------------------------------------
    const int stride = (a.B + kSeqTable - 1) / kSeqTable;
    int64_t W = 0;
    int longest = 0;
    __syncthreads();
    for (int b0 = 0; b0 < a.B; b0 += S::kThreads) {
        const int b = b0 + tid;
        int64_t own = 0;
        if (b < a.B) {
            Sequence q;
            if (!q.template enter<RT>(P, b) && blockIdx.x == 0) set_error(P.err, kErrBadSegments);
            own = q.work();
            if (own) longest = max(longest, q.tiles);
            if (b < kSeqTable) plan.t0[b] = q.t0, plan.n[b] = q.n, plan.prefix[b] = q.prefix;
        }
        int64_t run = own;
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t up = __shfl_up_sync(0xffffffffu, run, o);
            if (lane >= o) run += up;
        }
        if (b0) __syncthreads();  // the last round's sums have been read
        if (lane == 31) s_sum[warp] = run;
        __syncthreads();
        int64_t all = 0;
        for (int i = 0; i < kWarps; ++i) {
            if (i < warp) run += s_sum[i];
            all += s_sum[i];
        }
        if (b < a.B && b % stride == 0) plan.before[b / stride] = W + run - own;
        W += all;
    }
    longest = __reduce_max_sync(0xffffffffu, longest);
    if (lane == 0) atomicMax(&s_longest, longest);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    const int ctas = (int)gridDim.x;
    if (tid == 0) {
        plan.W = W;
        plan.stride = stride;
        // no more than kMaxParts parts or so of an item, for the join's sake
        plan.own = max(max((W + ctas - 1) / ctas, ((int64_t)s_longest + kMaxParts - 1) / kMaxParts), (int64_t)1);
        if (blockIdx.x == 0) *P.shares = (int)((W + plan.own - 1) / plan.own);
    }
    __syncthreads();
    if (plan.own * blockIdx.x >= W) {
        if (warp == kMmaWarp) tmem_dealloc(tmem, S::kTmem);
        return;
    }
    volatile int *const lost = &s_lost;
    const int D = a.D, group = P.group;
    const int cpr = D / 8;  // 16-byte chunks per row
    // a role's next segment, number i, is in s_seg[i % kSegs]
    auto segment_there = [&](int i) { return await(&seg_full[i % kSegs], (uint32_t)(i / kSegs) & 1, lost); };
    // A role takes an injected timeout as it would one of its waits.
    auto injected = [&](int role) {
        if (P.inject == role) *lost = 1;
        return P.inject == role;
    };
    int issued = 0;  // TMA copies of this warp: of Q (the walk), or K and V (the loaders)

    if (warp == kWalkWarp) {
        // ---- the walk along the line ---------------------------------------------
        const int id = (int)blockIdx.x;
        int64_t w = plan.own * id, base = 0;   // next tile; first tile of its sequence
        const int64_t w1 = min(W, w + plan.own);  // end of the share
        int see = 0, see_b = -1, see_rt = -1, see_user[2] = {-1, -1};
        Sequence q;
        {   // the table's last entry at or before w
            int lo = 0, hi = (a.B - 1) / plan.stride;
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (plan.before[mid] <= w) lo = mid;
                else hi = mid - 1;
            }
            base = plan.before[lo];
            q.template enter<RT>(P, lo * plan.stride, &plan);
        }
        if (lane == 0) P.cut[id] = Cut{};
        for (int i = 0; !injected(1); ++i) {
            if (i >= kSegs && !await(&seg_empty[i % kSegs], (uint32_t)(i / kSegs - 1) & 1, lost)) break;
            uint32_t item = 0;
            int tile = 0;
            while (w < w1) {
                while (w >= base + q.work()) {
                    base += q.work();
                    q.template enter<RT>(P, q.b + 1, &plan);
                }
                const uint32_t rel = (uint32_t)(w - base);
                item = rel / (uint32_t)q.each;
                tile = (int)(rel - item * (uint32_t)q.each);
                if (tile < q.tiles) break;
                w += q.each - tile;  // nothing to do for an end itself
            }
            if (w >= w1) {
                if (lane == 0) {
                    s_seg[i % kSegs].tile = s_seg[i % kSegs].end = 0;
                    mbar_arrive(&seg_full[i % kSegs]);
                }
                break;
            }
            const int h = (int)(item / (uint32_t)q.nrt), rt = (int)(item - (uint32_t)h * (uint32_t)q.nrt);
            const int end = w1 - w < q.tiles - tile ? tile + (int)(w1 - w) : q.tiles;
            const bool tree = end * P.tok > q.prefix, build = tree && (see_b != q.b || see_rt != rt);
            if (build) see ^= 1;
            if (lane == 0) {
                Segment &s = s_seg[i % kSegs];
                s.b = q.b;
                s.t0 = q.t0;
                s.n = q.n;
                s.prefix = q.prefix;
                s.total = q.total;
                s.h = h;
                s.rt = rt;
                s.tile = tile;
                s.end = end;
                s.whole = tile == 0 && end == q.tiles;
                s.slot = 2 * id + (tile == 0 ? 1 : 0);
                s.see = see;
                if (tile == 0 && !s.whole) {  // the share's last: the only item that it may begin and not end
                    Cut cut = {};
                    cut.t0 = q.t0;
                    cut.n = q.n;
                    cut.h = h;
                    cut.rt = rt;
                    cut.first = id;
                    cut.parts = (int)((w + q.tiles - 1) / plan.own) - id + 1;
                    P.cut[id] = cut;
                }
                *(volatile int *)&s_known = i + 1;
                mbar_arrive(&seg_full[i % kSegs]);
            }
            __syncwarp();
            w += end - tile;
            // the row tile's queries, and the rows' places
            const int qb = i % S::kQ, R = min(RT, q.n * group - rt * RT), halves = D > 64 ? 2 : 1;
            uint8_t *const qs = sm + S::kOffQ + (uint32_t)qb * S::kQBytes;
            int2 *const place = reinterpret_cast<int2 *>(sm + S::kOffRow) + (i % kSegs) * RT;
            auto bring_q = [&]() {
                if (P.q_box) {
                    // (rows past R are the next sequence's or zeros: finite or not,
                    // they end in columns of the products that nobody reads)
                    if (lane == 0) {
                        mbar_arrive_expect_tx(&q_full[qb], (uint32_t)halves * RT * 128u);
                        for (int half = 0; half < halves; ++half)
                            tma_load_3d(qs + half * S::kN * 128, &P.map_q, half * 64, h * group, q.t0 + rt * RT / group,
                                        &q_full[qb]);
                    }
                    __syncwarp();
                    issued = i + 1;
                    return;
                }
                for (int m = lane / cpr, c = lane % cpr; m < RT;) {
                    const T *src = static_cast<const T *>(a.q);
                    if (m < R) {
                        const int2 at = place[m];
                        src += (int64_t)(at.x < 0 ? ~at.x : at.x) * a.q_token + (int64_t)at.y * a.q_head + c * 8;
                    }
                    cp_async16(qs + (uint32_t)(c >> 3) * (S::kN * 128u) + sw128_offset(m, c & 7), src, m < R ? 16u : 0u);
                    m += 32 / cpr;
                    c += 32 % cpr;
                    if (c >= cpr) c -= cpr, ++m;
                }
                cp_async_arrive(&q_full[qb]);
            };
            if (i < S::kQ && P.q_box) bring_q();
            else if (P.q_box && lane < halves)  // its buffer is in use: as far as L2
                tma_prefetch_3d(&P.map_q, lane * 64, h * group, q.t0 + rt * RT / group);
            for (int r = lane; r < R; r += 32) place[r] = row_place(P, q.t0, h, rt * RT + r);
            __syncwarp();
            if (i < S::kQ && !P.q_box) bring_q();
            if (build) {
                // see[j]: the rows that see tree node j.  Every node of this row
                // tile marks itself and its ancestors with its rows' bits.
                see_b = q.b;
                see_rt = rt;
                // the table's last user is done (those kSegs back were waited for)
                const int u = see_user[see];
                if (u >= 0 && i - u < kSegs && !await(&seg_empty[u % kSegs], (uint32_t)(u / kSegs) & 1, lost)) break;
                uint32_t *const tab = reinterpret_cast<uint32_t *>(sm + S::kOffSee) +
                                      see * SGMV_TREE_MAX_NODES * S::kWords;
                for (int e = lane; e < q.n * S::kWords; e += 32) tab[e] = 0;
                for (int j = lane; j < q.n; j += 32) {
                    const int p = a.parents ? a.parents[q.t0 + j] : j - 1;
                    if (p < -2 || p >= j) set_error(P.err, kErrBadIndex);
                    s_parent[j] = (int16_t)(p < -1 || p >= j ? -2 : p);  // -2: padding
                }
                __syncwarp();
                const int node0 = rt * RT / group, node1 = (rt * RT + R - 1) / group;
                for (int node = node0 + lane; node <= node1; node += 32) {
                    const int lo = max(0, node * group - rt * RT), hi = min(R, (node + 1) * group - rt * RT);
                    for (int j = node; j >= 0 && s_parent[j] != -2; j = s_parent[j])
                        for (int k = lo >> 5; k <= (hi - 1) >> 5; ++k) {
                            const int l0 = max(lo - 32 * k, 0), l1 = min(hi - 32 * k, 32);
                            atomicOr(&tab[j * S::kWords + k], (0xffffffffu >> (32 - (l1 - l0))) << l0);
                        }
                }
                __syncwarp();
            }
            if (tree) see_user[see] = i;
            __syncwarp();
            if (lane == 0) mbar_arrive(&aux_full[i % kSegs]);
            if (i >= S::kQ) {
                if (!await(&q_empty[qb], (uint32_t)(i / S::kQ - 1) & 1, lost)) break;
                bring_q();
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp > kWalkWarp) {
        // ---- K and V: ring order K0, V0, K1, V1, ... ------------------------------
        const int lt = tid - S::kSoft - 64, halves = D > 64 ? 2 : 1;
        int st = 0;
        uint32_t ph = 1;  // parity of the stage's release that is waited for
        auto claim_stage = [&]() {
            if (issued >= S::kStages && !await(&empty[st], ph, lost)) return false;
            ++issued;
            return true;
        };
        auto advance = [&]() {
            if (++st == S::kStages) st = 0, ph ^= 1;
        };
        if (P.box) {
            // TMA: a box (tokens x 64 columns) per lane, dealt to the two warps
            const int box = P.box, nbox = P.tok / box, op = lane * (kLoaders / 32) + lt / 32;
            const int mine = op % nbox, half = op / nbox;
            const bool busy = half < halves;
            const uint32_t bytes = (uint32_t)__popc(__ballot_sync(0xffffffffu, busy)) * (uint32_t)box * 128u;
            const uint32_t at = (uint32_t)half * kHalf + (uint32_t)(mine * box) * 128u;
            int32_t page = 0;
            int in = -1;
            // page and place of this lane's box of a tile
            auto look = [&](const Segment &s, int tile) {
                const int j = tile * P.tok + mine * box;
                in = -1;
                if (j < s.total) {
                    const int pg = j / a.block_size;
                    in = j - pg * a.block_size;
                    page = a.block_table[s.b * a.table_row + pg];
                }
            };
            auto copy_boxes = [&](const CUtensorMap *map, int32_t pg, int row, int head) {
                if (!claim_stage()) return false;
                if (lane == 0) mbar_arrive_expect_tx(&full[st], bytes);
                __syncwarp();
                if (busy) tma_load_4d(sm + (uint32_t)st * kStage + at, map, half * 64, row, head, pg, &full[st]);
                advance();
                return true;
            };
            bool looked = false, stop = injected(2);
            for (int i = 0; !stop; ++i) {
                if (!segment_there(i)) break;
                const Segment s = s_seg[i % kSegs];
                if (s.end == 0) break;
                if (!looked) look(s, s.tile);
                for (int tile = s.tile; tile < s.end; ++tile) {
                    // boxes past the end, and pages out of range, read as zeros
                    int32_t pg = page;
                    int row = in;
                    if (row < 0 || pg < 0 || pg >= a.num_blocks) {
                        if (row >= 0) set_error(P.err, kErrBadIndex);
                        pg = a.num_blocks;
                        row = 0;
                    }
                    // the next tile's page is looked up meanwhile
                    looked = false;
                    if (tile + 1 < s.end) {
                        look(s, tile + 1);
                    } else if (__shfl_sync(0xffffffffu, *(volatile int *)&s_known, 0) > i + 1) {
                        looked = segment_there(i + 1);
                        if (looked) look(s_seg[(i + 1) % kSegs], s_seg[(i + 1) % kSegs].tile);
                    }
                    if (!copy_boxes(&P.map_k, pg, row, s.h) || !copy_boxes(&P.map_v, pg, row, s.h)) {
                        stop = true;
                        break;
                    }
                }
                if (lane == 0 && !stop) mbar_arrive(&seg_empty[i % kSegs]);
                __syncwarp();
            }
        } else {
            int64_t *const tab = reinterpret_cast<int64_t *>(sm + S::kOffTab);
            const int dm = kLoaders / cpr, dc = kLoaders - dm * cpr;
            constexpr int kBatch = 8;
            int g = 0;
            auto copy_tile = [&](const void *cache, int64_t off) {
                if (!claim_stage()) return false;
                const T *const from = static_cast<const T *>(cache) + off;
                const int64_t *const rows = tab + (g & 1) * kTok;
                uint8_t *const dst = sm + (uint32_t)st * kStage;
                // eight copies' row offsets are read before the first is used
                int m = lt / cpr, c = lt - m * cpr;
                while (m < kTok) {
                    int64_t o[kBatch];
                    uint32_t to[kBatch];
                    int cc[kBatch];
#pragma unroll
                    for (int i = 0; i < kBatch; ++i) {
                        o[i] = -2;
                        if (m < kTok) {
                            o[i] = rows[m];
                            to[i] = (uint32_t)(c >> 3) * kHalf + sw128_offset(m, c & 7);
                            cc[i] = c * 8;
                        }
                        m += dm;
                        c += dc;
                        if (c >= cpr) c -= cpr, ++m;
                    }
#pragma unroll
                    for (int i = 0; i < kBatch; ++i)
                        if (o[i] != -2)
                            cp_async16(dst + to[i], o[i] >= 0 ? from + o[i] + cc[i] : from, o[i] >= 0 ? 16u : 0u);
                }
                cp_async_arrive(&full[st]);
                advance();
                return true;
            };
            bool stop = injected(2);
            for (int i = 0; !stop; ++i) {
                if (!segment_there(i)) break;
                const Segment s = s_seg[i % kSegs];
                if (s.end == 0) break;
                for (int tile = s.tile; tile < s.end; ++tile, ++g) {
                    // where the tile's tokens are (elements from the cache's start)
                    for (int m = lt; m < kTok; m += kLoaders) {
                        int64_t off = -1;
                        const int j = tile * kTok + m;
                        if (j < s.total) {
                            const int pg = j / a.block_size;
                            const int32_t block = a.block_table[s.b * a.table_row + pg];
                            if (block >= 0 && block < a.num_blocks)
                                off = (int64_t)block * a.cache_block + (int64_t)(j - pg * a.block_size) * a.cache_token;
                            else
                                set_error(P.err, kErrBadIndex);
                        }
                        tab[(g & 1) * kTok + m] = off;
                    }
                    mbar_arrive(&tab_ready);  // (an mbarrier: its wait is bounded)
                    if (!await(&tab_ready, (uint32_t)g & 1, lost) ||
                        !copy_tile(a.k_cache, (int64_t)s.h * a.cache_head) ||
                        !copy_tile(a.v_cache, (int64_t)s.h * a.cache_head)) {
                        stop = true;
                        break;
                    }
                }
                if (lane == 0 && !stop) mbar_arrive(&seg_empty[i % kSegs]);
                __syncwarp();
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
        }
    } else if (warp == kMmaWarp) {
        // ---- MMA issuer ------------------------------------------------------
        const uint32_t idesc_s = idesc_f16(kBf16, kTok, S::kN) & ~(1u << 16);   // both K-major
        const uint32_t idesc_o = idesc_f16(kBf16, kTok, S::kN) | (1u << 15);  // both MN-major
        const uint32_t ring = smem_addr(sm), on = elect();
        // descriptors of the first stage and buffers; offsets add to them (bytes / 16)
        const uint64_t k_desc = sw128_desc(ring, 16, 1024), v_desc = sw128_desc(ring, kHalf, 1024);
        const uint64_t q_desc = sw128_desc(ring + S::kOffQ, 16, 1024);
        // 32-byte swizzle is layout 6, its 8-token groups are 256 bytes apart
        const uint64_t p_desc = S::kPRow == 128 ? sw128_desc(ring + S::kOffP, kHalf, 1024)
                                                : sw128_desc(ring + S::kOffP, kHalf, 256) ^ (4ull << 61);
        constexpr uint32_t p_step = 16 * S::kPRow >> 4;
        const bool wide = D > 64;
        int k_st = 0, v_st = 1 % S::kStages;  // ring stages of the next K and V
        uint32_t k_ph = 0, v_ph = 0;
        auto skip = [&](int &st, uint32_t &ph) {  // two operands on
            st += 2;
            if (st >= S::kStages) st -= S::kStages, ph ^= 1;
        };
        int ahead = -1, left = 0;             // segment of the next score product, its tiles not yet issued
        bool none = false, stop = false;      // no more of them; a wait ran out
        // Score product of tile g.  Its accumulator was last read for tile
        // g - 2, before that tile's P was complete.
        auto scores = [&](int g) {
            if (none) return;
            bool first = false;
            if (left == 0) {
                if (!segment_there(++ahead)) {
                    none = stop = true;
                    return;
                }
                const Segment &s = s_seg[ahead % kSegs];
                left = s.end - s.tile;
                if (s.end == 0) {
                    none = true;
                    return;
                }
                first = true;
            }
            const int qb = ahead % S::kQ;
            if ((first && !await(&q_full[qb], (uint32_t)(ahead / S::kQ) & 1, lost)) || !await(&full[k_st], k_ph, lost)) {
                none = stop = true;
                return;
            }
            --left;
            // cp.async (generic proxy) data -> tensor core (async proxy)
            if ((first && !P.q_box) || !P.box) fence_proxy_async();
            tc_fence_after();
            const uint64_t kd = k_desc + (uint32_t)k_st * (kStage >> 4);
            const uint64_t qd = q_desc + (uint32_t)qb * (S::kQBytes >> 4);
            const uint32_t d = tmem + (uint32_t)((g & 1) * S::kN);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) mma_on(on, d, kd + kk * 2, qd + kk * 2, idesc_s, kk != 0);
            if (wide) {
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    mma_on(on, d, kd + (kHalf >> 4) + kk * 2, qd + S::kN * 8u + kk * 2, idesc_s, 1);
            }
            commit_on(on, &empty[k_st]);  // also tells the softmax that the scores are there
            if (left == 0) commit_on(on, &q_empty[qb]);
            skip(k_st, k_ph);
        };
        scores(0);
        if (injected(3)) stop = true;
        int g = 0;
        for (int i = 0; !stop; ++i) {
            if (!segment_there(i)) break;
            const Segment &s = s_seg[i % kSegs];
            const int tiles = s.end - s.tile;
            if (s.end == 0) break;
            for (int t = 0; t < tiles; ++t, ++g) {
                // A tile ahead; but with one Q buffer the next segment's first scores
                // wait for its Q, and must not hold up this segment's last product.
                if (S::kQ > 1 || t + 1 < tiles) scores(g + 1);  // nothing at the end
                if (stop || !await(&full[v_st], v_ph, lost) || !await(&p_full, (uint32_t)g & 1, lost)) {
                    stop = true;
                    break;
                }
                if (!P.box) fence_proxy_async();
                tc_fence_after();
                const uint64_t vd = v_desc + (uint32_t)v_st * (kStage >> 4);
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                    mma_on(on, tmem + 2 * S::kN, vd + kk * 128, p_desc + kk * p_step, idesc_o, kk ? 1u : (uint32_t)t);
                commit_on(on, &empty[v_st]);
                commit_on(on, &pv_done);
                skip(v_st, v_ph);
                if (S::kQ == 1 && t + 1 == tiles) scores(g + 1);
            }
            if (lane == 0 && !stop) mbar_arrive(&seg_empty[i % kSegs]);
            __syncwarp();
        }
        // nothing of this kernel's is in flight when tensor memory is returned (a
        // wait with a limit of its own, whatever became of the others)
        commit_on(on, &drained);
        if (!mbar_wait(&drained, 0)) *lost = 1;
        __syncwarp();
    } else {
        // ---- softmax and output: thread = token, then = head column ------------
        const int wg = warp >> 2, tok = tid & 127, r0 = wg * S::kRows, d = tok;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t t_s = tmem + lanes + (uint32_t)r0, t_o = tmem + lanes + 2 * S::kN + (uint32_t)r0;
        // where this thread's 16-byte pieces of P go
        auto p_at = [&](int q) {
            return sm + S::kOffP + (S::kPRow == 128 ? (uint32_t)(wg >> 1) * kHalf + sw128_offset(tok, (wg & 1) * 4 + q)
                                                    : (uint32_t)(tok * 32 + ((q ^ (tok >> 2 & 1)) << 4)));
        };
        const float c = P.c;
        float l[S::kRows];
        int g = 0;              // tile
        // K of tile g is the ring's operand 2g, V is 2g + 1.  The commit that
        // frees K's stage is the signal that the scores are there: the stage can
        // be freed again only after this tile's P is complete.
        auto scores_done = [&](int g) {
            await(&empty[2 * g % S::kStages], (uint32_t)(2 * g / S::kStages) & 1, lost);
            tc_fence_after();
        };
        auto pv_finished = [&](int g) {
            await(&pv_done, (uint32_t)g & 1, lost);
            tc_fence_after();
        };
        // (one warp looks, so that all agree; once a wait has run out there are no more segments)
        auto look = [&](int seg) {
            const bool there = segment_there(seg);
            if (lane == 0) {
                if (there && !*lost) s_cur[seg & 1] = s_seg[seg % kSegs];
                else s_cur[seg & 1].end = 0;
            }
        };
        if (warp == 0) look(0);
        if (tid == 0) injected(4);
        for (int seg = 0;; ++seg) {
            named_sync<6, S::kSoft>();  // every thread is done with the last segment
            if (tid == 0 && seg > 0) mbar_arrive(&seg_empty[(seg - 1) % kSegs]);
            volatile Segment &cur = s_cur[seg & 1];
            const int prefix = cur.prefix, end = cur.end, first = cur.tile;
            if (end == 0) break;
            const int R = min(RT, cur.n * group - cur.rt * RT);  // rows in use
            const uint32_t *const see = reinterpret_cast<const uint32_t *>(sm + S::kOffSee) +
                                        cur.see * SGMV_TREE_MAX_NODES * S::kWords + wg;
            bool aux = false;  // the walk's tables for this segment are known to be there
#pragma unroll
            for (int r = 0; r < S::kRows; ++r) l[r] = 0.f;
            for (int tile = first; tile < end; ++tile, ++g) {
                const bool tree = (tile + 1) * P.tok > prefix, edge = tree || P.tok < kTok;
                if (tree) {
                    // while the scores are made: non-finite v of tree nodes, out of the
                    // tile and noted; what TMA brought from the last page past the end, zeroed
                    const int v0 = max(0, cur.prefix - tile * P.tok), v1 = min(P.tok, cur.total - tile * P.tok);
                    const int ve = P.box ? (v1 + P.box - 1) / P.box * P.box : v1;
                    const int pv = 2 * g + 1, cc = tid & 15;  // 16 lanes per token
                    await(&full[pv % S::kStages], (uint32_t)(pv / S::kStages) & 1, lost);
                    uint8_t *const vt = sm + (uint32_t)(pv % S::kStages) * kStage;
                    for (int m = v0 + (tid >> 4); m < ve && cc * 8 < D; m += S::kSoft / 16) {
                        uint8_t *const at = vt + (uint32_t)(cc >> 3) * kHalf + sw128_offset(m, cc & 7);
                        if (m >= v1) {
                            sts128(at, make_uint4(0, 0, 0, 0));
                            continue;
                        }
                        uint4 u = lds128(at);
                        uint32_t *const x = reinterpret_cast<uint32_t *>(&u);
                        bool any = false;
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            if (bad16<T>(x[q])) any = true, x[q] &= 0xffff0000u;
                            if (bad16<T>(x[q] >> 16)) any = true, x[q] &= 0xffffu;
                        }
                        if (any) {
                            s_poison = seg;
                            sts128(at, u);
                        }
                    }
                }
                scores_done(g);
                if (!aux && tree) {
                    await(&aux_full[seg % kSegs], (uint32_t)(seg / kSegs) & 1, lost);
                    aux = true;
                }
                const uint32_t ts = t_s + (uint32_t)((g & 1) * S::kN);
                // which rows see this token: all, none, or a node's
                const int j = tile * P.tok + tok;
                uint32_t vis = 0xffffffffu;
                if (edge && (tok >= P.tok || j >= prefix))
                    vis = tok < P.tok && j < cur.total ? see[(j - prefix) * S::kWords] : 0u;
                float s[S::kRows];
                // the weights, and their largest exponent; ref holds -ref
                float top;
                auto weights = [&]() {
                    tmem_load(ts, s);
#pragma unroll
                    for (int i = 0; i < S::kRows; i += 4) {
                        const uint4 u = lds128(&s_ref[r0 + i]);
                        fma_pair(s[i], s[i + 1], c, __uint_as_float(u.x), __uint_as_float(u.y));
                        fma_pair(s[i + 2], s[i + 3], c, __uint_as_float(u.z), __uint_as_float(u.w));
                    }
                    if (edge) {
#pragma unroll
                        for (int i = 0; i < S::kRows; ++i)
                            if (!(vis >> i & 1u)) s[i] = -INFINITY;
                    }
                    top = -INFINITY;
#pragma unroll
                    for (int i = 0; i < S::kRows; i += 2) {
                        top = fmaxf(top, fmaxf(s[i], s[i + 1]));
                        s[i] = exp2_approx(s[i]);
                        s[i + 1] = exp2_approx(s[i + 1]);
                    }
                };
                bool moved = tile == first;  // nothing to refer to yet
                if (!moved) {
                    weights();
                    moved = group_any(wg, top > kBias + kSlack);
                }
                if (moved) {
                    // new references: the larger of the old and this tile's maximum
                    tmem_load(ts, s);
#pragma unroll
                    for (int i = 0; i < S::kRows; ++i) s[i] = !edge || (vis >> i & 1u) ? s[i] * c : -INFINITY;
                    const int row = warp_rows<true>(s, lane);
                    s_red[warp & 3][r0 + row] = s[0];
                    group_bar(wg);
                    if (tok < S::kRows) {
                        const int r = r0 + tok;
                        float m = -INFINITY;
                        for (int w = 0; w < 4; ++w) {
                            const float x = s_red[w][r];
                            m = x > m || x != x ? x : m;
                        }
                        const float old = -s_ref[r];
                        float now = m - kBias;
                        now = now > old || now != now ? now : old;
                        s_fac[r] = old == kUnset ? 0.f : exp2_approx(old - now);
                        s_ref[r] = -now;
                    }
                    group_bar(wg);
                    if (tile != first) {
#pragma unroll
                        for (int r = 0; r < S::kRows; ++r) l[r] *= s_fac[r0 + r];
                        pv_finished(g - 1);
                        tmem_load(t_o, s);
#pragma unroll
                        for (int i = 0; i < S::kRows; ++i) s[i] *= s_fac[r0 + i];
                        tmem_store(t_o, s);
                    }
                    weights();
                }
                uint32_t p[S::kRows / 2];  // rounded to the tensor cores' operand type
#pragma unroll
                for (int i = 0; i < S::kRows; i += 2) {
                    add_pair(l[i], l[i + 1], s[i], s[i + 1]);
                    p[i / 2] = pack2<T>(s[i], s[i + 1]);
                }
                // the previous tile's P has been read
                if (g > 0) pv_finished(g - 1);
#pragma unroll
                for (int q = 0; q < S::kRows / 8; ++q)
                    sts128(p_at(q), make_uint4(p[4 * q], p[4 * q + 1], p[4 * q + 2], p[4 * q + 3]));
                fence_proxy_async();
                tc_fence_before();
                __syncwarp();  // one arrival per warp: a warp's own 32 would be served one by one
                if (lane == 0) mbar_arrive(&p_full);
            }
            if (!aux) await(&aux_full[seg % kSegs], (uint32_t)(seg / kSegs) & 1, lost);

            // ---- the segment's sums, then its rows -------------------------------
            {
                float v[S::kRows];
#pragma unroll
                for (int r = 0; r < S::kRows; ++r) v[r] = l[r];
                const int r = warp_rows<false>(v, lane);
                s_red[warp & 3][r0 + r] = v[0];
            }
            group_bar(wg);
            const bool whole = cur.whole != 0;
            const int slot = cur.slot;
            const int2 *const place = reinterpret_cast<const int2 *>(sm + S::kOffRow) + (seg % kSegs) * RT;
            // One warp does the factors, another the rest.  (A row that saw anything has
            // a weight of 2^kBias or more: the approximations of 1 / L and log2 L are at
            // their 2^-22 or so.)
            if ((tok & 31) < S::kRows && tok < 64) {
                const int r = r0 + (tok & 31);
                const float L = s_red[0][r] + s_red[1][r] + s_red[2][r] + s_red[3][r];
                const int2 to = place[r < R ? r : 0];
                const bool none = to.x < 0 || L == 0.f;
                if (tok < 32) {
                    s_fac[r] = none ? 0.f : __fdividef(1.f, L);
                } else {
                    const float ref = -s_ref[r];
                    if (!whole)
                        *reinterpret_cast<float2 *>(P.ml + ((int64_t)slot * RT + r) * 2) = make_float2(ref, L);
                    else if (a.lse && r < R && !*lost)
                        a.lse[(int64_t)(to.x < 0 ? ~to.x : to.x) * a.Hq + to.y] =
                            none ? -INFINITY : (ref + __log2f(L)) * 0.693147180559945309f;
                    s_ref[r] = -kUnset;
                }
            }
            pv_finished(g - 1);
            group_bar(wg);
            {
                const bool poison = *(volatile int *)&s_poison == seg, ok = !*lost;
                float v[S::kRows];
                tmem_load(t_o, v);
                if (poison && d < D) {
                    for (int jn = max(0, first * P.tok - prefix); jn < min(cur.n, end * P.tok - prefix); ++jn) {
                        const int j = prefix + jn, pg = j / a.block_size;
                        const int32_t block = a.block_table[cur.b * a.table_row + pg];
                        if (block < 0 || block >= a.num_blocks) continue;
                        const T x = static_cast<const T *>(a.v_cache)[(int64_t)block * a.cache_block +
                                                                     (int64_t)(j - pg * a.block_size) * a.cache_token +
                                                                     (int64_t)cur.h * a.cache_head + d];
                        if (!bad16<T>(*reinterpret_cast<const unsigned short *>(&x))) continue;
                        const uint32_t bits = see[jn * S::kWords];
#pragma unroll
                        for (int i = 0; i < S::kRows; ++i)
                            if (bits >> i & 1u) v[i] += to_f<T>(x);
                    }
                }
                if (whole) {
                    // through the idle P buffer, a row of 256 bytes each, to whole
                    // vectors (and little code: this path is cold in the instruction cache)
                    uint8_t *const rows = sm + S::kOffP + r0 * 256;
#pragma unroll
                    for (int i = 0; i < S::kRows; i += 2) {
                        const uint32_t two = pack2<T>(v[i] * s_fac[r0 + i], v[i + 1] * s_fac[r0 + i + 1]);
                        sts16(rows + i * 256 + d * 2, (uint16_t)two);
                        sts16(rows + (i + 1) * 256 + d * 2, (uint16_t)(two >> 16));
                    }
                    group_bar(wg);
                    const int used = min(S::kRows, R - r0);
#pragma unroll 1
                    for (int m = tok >> 4; m < used; m += 8) {  // 16 lanes per row
                        const int2 to = place[r0 + m];
                        T *const out = static_cast<T *>(a.out) + (int64_t)(to.x < 0 ? ~to.x : to.x) * a.out_token +
                                       (int64_t)to.y * a.out_head;
                        const int col = (tok & 15) * 8;
                        if (col < D && ok)  // (no weights at all: zeros, whatever v holds)
                            *reinterpret_cast<uint4 *>(out + col) =
                                s_fac[r0 + m] == 0.f ? make_uint4(0, 0, 0, 0) : lds128(rows + m * 256 + col * 2);
                    }
                } else {
                    float *const part = P.part + ((int64_t)slot * RT + r0) * 128 + d;
#pragma unroll
                    for (int i = 0; i < S::kRows; ++i)
                        if (r0 + i < R) part[i * 128] = v[i];
                }
            }
            if (warp == 0) look(seg + 1);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) tmem_dealloc(tmem, S::kTmem);
    if (*lost) {
        if (tid == 0) set_error(P.err, kErrTimeout);
        // the join leaves items with parts of this share alone
        for (int r = tid; r < 2 * RT; r += S::kThreads)
            *reinterpret_cast<float2 *>(P.ml + ((int64_t)blockIdx.x * 2 * RT + r) * 2) = make_float2(kUnset, -1.f);
        // copies under way land while this shared memory is the CTA's
        if (P.q_box && warp == kWalkWarp)
            for (int i = max(0, issued - S::kQ); i < issued; ++i)
                if (!mbar_wait(&q_full[i % S::kQ], (uint32_t)(i / S::kQ) & 1)) break;
        if (P.box && warp > kWalkWarp)
            for (int i = max(0, issued - S::kStages); i < issued; ++i)
                if (!mbar_wait(&full[i % S::kStages], (uint32_t)(i / S::kStages) & 1)) break;
    }
}

// Joins the parts of cut items: a warp per (share, row), the item being the one
// that begins in the share; a lane owns four head columns.  A chain of loads: the
// cut, then references, sums and the first kJoinBatch parts of O at once, then the rest by
// as many.  (One part after the other, each against the running maximum, 8 items of
// 19 parts and 32 rows took 10 us: 5 now.  With 3 parts at a time and six CTAs per SM, for
// large row tiles, whose parts are few, 8 trees of 8 nodes took 114 us against 111.)
constexpr int kJoinThreads = 256;
constexpr int kJoinBatch = 8;
template <typename T, int RT>
__global__ void __launch_bounds__(kJoinThreads, 4) sgmv_tree_join_kernel(const __grid_constant__ MmaParams P) {
    const sgmv_tree_attention_args &a = P.a;
    pdl_wait();
    pdl_trigger();
    const int warps = gridDim.x * (kJoinThreads / 32), lane = threadIdx.x & 31;
    const int shares = *P.shares;
    for (int u = blockIdx.x * (kJoinThreads / 32) + threadIdx.x / 32; u < P.ctas * RT; u += warps) {
        const int id = u / RT, r = u % RT;
        const Cut cut = P.cut[id];
        if (id >= shares) break;
        if (cut.parts == 0 || cut.rt * RT + r >= cut.n * P.group) continue;
        const int2 to = row_place(P, cut.t0, cut.h, cut.rt * RT + r);
        auto row_of = [&](int k) { return (int64_t)(2 * (id + k) + (k == 0)) * RT + r; };
        float M = kUnset, L = 0.f;
        bool gone = false;  // a part's waits ran out: no output
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k0 = 0; k0 < cut.parts; k0 += 32) {  // a lane per part
            const int n = min(32, cut.parts - k0);
            float2 ml = make_float2(kUnset, 0.f);
            if (lane < n) ml = *reinterpret_cast<const float2 *>(P.ml + row_of(k0 + lane) * 2);
            gone |= __any_sync(0xffffffffu, ml.y < 0.f);
            float4 x[kJoinBatch];
            auto fetch = [&](int k) {
#pragma unroll
                for (int i = 0; i < kJoinBatch; ++i)
                    if (k + i < n) x[i] = reinterpret_cast<const float4 *>(P.part + row_of(k0 + k + i) * 128)[lane];
            };
            fetch(0);
            float m = fmaxf(M, ml.x);
            for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
            const float was = exp2_approx(M - m);
            M = m;
            // -1: the row saw nothing there
            const float w = ml.x == kUnset ? -1.f : exp2_approx(ml.x - m);
            float l = ml.x == kUnset ? 0.f : ml.y * w;
            for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
            L = L * was + l;
            o.x *= was, o.y *= was, o.z *= was, o.w *= was;
            for (int k = 0; k < n; k += kJoinBatch) {
                if (k) fetch(k);
#pragma unroll
                for (int i = 0; i < kJoinBatch; ++i) {
                    const float f = __shfl_sync(0xffffffffu, w, (k + i) & 31);
                    if (k + i >= n || f == -1.f) continue;
                    o.x += x[i].x * f;
                    o.y += x[i].y * f;
                    o.z += x[i].z * f;
                    o.w += x[i].w * f;
                }
            }
        }
        if (gone) continue;
        const int64_t t = to.x < 0 ? ~to.x : to.x;
        const bool none = to.x < 0 || L == 0.f;
        const float f = none ? 0.f : 1.f / L;
        if (lane * 4 < a.D) {
            T v[4] = {from_f<T>(none ? 0.f : o.x * f), from_f<T>(none ? 0.f : o.y * f),
                      from_f<T>(none ? 0.f : o.z * f), from_f<T>(none ? 0.f : o.w * f)};
            *reinterpret_cast<uint2 *>(static_cast<T *>(a.out) + t * a.out_token + (int64_t)to.y * a.out_head + lane * 4) =
                *reinterpret_cast<const uint2 *>(v);
        }
        if (a.lse && lane == 0)
            a.lse[t * a.Hq + to.y] = none ? -INFINITY : (M + log2f(L)) * 0.693147180559945309f;
    }
}

template <typename T, int RT>
int launch(const MmaParams &p, int ctas, cudaStream_t stream) {
    static_assert((Shape<RT>::kBytes + 4096) * Shape<RT>::kPerSm <= 227 * 1024, "shared memory");
    const cudaError_t e = cudaFuncSetAttribute(sgmv_tree_mma_kernel<T, RT>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)Shape<RT>::kBytes);
    if (e != cudaSuccess) return (int)e;
    const int r = spec_launch(sgmv_tree_mma_kernel<T, RT>, dim3((unsigned)ctas), Shape<RT>::kThreads,
                              Shape<RT>::kBytes, 1, stream, p);
    if (r != (int)cudaSuccess) return r;
    const int join = std::min(8 * kMaxSms, (ctas * RT * 32 + kJoinThreads - 1) / kJoinThreads);
    return spec_launch(sgmv_tree_join_kernel<T, RT>, dim3((unsigned)join), kJoinThreads, 0, 1, stream, p);
}

// Rows per tile: what a sequence of average length fills.  8 rows are half the
// softmax's work of 16 (512 sequences of 100 tokens, 32 heads on 8: 62 us against 74; 256 of
// 512 tokens: 76 against 89), and are taken where there are no more rows than
// sequences.  Then a sequence has one row, or others have none; K and V of one
// that has more all the same are read for every 8 of its rows.  Batches far from their mean
// (127 decode rows over up to 4096 tokens, 32 heads on 8, and one chunk of 256 rows over 2200:
// 237 us, row tiles of 16) take about what their parts take alone (192 and 50).
int row_tile(int32_t T, int32_t B, int32_t group) {
    if (T <= B && group <= 8) return 8;
    const int64_t rows = ((int64_t)T + B - 1) / B * group;
    return rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128;
}

constexpr size_t kHeadBytes = 256;

// CTAs, and so shares, at most.
int max_ctas(int rt) { return kMaxSms * (rt <= 16 ? Shape<16>::kPerSm : 1); }

}  // namespace

// For the batch and every smaller one: fewer sequences or rows may make higher row
// tiles, up to those of a single sequence with all the rows.
size_t tree_mma_workspace(int32_t T, int32_t group) {
    size_t most = 0;
    for (int rt = 8, last = row_tile(T, 1, group); rt <= last; rt *= 2)
        most = std::max(most, kHeadBytes + (size_t)max_ctas(rt) * (sizeof(Cut) + 2u * (size_t)rt * 130u * 4u));
    return most;
}

int tree_mma_launch(const sgmv_tree_attention_args &a, int nsm, int *err, cudaStream_t stream) {
    const int group = a.Hq / a.Hkv, rt = row_tile(a.T, a.B, group);
    const int ctas = std::min(std::max(1, nsm) * (max_ctas(rt) / kMaxSms), max_ctas(rt));
    MmaParams p;
    p.a = a;
    p.c = a.scale * 1.4426950408889634f;
    p.group = group;
    p.ctas = ctas;
    p.shares = static_cast<int *>(a.workspace);
    p.cut = reinterpret_cast<Cut *>(static_cast<uint8_t *>(a.workspace) + kHeadBytes);
    p.ml = reinterpret_cast<float *>(p.cut + max_ctas(rt));
    p.part = p.ml + max_ctas(rt) * 2 * rt * 2;
    p.err = err;
    p.inject = injected_timeout();
    const bool bf16 = a.dtype == SGMV_BF16;
    // Boxes are as high as pages allow, for TMA's cost here is per box: at pages of
    // 24 tokens, boxes of 8 filling every tile took 115 us, boxes of 24 and tiles of
    // 120 tokens 109 us (128 sequences of up to 2100 tokens, 4 heads of 80).
    p.tok = tree_tile(a.block_size);
    p.box = p.tok < kTok ? a.block_size : std::gcd(a.block_size, kTok);
    if (p.box >= 8) {
        const cuuint64_t dims[4] = {(cuuint64_t)a.D, (cuuint64_t)a.block_size, (cuuint64_t)a.Hkv,
                                    (cuuint64_t)a.num_blocks};
        const cuuint64_t strides[3] = {(cuuint64_t)a.cache_token * 2u, (cuuint64_t)a.cache_head * 2u,
                                       (cuuint64_t)a.cache_block * 2u};
        const cuuint32_t box[4] = {64, (cuuint32_t)p.box, 1, 1};
        // What L2 fetches around a row of a box is this head's only if the rows of
        // a head are contiguous or as wide; else it is another CTA's (32 x 4 rows over up
        // to 4096 tokens, 32 heads side by side: of 64 columns 142 us with 256 bytes,
        // 122 with 128; of 96 columns 220 with 256, 167 with 64)
        const int row = a.D * 2;
        const CUtensorMapL2promotion fetch =
            a.cache_token == a.D || row % 256 == 0 ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B
            : row % 128 == 0                       ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B
            : row % 64 == 0                        ? CU_TENSOR_MAP_L2_PROMOTION_L2_64B
                                                   : CU_TENSOR_MAP_L2_PROMOTION_NONE;
        if (!tmap_encode(&p.map_k, bf16, 4, a.k_cache, dims, strides, box, true, fetch) ||
            !tmap_encode(&p.map_v, bf16, 4, a.v_cache, dims, strides, box, true, fetch))
            p.box = 0, p.tok = kTok;  // strides that a tensor map cannot hold
    } else {
        p.box = 0;
    }
    p.q_box = 0;
    if (rt % group == 0) {
        const cuuint64_t dims[3] = {(cuuint64_t)a.D, (cuuint64_t)a.Hq, (cuuint64_t)a.T};
        const cuuint64_t strides[2] = {(cuuint64_t)a.q_head * 2u, (cuuint64_t)a.q_token * 2u};
        const cuuint32_t box[3] = {64, (cuuint32_t)group, (cuuint32_t)(rt / group)};
        p.q_box = tmap_encode(&p.map_q, bf16, 3, a.q, dims, strides, box, true);
    }
    const bool h = a.dtype == SGMV_F16;
    using B16 = __nv_bfloat16;
    switch (rt) {
        case 8: return h ? launch<__half, 8>(p, ctas, stream) : launch<B16, 8>(p, ctas, stream);
        case 16: return h ? launch<__half, 16>(p, ctas, stream) : launch<B16, 16>(p, ctas, stream);
        case 32: return h ? launch<__half, 32>(p, ctas, stream) : launch<B16, 32>(p, ctas, stream);
        case 64: return h ? launch<__half, 64>(p, ctas, stream) : launch<B16, 64>(p, ctas, stream);
        default: return h ? launch<__half, 128>(p, ctas, stream) : launch<B16, 128>(p, ctas, stream);
    }
}

}  // namespace sgmv
