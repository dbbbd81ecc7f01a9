// sgmv_tree_mma.cu -- tree attention on the tensor cores, for heads of up to
// 128 columns.
//
// The rows of one sequence that share a KV head (nodes x query heads of the
// group) are cut into row tiles of RT = 16, 32, 64 or 128, the tokens into
// tiles of 128.  Both products run transposed, so that the long axis (tokens,
// then head columns) fills the 128 lanes of the tensor cores however few rows
// there are:
//
//   S^T [tokens x RT] = K . Q^T          A = K tile (K-major),  B = Q rows
//   O^T [columns x RT] += V^T . P^T      A = V tile (M-major),  B = P
//
// with S^T and O^T in tensor memory.  A softmax thread owns one token: it
// reads its RT scores, makes p = 2^(c s - ref[row]) and writes them as one row
// of P.  ref[row] is the row's running maximum, moved only when a score
// exceeds it by more than 2^kSlack (then O^T and the sums are scaled), so an
// ordinary tile needs one vote and no reduction over tokens.
//
// Decomposition: the (sequence, head, row tile) items, each of ceil(length /
// 128) token tiles, form one line that is cut into equal shares, one per CTA
// (one CTA per SM).  A share that covers an item writes its output; items cut
// across shares leave unnormalised O, sum and maximum in the workspace, and
// the CTA that finishes last joins them in share order.
//
// Warps: 4 (RT <= 64) or 8 softmax warps, then one that issues the MMAs, then
// three that bring K, V (a ring of 32 KB stages) and Q in with cp.async, 16
// bytes per lane, through the block table: any page size, and tokens past the
// end become zeros.  The MMA warp runs one score product ahead of the softmax.
//
// Values of rows a query does not see never reach it: scores are masked after
// the product, and non-finite v of tree nodes are taken out of the staged
// tile (a masked weight of 0 times infinity would be NaN) and added back for
// the rows that do see them.
#include <math.h>

#include <numeric>
#include <type_traits>

#include "sgmv_device.cuh"
#include "sgmv_internal.h"
#include "sgmv_spec.h"
#include "sgmv_tcgen05.cuh"

namespace sgmv {
namespace {

constexpr int kTok = 128;                // tokens per tile
constexpr uint32_t kHalf = kTok * 128u;  // bytes of 64 columns of a tile
constexpr uint32_t kStage = 2 * kHalf;   // a K or V tile, 128 columns
constexpr int kLoaders = 96;             // loading threads
constexpr float kUnset = -3e38f;         // ref of a row that has seen nothing
constexpr float kBias = 7.f;             // weights are 2^(kBias + score - ref) ...
constexpr float kSlack = 8.f;            // ... <= 2^(kBias + kSlack), finite in f16
constexpr int kMaxCtas = 152;

template <int RT> struct Shape {
    static constexpr int kGroups = RT > 32 ? RT / 32 : 1;  // softmax warpgroups
    static constexpr int kRows = RT / kGroups;            // rows per warpgroup
    static constexpr int kSoft = 128 * kGroups;           // softmax threads
    static constexpr int kThreads = kSoft + 32 + kLoaders;
    static constexpr int kQ = RT > 64 ? 1 : 2;            // Q buffers
    static constexpr int kStages = RT > 64 ? 4 : 5;
    static constexpr int kWords = RT < 32 ? 1 : RT / 32;  // words of one bit per row
    static constexpr uint32_t kQBytes = RT * 256u;
    static constexpr uint32_t kPBytes = (RT > 64 ? 2 : 1) * kHalf;
    static constexpr uint32_t kTmem = RT <= 16 ? 64 : RT <= 32 ? 128 : RT <= 64 ? 256 : 512;
    // dynamic shared memory
    static constexpr uint32_t kOffQ = kStages * kStage;
    static constexpr uint32_t kOffP = kOffQ + kQ * kQBytes;
    static constexpr uint32_t kOffTab = kOffP + kPBytes;                 // row offsets of 4 tiles
    static constexpr uint32_t kOffSee = kOffTab + 4u * kTok * 8u;        // who sees each node
    static constexpr uint32_t kOffRow = kOffSee + SGMV_TREE_MAX_NODES * kWords * 4u;  // rows' outputs
    static constexpr uint32_t kBytes = kOffRow + RT * 8u + 1024u;        // + alignment
};

struct MmaParams {
    // the caches as [page][head][token][D], boxes of `box` tokens by 64 columns
    CUtensorMap map_k, map_v;
    int32_t box;      // tokens per box; 0: cp.async
    int32_t tok;      // tokens per tile: 128, or the boxes that fit in 128
    sgmv_tree_attention_args a;
    float c;          // scale * log2(e)
    int32_t group;    // query heads per KV head
    int *count;       // [CTA]: partial items finished, by their first CTA
    float *ml;        // [CTA][2][RT][2]: reference and sum of partial items
    float *part;      // [CTA][2][RT][128]
    int *err;
};

// A place in the line of work, advanced segment by segment (a segment: the
// tiles of one item inside this CTA's share).
template <int RT> struct Cursor {
    int b, t0, n, prefix, total, tiles, nrt;
    int64_t base, w, w1;  // first tile of sequence b; next tile; end of the share
    uint32_t items;
    // the current segment
    int h, rt, tile, end, item_tiles;
    int64_t item0;

    __device__ __forceinline__ static bool sequence(const MmaParams &P, int b, int &t0, int &n,
                                                    int &prefix) {
        const sgmv_tree_attention_args &a = P.a;
        t0 = a.tree_ptr[b];
        n = a.tree_ptr[b + 1] - t0;
        prefix = a.prefix_lens[b];
        return t0 >= 0 && n >= 0 && n <= SGMV_TREE_MAX_NODES && (int64_t)t0 + n <= a.T && prefix >= 0 &&
               (int64_t)prefix + n <= (int64_t)a.max_blocks * a.block_size;
    }
    __device__ __forceinline__ static uint32_t work(const MmaParams &P, int b) {
        int t0, n, prefix;
        if (!sequence(P, b, t0, n, prefix) || n == 0) return 0;
        return (uint32_t)((prefix + n + P.tok - 1) / P.tok) * (uint32_t)((n * P.group + RT - 1) / RT) *
               (uint32_t)P.a.Hkv;
    }
    __device__ __forceinline__ void enter(const MmaParams &P) {
        sequence(P, b, t0, n, prefix);
        total = prefix + n;
        tiles = (total + P.tok - 1) / P.tok;
        nrt = (n * P.group + RT - 1) / RT;
        items = (uint32_t)P.a.Hkv * (uint32_t)nrt;
    }
    __device__ __forceinline__ void start(const MmaParams &P, int b_, int64_t base_, int64_t w_,
                                          int64_t w1_) {
        b = b_;
        base = base_;
        w = w_;
        w1 = w1_;
        enter(P);
    }
    // the segment at w; false at the end of the share
    __device__ __forceinline__ bool next(const MmaParams &P) {
        if (w >= w1) return false;
        while (w >= base + (int64_t)items * tiles) {
            base += (int64_t)items * tiles;
            do ++b;
            while (b < P.a.B - 1 && work(P, b) == 0);
            enter(P);
        }
        const uint32_t rel = (uint32_t)(w - base), item = rel / (uint32_t)tiles;
        h = (int)(item / (uint32_t)nrt);
        rt = (int)(item - (uint32_t)h * (uint32_t)nrt);
        tile = (int)(rel - item * (uint32_t)tiles);
        item_tiles = tiles;
        item0 = base + (int64_t)item * tiles;
        const int64_t left = w1 - w;
        end = left < tiles - tile ? tile + (int)left : tiles;
        w += end - tile;
        return true;
    }
};

// Bounded wait of a whole warp.  When one runs out (or another role's did),
// `lost` is set and every later wait returns at once: the roles then run
// through their remaining steps on whatever the buffers hold, so that barriers
// still meet and the kernel ends, and write no output.
__device__ __forceinline__ void await(uint64_t *bar, uint32_t parity, volatile int *lost) {
    if (!mbar_try_wait(bar, parity)) {
        const uint64_t t0 = global_ns();
        for (uint32_t i = 0; !mbar_try_wait(bar, parity); ++i) {
            if (*lost || i >= kMaxPolls || global_ns() - t0 > kWaitLimitNs) {
                *lost = 1;
                break;
            }
        }
    }
    __syncwarp();
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
// floats as integers of the same order
__device__ __forceinline__ int ordered(float f) {
    const int i = __float_as_int(f);
    return i ^ ((i >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float unordered(int i) {
    return __int_as_float(i ^ ((i >> 31) & 0x7fffffff));
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
template <int N> __device__ __forceinline__ void tmem_load(uint32_t addr, float (&v)[N]) {
    if constexpr (N == 32)
        tmem_ld32(addr, v);
    else
        tmem_ld16(addr, v);
}
template <int N> __device__ __forceinline__ void tmem_store(uint32_t addr, const float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N; i += 16)
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
// v[i], i < N: row i's partial of every lane.  Afterwards each lane holds the
// sums over the warp of N / 32 (at least 1) rows, the first of them returned.
template <int N> __device__ __forceinline__ int warp_sums(float (&v)[N], int lane) {
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
                    v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
                }
        } else {
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
        }
    }
    return row;
}

// Non-finite 16-bit values: all ones in the exponent.
template <typename T> __device__ __forceinline__ bool bad16(uint32_t h) {
    constexpr uint32_t e = std::is_same<T, __half>::value ? 0x7C00u : 0x7F80u;
    return (h & e) == e;
}

template <typename T, int RT>
__global__ void __launch_bounds__(Shape<RT>::kThreads, 1)
    sgmv_tree_mma_kernel(const __grid_constant__ MmaParams P) {
    using S = Shape<RT>;
    constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
    const sgmv_tree_attention_args &a = P.a;
    extern __shared__ __align__(1024) uint8_t dsm[];
    __shared__ __align__(8) uint64_t full[S::kStages], empty[S::kStages], q_full[S::kQ], q_empty[S::kQ];
    __shared__ __align__(8) uint64_t p_full, drained;
    __shared__ uint32_t s_tmem;
    __shared__ int s_lost, s_poison, s_last;
    __shared__ int s_b;
    __shared__ int64_t s_base, s_sum[32];
    __shared__ __align__(16) float s_ref[RT], s_fac[RT];
    __shared__ float s_red[4][RT];
    uint8_t *const sm = align1024(dsm);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    constexpr int kWarps = S::kThreads / 32, kMmaWarp = S::kSoft / 32;

    if (warp == kMmaWarp) {
        if (lane == 0) {
            for (int i = 0; i < S::kStages; ++i)
                mbar_init(&full[i], P.box ? kLoaders / 32 : kLoaders), mbar_init(&empty[i], 1);
            for (int i = 0; i < S::kQ; ++i) mbar_init(&q_full[i], kLoaders), mbar_init(&q_empty[i], 1);
            mbar_init(&p_full, S::kSoft);
            mbar_init(&drained, 1);
            mbar_init_fence();
            s_lost = 0;
            s_poison = -1;
        }
        __syncwarp();
        tmem_alloc(&s_tmem, S::kTmem);
    }
    for (int i = tid; i < RT; i += S::kThreads) s_ref[i] = kUnset;
    // columns past D that the products read are zero: in Q, and in K where TMA
    // does not fill them; so are the rows past a short tile
    if (P.tok < kTok)
        for (uint32_t i = tid * 16u; i < S::kOffQ; i += S::kThreads * 16u)
            sts128(sm + i, make_uint4(0, 0, 0, 0));
    if (a.D % 64 != 0)
        for (uint32_t i = (P.box ? S::kOffQ : 0u) + tid * 16u; i < S::kOffP; i += S::kThreads * 16u)
            sts128(sm + i, make_uint4(0, 0, 0, 0));
    fence_proxy_async();
    pdl_wait();
    pdl_trigger();

    // ---- this CTA's share of the line -------------------------------------
    using Cur = Cursor<RT>;
    int64_t sum = 0;
    for (int b = tid; b < a.B; b += S::kThreads) {
        int t0, n, prefix;
        if (!Cur::sequence(P, b, t0, n, prefix) && blockIdx.x == 0) set_error(P.err, kErrBadSegments);
        sum += Cur::work(P, b);
    }
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) s_sum[warp] = sum;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    int64_t W = 0;
    for (int i = 0; i < kWarps; ++i) W += s_sum[i];
    const int64_t share = (W + gridDim.x - 1) / gridDim.x;
    const int64_t w0 = share * blockIdx.x, w1 = w0 + share < W ? w0 + share : W;
    const uint32_t tmem = s_tmem;
    if (w0 >= w1) {
        __syncthreads();
        if (warp == kMmaWarp) tmem_dealloc(tmem, S::kTmem);
        return;
    }
    {
        int64_t base = 0;
        for (int b0 = 0; b0 < a.B; b0 += S::kThreads) {  // the sequence that holds tile w0
            const int b = b0 + tid;
            const int64_t own = b < a.B ? Cur::work(P, b) : 0;
            int64_t run = own;
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t up = __shfl_up_sync(0xffffffffu, run, o);
                if (lane >= o) run += up;
            }
            __syncthreads();
            if (lane == 31) s_sum[warp] = run;
            __syncthreads();
            int64_t before = base, all = 0;
            for (int i = 0; i < kWarps; ++i) {
                if (i < warp) before += s_sum[i];
                all += s_sum[i];
            }
            if (before + run - own <= w0 && w0 < before + run) s_b = b, s_base = before + run - own;
            base += all;
            if (w0 < base) break;
        }
        __syncthreads();
    }
    Cur cur;
    cur.start(P, s_b, s_base, w0, w1);
    volatile int *const lost = &s_lost;
    const int D = a.D, group = P.group;

    if (warp > kMmaWarp) {
        // ---- loaders: ring order K0, K1, V0, K2, V1, ..., V(last) -----------
        const int lt = tid - S::kSoft - 32;
        const int cpr = D / 8;                     // 16-byte chunks per row
        const int dm = kLoaders / cpr, dc = kLoaders - dm * cpr;
        constexpr int kBatch = 8, kOwn = (kTok + kLoaders - 1) / kLoaders;
        int64_t *const tab = reinterpret_cast<int64_t *>(sm + S::kOffTab);
        const int halves = D > 64 ? 2 : 1;
        int pos = 0, g = 0, seg = 0;               // ring position, tile, segment
        // the queries of segment seg's row tile, by `count` threads
        auto load_q = [&](int i0, int count) {
            const int qb = seg % S::kQ;
            if (seg >= S::kQ) await(&q_empty[qb], (uint32_t)(seg / S::kQ - 1) & 1, lost);
            uint8_t *const dst = sm + S::kOffQ + (uint32_t)qb * S::kQBytes;
            const int R = cur.n * group;
            for (int i = i0; i < RT * cpr; i += count) {
                const int m = i / cpr, c = i - m * cpr, r = cur.rt * RT + m;
                const int node = r / group, hq = cur.h * group + (r - node * group);
                const bool in = r < R;
                const T *src = static_cast<const T *>(a.q) +
                               (in ? (int64_t)(cur.t0 + node) * a.q_token + (int64_t)hq * a.q_head + c * 8 : 0);
                cp_async16(dst + (uint32_t)(c >> 3) * (RT * 128u) + sw128_offset(m, c & 7), src, in ? 16u : 0u);
            }
            cp_async_arrive(&q_full[qb]);
            ++seg;
        };
        if (P.box) {
            // TMA: a box (tokens x 64 columns) per lane, dealt to the three warps
            const int box = P.box, nbox = P.tok / box, op = lane * (kLoaders / 32) + lt / 32;
            const int mine = op % nbox, half = op / nbox;
            const bool busy = half < halves;
            const uint32_t bytes = (uint32_t)__popc(__ballot_sync(0xffffffffu, busy)) * (uint32_t)box * 128u;
            const uint32_t at = (uint32_t)half * kHalf + (uint32_t)(mine * box) * 128u;
            Cur peek = cur;   // the tile whose page is looked up next
            int peek_tile = 0, peek_end = 0;
            int32_t next_page = 0;
            int next_in = 0;
            auto look = [&]() {
                if (peek_tile == peek_end) {
                    if (!peek.next(P)) return;
                    peek_tile = peek.tile;
                    peek_end = peek.end;
                }
                const int j = peek_tile * P.tok + mine * box;
                next_in = -1;
                if (j < peek.total) {
                    const int pg = j / a.block_size;
                    next_in = j - pg * a.block_size;
                    next_page = a.block_table[peek.b * a.table_row + pg];
                }
                ++peek_tile;
            };
            auto copy_boxes = [&](const CUtensorMap *map, int32_t page, int in, int head) {
                const int st = pos % S::kStages;
                if (pos >= S::kStages) await(&empty[st], (uint32_t)(pos / S::kStages - 1) & 1, lost);
                if (lane == 0) mbar_arrive_expect_tx(&full[st], bytes);
                __syncwarp();
                if (busy) tma_load_4d(sm + (uint32_t)st * kStage + at, map, half * 64, in, head, page, &full[st]);
                ++pos;
            };
            int32_t page = 0, old_page = 0;
            int in = 0, old_in = 0, old_h = 0;
            look();
            while (cur.next(P)) {
                load_q(lt, kLoaders);
                for (int tile = cur.tile; tile < cur.end; ++tile, ++g) {
                    // boxes past the end, and pages out of range, read as zeros
                    page = next_page;
                    in = next_in;
                    if (in < 0 || page < 0 || page >= a.num_blocks) {
                        if (in >= 0) set_error(P.err, kErrBadIndex);
                        page = a.num_blocks;
                        in = 0;
                    }
                    look();
                    copy_boxes(&P.map_k, page, in, cur.h);
                    if (g > 0) copy_boxes(&P.map_v, old_page, old_in, old_h);
                    old_page = page;
                    old_in = in;
                    old_h = cur.h;
                }
            }
            copy_boxes(&P.map_v, old_page, old_in, old_h);
            asm volatile("cp.async.wait_all;" ::: "memory");
        } else {
        int64_t head_off = 0, prev_head = 0;
        auto copy_tile = [&](const void *cache, int64_t off, int tile) {
            const int st = pos % S::kStages;
            if (pos >= S::kStages) await(&empty[st], (uint32_t)(pos / S::kStages - 1) & 1, lost);
            const T *const base = static_cast<const T *>(cache) + off;
            const int64_t *const rows = tab + (tile & 3) * kTok;
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
                        cp_async16(dst + to[i], o[i] >= 0 ? base + o[i] + cc[i] : base, o[i] >= 0 ? 16u : 0u);
            }
            cp_async_arrive(&full[st]);
            ++pos;
        };
        // the tile after the current one: its pages are looked up while the
        // current one's copies are issued
        Cur peek = cur;
        int peek_tile = 0, peek_end = 0;
        int32_t block[kOwn];
        int in_page[kOwn];
        auto look = [&]() {
            if (peek_tile == peek_end) {
                if (!peek.next(P)) return;
                peek_tile = peek.tile;
                peek_end = peek.end;
            }
#pragma unroll
            for (int e = 0; e < kOwn; ++e) {
                const int m = lt + e * kLoaders, j = peek_tile * kTok + m;
                in_page[e] = -1;
                if (m < kTok && j < peek.total) {
                    const int pg = j / a.block_size;
                    in_page[e] = j - pg * a.block_size;
                    block[e] = a.block_table[peek.b * a.table_row + pg];
                }
            }
            ++peek_tile;
        };
        look();
        while (cur.next(P)) {
            prev_head = head_off;
            head_off = (int64_t)cur.h * a.cache_head;
            load_q(lt, kLoaders);
            for (int tile = cur.tile; tile < cur.end; ++tile, ++g) {
                // where the tile's tokens are (elements from the cache's start)
#pragma unroll
                for (int e = 0; e < kOwn; ++e) {
                    const int m = lt + e * kLoaders;
                    const bool in = in_page[e] >= 0, good = in && block[e] >= 0 && block[e] < a.num_blocks;
                    if (in && !good) set_error(P.err, kErrBadIndex);
                    if (m < kTok)
                        tab[(g & 3) * kTok + m] =
                            good ? (int64_t)block[e] * a.cache_block + (int64_t)in_page[e] * a.cache_token : -1;
                }
                named_sync<1, kLoaders>();
                look();
                copy_tile(a.k_cache, head_off, g);
                if (g > 0) copy_tile(a.v_cache, tile == cur.tile ? prev_head : head_off, g - 1);
            }
        }
        copy_tile(a.v_cache, head_off, g - 1);
        asm volatile("cp.async.wait_all;" ::: "memory");
        }
    } else if (warp == kMmaWarp) {
        // ---- MMA issuer ------------------------------------------------------
        const uint32_t idesc_s = idesc_f16(kBf16, kTok, RT) & ~(1u << 16);   // both K-major
        const uint32_t idesc_o = idesc_f16(kBf16, kTok, RT) | (1u << 15);    // both MN-major
        const uint32_t ring = smem_addr(sm), on = elect();
        // descriptors of the first stage and buffers; offsets add to them (bytes / 16)
        const uint64_t k_desc = sw128_desc(ring, 16, 1024), v_desc = sw128_desc(ring, kHalf, 1024);
        const uint64_t q_desc = sw128_desc(ring + S::kOffQ, 16, 1024);
        const uint64_t p_desc = sw128_desc(ring + S::kOffP, kHalf, 1024);
        const int N = (int)(w1 - w0);
        const bool wide = D > 64;
        int st = 0, seg = -1;        // ring stage of the next operand
        uint32_t ph = 0;             // and its phase
        auto advance = [&]() {
            if (++st == S::kStages) st = 0, ph ^= 1;
        };
        Cur ahead = cur;             // segment of the next score product
        int left = 0;                // its tiles not yet issued
        // Score product of tile g.  Its accumulator was last read for tile
        // g - 2, before that tile's P was complete.
        auto scores = [&](int g) {
            bool first = false;
            if (left == 0) {
                ahead.next(P);
                left = ahead.end - ahead.tile;
                ++seg;
                first = true;
            }
            const int qb = seg % S::kQ;
            if (first) await(&q_full[qb], (uint32_t)(seg / S::kQ) & 1, lost);
            await(&full[st], ph, lost);
            --left;
            // cp.async (generic proxy) data -> tensor core (async proxy)
            if (first || !P.box) fence_proxy_async();
            tc_fence_after();
            const uint64_t kd = k_desc + (uint32_t)st * (kStage >> 4);
            const uint64_t qd = q_desc + (uint32_t)qb * (S::kQBytes >> 4);
            const uint32_t d = tmem + (uint32_t)((g & 1) * RT);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) mma_on(on, d, kd + kk * 2, qd + kk * 2, idesc_s, kk != 0);
            if (wide) {
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    mma_on(on, d, kd + (kHalf >> 4) + kk * 2, qd + RT * 8u + kk * 2, idesc_s, 1);
            }
            commit_on(on, &empty[st]);  // also tells the softmax that the scores are there
            if (left == 0) commit_on(on, &q_empty[qb]);
            advance();
        };
        scores(0);
        cur.next(P);
        int tile = cur.tile;
        for (int g = 0; g < N; ++g) {
            if (g + 1 < N) scores(g + 1);
            await(&full[st], ph, lost);
            await(&p_full, (uint32_t)g & 1, lost);
            if (tile == cur.end) {
                cur.next(P);
                tile = cur.tile;
            }
            if (!P.box) fence_proxy_async();
            tc_fence_after();
            const uint64_t vd = v_desc + (uint32_t)st * (kStage >> 4);
            const uint32_t more = tile != cur.tile;
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
                mma_on(on, tmem + 2 * RT, vd + kk * 128, p_desc + kk * 128, idesc_o, kk ? 1u : more);
            commit_on(on, &empty[st]);  // also tells the softmax that P has been read
            advance();
            ++tile;
        }
        // nothing of this kernel's is in flight when tensor memory is returned
        commit_on(on, &drained);
        await(&drained, 0, lost);
    } else {
        // ---- softmax and output: thread = token, then = head column ------------
        const int wg = warp >> 2, tok = tid & 127, r0 = wg * S::kRows;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t t_s = tmem + lanes + (uint32_t)r0, t_o = tmem + lanes + 2 * RT + (uint32_t)r0;
        uint32_t *const see = reinterpret_cast<uint32_t *>(sm + S::kOffSee);
        int64_t *const row_out = reinterpret_cast<int64_t *>(sm + S::kOffRow);
        uint8_t *const prow = sm + S::kOffP + (uint32_t)(wg >> 1) * kHalf;
        const int pchunk = (wg & 1) * 4;
        const float c = P.c;
        float l[S::kRows];
        int see_b = -1, see_rt = -1;
        const int N = (int)(w1 - w0);
        int g = 0;  // tile
        // K of tile g is the ring's operand 2g - 1 (0 for the first), V is 2g + 2
        // (2g + 1 for the last).  The commit that frees an operand's stage is
        // the softmax's signal that the product is done; it waits for each
        // before the stage can be freed again.
        auto v_pos = [&](int g) { return g + 1 < N ? 2 * g + 2 : 2 * g + 1; };
        auto done = [&](int pos) {
            await(&empty[pos % S::kStages], (uint32_t)(pos / S::kStages) & 1, lost);
            tc_fence_after();
        };
        for (int seg = 0; cur.next(P); ++seg) {
            const int R = min(RT, cur.n * group - cur.rt * RT);  // rows in use
            if (cur.end * P.tok > cur.prefix && (see_b != cur.b || see_rt != cur.rt)) {
                // see[j]: the rows that see tree node j.  Ancestors by pointer
                // doubling in the (idle) P buffer; invalid parents count as padding.
                see_b = cur.b;
                see_rt = cur.rt;
                const int n = cur.n;
                uint32_t *const anc = reinterpret_cast<uint32_t *>(sm + S::kOffP);  // [n][8]
                int *const up = reinterpret_cast<int *>(anc + SGMV_TREE_MAX_NODES * 8);
                auto parent = [&](int i) {
                    const int p = a.parents ? a.parents[cur.t0 + i] : i - 1;
                    if (p < -2 || p >= i) set_error(P.err, kErrBadIndex);
                    return p < -1 || p >= i ? -2 : p;
                };
                named_sync<6, S::kSoft>();
                for (int i = tid; i < n; i += S::kSoft) up[i] = parent(i);
                named_sync<6, S::kSoft>();
                constexpr int kPer = (SGMV_TREE_MAX_NODES + S::kSoft - 1) / S::kSoft;
                uint32_t word[kPer][8];
                int to[kPer];
#pragma unroll
                for (int e = 0; e < kPer; ++e) {
                    const int i = tid + e * S::kSoft;
                    to[e] = -1;
                    if (i >= n) continue;
                    const int p = up[i];
                    to[e] = p >= 0 && up[p] != -2 ? p : -1;
#pragma unroll
                    for (int k = 0; k < 8; ++k) anc[i * 8 + k] = p != -2 && (i >> 5) == k ? 1u << (i & 31) : 0u;
                }
                named_sync<6, S::kSoft>();
#pragma unroll
                for (int e = 0; e < kPer; ++e)
                    if (tid + e * S::kSoft < n) up[tid + e * S::kSoft] = to[e];
                named_sync<6, S::kSoft>();
                for (int reach = 1; reach < n; reach <<= 1) {
#pragma unroll
                    for (int e = 0; e < kPer; ++e) {
                        const int i = tid + e * S::kSoft;
                        if (i >= n) continue;
                        const int p = up[i];
                        to[e] = p >= 0 ? up[p] : -1;
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            word[e][k] = anc[i * 8 + k] | (p >= 0 ? anc[p * 8 + k] : 0u);
                    }
                    named_sync<6, S::kSoft>();
#pragma unroll
                    for (int e = 0; e < kPer; ++e) {
                        const int i = tid + e * S::kSoft;
                        if (i >= n) continue;
                        up[i] = to[e];
#pragma unroll
                        for (int k = 0; k < 8; ++k) anc[i * 8 + k] = word[e][k];
                    }
                    named_sync<6, S::kSoft>();
                }
                for (int i = tid; i < n * S::kWords; i += S::kSoft) {
                    const int j = i / S::kWords, k = i - j * S::kWords;
                    uint32_t bits = 0;
                    for (int e = 0; e < (RT < 32 ? RT : 32); ++e) {
                        const int m = k * 32 + e;
                        if (m < R) {
                            const int node = (cur.rt * RT + m) / group;
                            bits |= (anc[node * 8 + (j >> 5)] >> (j & 31) & 1u) << e;
                        }
                    }
                    see[i] = bits;
                }
                named_sync<6, S::kSoft>();
            }
#pragma unroll
            for (int r = 0; r < S::kRows; ++r) l[r] = 0.f;
            for (int tile = cur.tile; tile < cur.end; ++tile, ++g) {
                done(g > 0 ? 2 * g - 1 : 0);
                const uint32_t ts = t_s + (uint32_t)((g & 1) * RT);
                // which rows see this token: all, none, or a node's
                const int j = tile * P.tok + tok;
                const bool tree = (tile + 1) * P.tok > cur.prefix, edge = tree || P.tok < kTok;
                uint32_t vis = 0xffffffffu;
                if (edge && (tok >= P.tok || j >= cur.prefix))
                    vis = tok < P.tok && j < cur.total ? see[(j - cur.prefix) * S::kWords + wg] : 0u;
                float s[S::kRows];
                // the masked exponents
                auto exponents = [&]() {
                    tmem_load(ts, s);
#pragma unroll
                    for (int i = 0; i < S::kRows; i += 4) {
                        const uint4 u = lds128(&s_ref[r0 + i]);
                        s[i] = fmaf(s[i], c, -__uint_as_float(u.x));
                        s[i + 1] = fmaf(s[i + 1], c, -__uint_as_float(u.y));
                        s[i + 2] = fmaf(s[i + 2], c, -__uint_as_float(u.z));
                        s[i + 3] = fmaf(s[i + 3], c, -__uint_as_float(u.w));
                    }
                    if (edge) {
#pragma unroll
                        for (int i = 0; i < S::kRows; ++i)
                            if (!(vis >> i & 1u)) s[i] = -INFINITY;
                    }
                };
                exponents();
                float top = -INFINITY;
#pragma unroll
                for (int i = 0; i < S::kRows; ++i) top = fmaxf(top, s[i]);
                if (group_any(wg, top > kBias + kSlack)) {
                    // new references: the larger of the old and this tile's maximum
                    tmem_load(ts, s);
                    int mine = 0;
#pragma unroll
                    for (int i = 0; i < S::kRows; ++i) {
                        const float y = !edge || (vis >> i & 1u) ? s[i] * c : -INFINITY;
                        const int m = __reduce_max_sync(0xffffffffu, ordered(y));
                        if (lane == i) mine = m;
                    }
                    if (lane < S::kRows) s_red[warp & 3][r0 + lane] = unordered(mine);
                    group_bar(wg);
                    if (tok < S::kRows) {
                        const int r = r0 + tok;
                        float m = -INFINITY;
                        for (int w = 0; w < 4; ++w) {
                            const float x = s_red[w][r];
                            m = x > m || x != x ? x : m;
                        }
                        const float old = s_ref[r];
                        float now = m - kBias;
                        now = now > old || now != now ? now : old;
                        s_fac[r] = old == kUnset ? 0.f : exp2_approx(old - now);
                        s_ref[r] = now;
                    }
                    group_bar(wg);
#pragma unroll
                    for (int r = 0; r < S::kRows; ++r) l[r] *= s_fac[r0 + r];
                    if (tile != cur.tile) {
                        done(v_pos(g - 1));
                        tmem_load(t_o, s);
#pragma unroll
                        for (int i = 0; i < S::kRows; ++i) s[i] *= s_fac[r0 + i];
                        tmem_store(t_o, s);
                    }
                    exponents();
                }
                T p[S::kRows];  // rounded to the tensor cores' operand type
#pragma unroll
                for (int i = 0; i < S::kRows; ++i) {
                    const float e = exp2_approx(s[i]);
                    l[i] += e;
                    p[i] = from_f<T>(e);
                }
                // the previous tile's P has been read
                if (g > 0) done(v_pos(g - 1));
#pragma unroll
                for (int q = 0; q < S::kRows / 8; ++q)
                    sts128(prow + sw128_offset(tok, pchunk + q), reinterpret_cast<const uint4 *>(p)[q]);
                if (tree) {
                    // non-finite v of tree nodes: out of the tile, noted; what TMA
                    // brought from the last page past the end: zeroed
                    const int v0 = max(0, cur.prefix - tile * P.tok), v1 = min(P.tok, cur.total - tile * P.tok);
                    const int ve = P.box ? (v1 + P.box - 1) / P.box * P.box : v1;
                    const int cpr = D / 8;
                    const int pv = v_pos(g);
                    await(&full[pv % S::kStages], (uint32_t)(pv / S::kStages) & 1, lost);
                    uint8_t *const vt = sm + (uint32_t)(pv % S::kStages) * kStage;
                    for (int i = tid; i < (ve - v0) * cpr; i += S::kSoft) {
                        const int m = v0 + i / cpr, cc = i % cpr;
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
                            sts128(at, u);
                            s_poison = seg;
                        }
                    }
                }
                fence_proxy_async();
                tc_fence_before();
                mbar_arrive(&p_full);
            }
            done(v_pos(g - 1));

            // ---- the segment's sums and rows' places -----------------------------
            {
                float v[S::kRows];
#pragma unroll
                for (int r = 0; r < S::kRows; ++r) v[r] = l[r];
                const int r = warp_sums(v, lane);
                if (S::kRows == 32 || (lane & 1) == 0) s_red[warp & 3][r0 + r] = v[0];
            }
            group_bar(wg);
            const bool whole = cur.tile == 0 && cur.end == cur.item_tiles;
            const int slot = 2 * (int)blockIdx.x + (cur.tile == 0 ? 1 : 0);
            if (tok < S::kRows) {
                const int r = r0 + tok;
                const float L = s_red[0][r] + s_red[1][r] + s_red[2][r] + s_red[3][r], ref = s_ref[r];
                int64_t to = -1;
                if (r < R) {
                    const int i = cur.rt * RT + r, node = i / group, hq = cur.h * group + (i - node * group);
                    const int64_t t = cur.t0 + node;
                    to = t * a.out_token + (int64_t)hq * a.out_head;
                    bool pad = false;
                    if (a.parents) {
                        const int p = a.parents[t];
                        pad = p < -1 || p >= node;
                    }
                    s_fac[r] = pad || L == 0.f ? 0.f : 1.f / L;
                    if (pad) to = ~to - 1;  // below -1: written as zeros
                    if (whole && a.lse)
                        a.lse[t * a.Hq + hq] = pad || L == 0.f ? -INFINITY : (ref + log2f(L)) * 0.693147180559945309f;
                }
                row_out[r] = to;
                if (!whole) {
                    float *const ml = P.ml + ((int64_t)slot * RT + r) * 2;
                    ml[0] = ref;
                    ml[1] = L;
                }
                s_ref[r] = kUnset;
            }
            group_bar(wg);
            const bool poison = *(volatile int *)&s_poison == seg, ok = !*lost;
            const int d = tok;
            {
                float v[S::kRows];
                tmem_load(t_o, v);
                if (poison && d < D) {
                    for (int jn = max(0, cur.tile * P.tok - cur.prefix); jn < min(cur.n, cur.end * P.tok - cur.prefix); ++jn) {
                        const int j = cur.prefix + jn, pg = j / a.block_size;
                        const int32_t block = a.block_table[cur.b * a.table_row + pg];
                        if (block < 0 || block >= a.num_blocks) continue;
                        const T x = static_cast<const T *>(a.v_cache)[(int64_t)block * a.cache_block +
                                                                     (int64_t)(j - pg * a.block_size) * a.cache_token +
                                                                     (int64_t)cur.h * a.cache_head + d];
                        if (!bad16<T>(*reinterpret_cast<const unsigned short *>(&x))) continue;
                        const uint32_t bits = see[jn * S::kWords + wg];
#pragma unroll
                        for (int i = 0; i < S::kRows; ++i)
                            if (bits >> i & 1u) v[i] += to_f<T>(x);
                    }
                }
                if (whole) {
                    if (d < D && ok) {
#pragma unroll
                        for (int i = 0; i < S::kRows; ++i) {
                            const int64_t to = row_out[r0 + i];
                            const float f = s_fac[r0 + i];
                            if (to >= 0)
                                static_cast<T *>(a.out)[to + d] = from_f<T>(f == 0.f ? 0.f : v[i] * f);
                            else if (to < -1)
                                static_cast<T *>(a.out)[~(to + 1) + d] = from_f<T>(0.f);
                        }
                    }
                } else {
                    float *const part = P.part + ((int64_t)slot * RT + r0) * 128 + d;
#pragma unroll
                    for (int i = 0; i < S::kRows; ++i)
                        if (r0 + i < R) part[i * 128] = v[i];
                }
            }
            if (!whole) {
                // the last CTA of the item to finish joins its parts, in share order
                const int first = (int)(cur.item0 / share), last = (int)((cur.item0 + cur.item_tiles - 1) / share);
                __threadfence();
                named_sync<6, S::kSoft>();
                if (tid == 0) {
                    const int done = atomicAdd(&P.count[first], 1);
                    s_last = done == last - first;
                    if (done == last - first) P.count[first] = 0;  // ready for the next call
                    __threadfence();
                }
                named_sync<6, S::kSoft>();
                if (s_last) {
                    auto at = [&](int k, int r) { return (int64_t)(2 * k + (k == first)) * RT + r; };
                    for (int r = tid; r < R; r += S::kSoft) {
                        float M = kUnset, L = 0.f;
                        bool nan = false;
                        for (int k = first; k <= last; ++k) {
                            const float m = __ldcg(P.ml + at(k, r) * 2);
                            nan |= m != m;
                            M = fmaxf(M, m);
                        }
                        if (nan) M = NAN;
                        for (int k = first; k <= last; ++k) {
                            const float m = __ldcg(P.ml + at(k, r) * 2), x = __ldcg(P.ml + at(k, r) * 2 + 1);
                            if (m != kUnset) L += exp2_approx(m - M) * x;
                        }
                        const bool none = row_out[r] < -1 || L == 0.f;
                        s_red[0][r] = M;
                        s_red[1][r] = none ? 0.f : 1.f / L;
                        if (a.lse && ok) {
                            const int i = cur.rt * RT + r, node = i / group;
                            a.lse[(int64_t)(cur.t0 + node) * a.Hq + cur.h * group + (i - node * group)] =
                                none ? -INFINITY : (M + log2f(L)) * 0.693147180559945309f;
                        }
                    }
                    named_sync<6, S::kSoft>();
                    constexpr int kJoin = 8;  // rows whose parts are in flight together
                    for (int rc = wg * kJoin; rc < R && d < D; rc += kJoin * S::kGroups) {
                        float o[kJoin] = {};
#pragma unroll 2
                        for (int k = first; k <= last; ++k) {
#pragma unroll
                            for (int i = 0; i < kJoin; ++i) {
                                if (rc + i >= R) continue;
                                const float m = __ldcg(P.ml + at(k, rc + i) * 2);
                                const float x = __ldcg(P.part + at(k, rc + i) * 128 + d);
                                if (m != kUnset) o[i] += exp2_approx(m - s_red[0][rc + i]) * x;
                            }
                        }
#pragma unroll
                        for (int i = 0; i < kJoin; ++i) {
                            if (rc + i >= R || !ok) continue;
                            const int64_t to = row_out[rc + i];
                            const float f = s_red[1][rc + i];
                            static_cast<T *>(a.out)[(to < -1 ? ~(to + 1) : to) + d] =
                                from_f<T>(f == 0.f ? 0.f : o[i] * f);
                        }
                    }
                }
            }
            // every thread has read the rows' places, sums and the poison mark
            named_sync<6, S::kSoft>();
        }
        if (tid == 0 && *lost) set_error(P.err, kErrTimeout);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) tmem_dealloc(tmem, S::kTmem);
}

template <typename T, int RT>
int launch(const MmaParams &p, int ctas, cudaStream_t stream) {
    static_assert(Shape<RT>::kBytes <= 227 * 1024 - 8192, "shared memory");
    const cudaError_t e = cudaFuncSetAttribute(sgmv_tree_mma_kernel<T, RT>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)Shape<RT>::kBytes);
    if (e != cudaSuccess) return (int)e;
    return spec_launch(sgmv_tree_mma_kernel<T, RT>, dim3((unsigned)ctas), Shape<RT>::kThreads,
                       Shape<RT>::kBytes, 1, stream, p);
}

// Rows per tile: what a sequence of average length fills.
int row_tile(int32_t T, int32_t B, int32_t group) {
    const int64_t rows = ((int64_t)T + B - 1) / B * group;
    return rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128;
}

constexpr size_t kCountBytes = 1024;

}  // namespace

size_t tree_mma_workspace(int32_t T, int32_t B, int32_t group) {
    return kCountBytes + (size_t)kMaxCtas * 2u * (size_t)row_tile(T, B, group) * 130u * 4u;
}

int tree_mma_launch(const sgmv_tree_attention_args &a, int nsm, int *err, cudaStream_t stream) {
    const int group = a.Hq / a.Hkv, rt = row_tile(a.T, a.B, group);
    const int ctas = nsm < 1 ? 1 : nsm < kMaxCtas ? nsm : kMaxCtas;
    MmaParams p;
    p.a = a;
    p.c = a.scale * 1.4426950408889634f;
    p.group = group;
    p.count = static_cast<int *>(a.workspace);
    p.ml = reinterpret_cast<float *>(static_cast<uint8_t *>(a.workspace) + kCountBytes);
    p.part = p.ml + (size_t)kMaxCtas * 2 * rt * 2;
    p.err = err;
    const bool bf16 = a.dtype == SGMV_BF16;
    // Boxes are as high as pages allow: TMA's cost here is per box (at pages
    // of 24 tokens, boxes of 8 filling every tile measured 115 us, boxes of 24 and tiles of
    // 120 tokens XX us, on 128 sequences of up to 2100 tokens, 4 heads of 80)
    p.box = std::gcd(a.block_size, kTok);
    p.tok = kTok;
    if (a.block_size % 8 == 0 && a.block_size < kTok && a.block_size > p.box) {
        p.box = a.block_size;
        p.tok = kTok / p.box * p.box;
    }
    if (p.box >= 8) {
        const cuuint64_t dims[4] = {(cuuint64_t)a.D, (cuuint64_t)a.block_size, (cuuint64_t)a.Hkv,
                                    (cuuint64_t)a.num_blocks};
        const cuuint64_t strides[3] = {(cuuint64_t)a.cache_token * 2u, (cuuint64_t)a.cache_head * 2u,
                                       (cuuint64_t)a.cache_block * 2u};
        const cuuint32_t box[4] = {64, (cuuint32_t)p.box, 1, 1};
        if (!tmap_encode(&p.map_k, bf16, 4, a.k_cache, dims, strides, box, true) ||
            !tmap_encode(&p.map_v, bf16, 4, a.v_cache, dims, strides, box, true))
            p.box = 0, p.tok = kTok;  // strides that a tensor map cannot hold
    } else {
        p.box = 0;
    }
    const bool h = a.dtype == SGMV_F16;
    using B16 = __nv_bfloat16;
    switch (rt) {
        case 16: return h ? launch<__half, 16>(p, ctas, stream) : launch<B16, 16>(p, ctas, stream);
        case 32: return h ? launch<__half, 32>(p, ctas, stream) : launch<B16, 32>(p, ctas, stream);
        case 64: return h ? launch<__half, 64>(p, ctas, stream) : launch<B16, 64>(p, ctas, stream);
        default: return h ? launch<__half, 128>(p, ctas, stream) : launch<B16, 128>(p, ctas, stream);
    }
}

}  // namespace sgmv
