// sgmv_verify.cu -- verification of drafted tokens: the walk down each
// sequence's tree, and the token drawn where it ends.
//
// Probabilities become whole multiples of 2^-38, so that a distribution's sum
// is exact in 64 bits whatever the order of summation, and the drawn token is
// the same for any division of the vocabulary among threads.  The products
// q * W are single fp32 multiplications of each element.
//
// Every node's p and q at its own token are looked up first, all at once, so
// the walk itself touches no memory; only a rejected child costs a pass over
// the vocabulary, for the sum of what is left.  The rest of a distribution
// after k rejections is recomputed from p, q and the k earlier sums instead of
// being stored.  Without a draft a rejection only takes the token out, so one
// pass per node is enough.
//
// A cluster of CTAs shares a sequence's vocabulary when there are few
// sequences; all of its CTAs walk alike and exchange their sums through
// distributed shared memory.
#include <algorithm>

#include "sgmv_device.cuh"
#include "sgmv_spec.h"

namespace sgmv {
namespace {

constexpr int kVerifyThreads = 512;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kVerifyMaxCluster = 8;
constexpr int kVerifyUnroll = 4;  // vectors in flight per thread and distribution
constexpr int64_t kOne = 1ll << 38;

__device__ __forceinline__ float prob(float p) { return fminf(fmaxf(p, 0.f), 1.f); }  // NaN -> 0
// Whole part of f >= 0, f < 2^63, times 2^up.  Conversions between fp32 and
// 64-bit integers run at a fraction of the rate of these shifts here (they took
// 44 of 110 us on 128 rows of 100277).
__device__ __forceinline__ int64_t whole(float f, int up) {
    const uint32_t bits = __float_as_uint(f), m = (bits & 0x7fffffu) | 0x800000u;
    const int s = (int)(bits >> 23) - 150 + up;
    return s >= 0 ? (int64_t)((uint64_t)m << s) : (int64_t)(m >> min(31, -s));
}
__device__ __forceinline__ int64_t weight(float p) { return whole(prob(p), 38); }

struct VerifyShared {
    float p[SGMV_TREE_MAX_NODES], q[SGMV_TREE_MAX_NODES];  // at the node's token, after its parent
    float u[SGMV_TREE_MAX_NODES];
    int32_t token[SGMV_TREE_MAX_NODES];
    int16_t parent[SGMV_TREE_MAX_NODES];  // -2: not to be tried
    float W[SGMV_TREE_MAX_NODES];         // W before each rejection at this node
    int32_t out[SGMV_TREE_MAX_NODES];     // rejected tokens (without a draft)
    int64_t part[kVerifyWarps];           // sums of the warps' ranges
    int64_t mine[2];                      // sum of this CTA's range, by pass
    int64_t scan[kVerifyWarps];
};

// The rest after k rejections of a token with p, q (with a draft).
__device__ __forceinline__ int64_t shrink(float p, float q, int k, const float *W) {
    int64_t w = weight(p);
    const float qc = prob(q);
    for (int i = 0; i < k; ++i) {
        w -= whole(__fmul_rn(qc, W[i]), 0);
        w = w < 0 ? 0 : w;
    }
    return w;
}

// The sum of four tokens' rests.  Small probabilities have weights below 2^32,
// as nearly all of a vocabulary's are: then 32-bit conversions, which saturate
// at both ends and take NaN as 0, do for weights and products alike.
__device__ __forceinline__ int64_t shrink4(const float4 &x, const float4 &y, int k, const float *W) {
    const float *const p = &x.x, *const q = &y.x;
    uint32_t w[4], top = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) top = max(top, w[e] = __float2uint_rz(p[e] * 0x1p38f));
    for (int i = 0; i < k; ++i) {
        const float Wi = W[i];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t r = __float2uint_rz(__fmul_rn(fminf(q[e], 1.f), Wi));
            top = max(top, r);
            w[e] = w[e] > r ? w[e] - r : 0u;
        }
    }
    if (top == 0xffffffffu)
        return shrink(x.x, y.x, k, W) + shrink(x.y, y.y, k, W) + shrink(x.z, y.z, k, W) + shrink(x.w, y.w, k, W);
    return (int64_t)((uint64_t)w[0] + w[1] + w[2] + w[3]);
}

__global__ void __launch_bounds__(kVerifyThreads, 2)
    sgmv_verify_kernel(const __grid_constant__ sgmv_tree_verify_args a, int *err) {
    __shared__ VerifyShared s;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cl = (int)cluster_size(), rank = (int)cluster_rank(), b = (int)blockIdx.x / cl;
    pdl_wait();
    pdl_trigger();
    const int t0 = a.tree_ptr[b], n = a.tree_ptr[b + 1] - t0;
    int32_t *path = a.path + (int64_t)b * a.max_path;
    const bool writer = rank == 0 && tid == 0;
    const bool bad = t0 < 0 || n < 0 || n > SGMV_TREE_MAX_NODES || (int64_t)t0 + n > a.T;
    if (bad && writer) set_error(err, kErrBadSegments);
    if (bad || n == 0) {  // the whole cluster alike
        if (rank == 0)
            for (int i = tid; i < a.max_path; i += kVerifyThreads) path[i] = -1;
        if (writer) a.count[b] = 0, a.token[b] = -1;
        return;
    }
    for (int i = tid; i < n; i += kVerifyThreads) {
        int par = a.parents ? a.parents[t0 + i] : i - 1;
        const int tok = a.tokens[t0 + i];
        if (par >= i || par < -2) {
            if (rank == 0) set_error(err, kErrBadIndex);
            par = -2;
        }
        if (i > 0 && par >= 0 && (tok < 0 || tok >= a.V)) {
            if (rank == 0) set_error(err, kErrBadIndex);
            par = -2;
        }
        s.parent[i] = (int16_t)(i > 0 && par >= 0 ? par : -2);
        s.token[i] = tok;
        if (i > 0 && par >= 0) {
            s.p[i] = a.target[(int64_t)(t0 + par) * a.target_row + tok];
            s.q[i] = a.draft ? a.draft[(int64_t)(t0 + par) * a.draft_row + tok] : 1.f;
            s.u[i] = a.u_accept[t0 + i];
        }
    }
    __syncthreads();
    // This warp's range of the vocabulary, whole vectors long.
    const int share = ((a.V + cl * kVerifyWarps - 1) / (cl * kVerifyWarps) + 3) / 4 * 4;
    const int v0 = min(a.V, (rank * kVerifyWarps + warp) * share), v1 = min(a.V, v0 + share);
    int cur = 0, count = 1, k = 0;  // last accepted node, nodes accepted, rejections at it
    int passes = 0, held = -1;      // held: the node whose p and q the registers hold
    // a lane's vectors of one batch, and one element before or behind them
    float4 x[kVerifyUnroll], y[kVerifyUnroll];
    float xs = 0.f, ys = 0.f;
    // Sum of the rest after k rejections (k = 0 without a draft: of p itself).
    // Leaves the warps' sums in part[], every CTA's in mine[], returns the total.
    auto sum_pass = [&](const float *p, const float *q, int k) -> int64_t {
        int64_t sum = 0;
        const int skew = (int)(reinterpret_cast<uintptr_t>(p) >> 2) & 3;
        const bool vec = k == 0 || ((reinterpret_cast<uintptr_t>(q) >> 2) & 3) == (uintptr_t)skew;
        if (vec) {
            // whole 16-byte vectors [a0, a1) and up to six elements around them
            const int a0 = min(v1, v0 + ((4 - skew) & 3)), a1 = a0 + (v1 - a0) / 4 * 4;
            const bool one = a1 - a0 <= 128 * kVerifyUnroll;  // one batch: kept for the node's next pass
            const bool have = one && k > 0 && held == cur;
            if (!have) {
                const int e = lane < a0 - v0 ? v0 + lane : a1 + lane - (a0 - v0);
                xs = ys = 0.f;
                if (e < v1 && (e < a0 || e >= a1)) {
                    xs = p[e];
                    if (k > 0) ys = q[e];
                }
            }
            sum += shrink(xs, ys, k, s.W);
            for (int j0 = a0; j0 < a1; j0 += 128 * kVerifyUnroll) {
#pragma unroll
                for (int e = 0; e < kVerifyUnroll; ++e) {
                    if (have) continue;
                    const int j = j0 + 128 * e + lane * 4;
                    x[e] = y[e] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (j < a1) {
                        x[e] = *reinterpret_cast<const float4 *>(p + j);
                        if (k > 0) y[e] = *reinterpret_cast<const float4 *>(q + j);
                    }
                }
#pragma unroll
                for (int e = 0; e < kVerifyUnroll; ++e)
                    if (j0 + 128 * e < a1)
                        sum += shrink4(x[e], y[e], k, s.W);
            }
            held = one && k > 0 ? cur : -1;
        } else {
            for (int j = v0 + lane; j < v1; j += 32) sum += shrink(p[j], q[j], k, s.W);
        }
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0) s.part[warp] = sum;
        __syncthreads();
        int64_t total = 0;
        for (int w = 0; w < kVerifyWarps; ++w) total += s.part[w];
        if (cl > 1) {
            // two buffers: a CTA may be a pass ahead of those that still read
            const int at = passes++ & 1;
            if (tid == 0) s.mine[at] = total;
            cluster_sync();
            total = 0;
            for (int r = 0; r < cl; ++r) {
                const uint32_t addr = peer_addr(&s.mine[at], (uint32_t)r);
                uint64_t v;
                asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
                total += (int64_t)v;
            }
        } else {
            passes++;
            if (tid == 0) s.mine[0] = total;
        }
        return total;
    };
    int64_t total = kOne;           // W
    bool summed = false;            // part[] and mine[] hold this node's rest
    const float *p = a.target + (int64_t)t0 * a.target_row;
    const float *q = a.draft ? a.draft + (int64_t)t0 * a.draft_row : nullptr;
    if (writer) path[0] = 0;
    for (int i = 1; i < n && count < a.max_path; ++i) {  // every thread walks alike
        if (s.parent[i] != cur) continue;
        const int tok = s.token[i];
        int64_t have = q ? shrink(s.p[i], s.q[i], k, s.W) : weight(s.p[i]);
        if (!q)
            for (int e = 0; e < k; ++e)
                if (s.out[e] == tok) have = 0;
        if (__fmul_rn(__fmul_rn(s.u[i], prob(s.q[i])), __ll2float_rn(total)) < __ll2float_rn(have)) {
            if (writer) path[count] = i;
            ++count;
            cur = i;
            k = 0;
            total = kOne;
            summed = false;
            p = a.target + (int64_t)(t0 + i) * a.target_row;
            if (q) q = a.draft + (int64_t)(t0 + i) * a.draft_row;
            continue;
        }
        __syncthreads();  // W, out and part[] are no longer read
        if (q) {
            if (tid == 0) s.W[k] = __ll2float_rn(total);
            ++k;
            __syncthreads();
            total = sum_pass(p, q, k);
        } else {
            if (!summed) total = sum_pass(p, nullptr, 0);
            __syncthreads();
            total -= have;
            // the token's weight leaves its warp's and its CTA's sums
            const int owner = tok / share;
            if (tid == 0) {
                s.out[k] = tok;
                if (owner / kVerifyWarps == rank) s.part[owner % kVerifyWarps] -= have;
            }
            ++k;
            __syncthreads();
        }
        summed = true;
    }
    if (rank == 0)
        for (int i = count + tid; i < a.max_path; i += kVerifyThreads) path[i] = -1;
    if (writer) a.count[b] = count;
    __syncthreads();
    if (!summed) total = sum_pass(p, q, 0);
    if (total == 0 && k > 0) {  // nothing left: the target's own
        k = 0;
        __syncthreads();
        total = sum_pass(p, q, 0);
    }
    if (total > 0) {
        const int64_t unit = 1ll << 24;
        int64_t m = (int64_t)__fmul_rn(a.u_sample[b], 0x1p24f);
        m = m < 0 ? 0 : m >= unit ? unit - 1 : m;
        const int64_t mark = (total >> 24) * m + (((total & (unit - 1)) * m) >> 24);
        // where this CTA's range begins in the running sum
        int64_t mine = 0, before = 0;
        for (int w = 0; w < kVerifyWarps; ++w) mine += s.part[w];
        if (cl > 1) {
            const int at = passes & 1;
            if (tid == 0) s.mine[at] = mine;
            cluster_sync();
            for (int r = 0; r < rank; ++r) {
                const uint32_t addr = peer_addr(&s.mine[at], (uint32_t)r);
                uint64_t v;
                asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
                before += (int64_t)v;
            }
        }
        if (before <= mark && mark < before + mine) {  // the token is in this CTA's range
            int w = 0;
            while (mark >= before + s.part[w]) before += s.part[w++];
            const int j0 = min(a.V, (rank * kVerifyWarps + w) * share), j1 = min(a.V, j0 + share);
            // the first token of warp w's range whose running sum passes the mark
            for (int jb = j0; jb < j1; jb += kVerifyThreads) {
                const int j = jb + tid;
                int64_t run = 0;
                if (j < j1) {
                    run = q ? shrink(p[j], k > 0 ? q[j] : 0.f, k, s.W) : weight(p[j]);
                    if (!q)
                        for (int e = 0; e < k; ++e)
                            if (s.out[e] == j) run = 0;
                }
                for (int o = 1; o < 32; o <<= 1) {
                    const int64_t up = __shfl_up_sync(0xffffffffu, run, o);
                    if (lane >= o) run += up;
                }
                if (lane == 31) s.scan[warp] = run;
                __syncthreads();
                int64_t all = 0, here = before;
                for (int e = 0; e < kVerifyWarps; ++e) {
                    if (e < warp) here += s.scan[e];
                    all += s.scan[e];
                }
                const unsigned over = __ballot_sync(0xffffffffu, here + run > mark);
                if (here <= mark && over && lane == 0) a.token[b] = jb + warp * 32 + __ffs(over) - 1;
                before += all;
                if (before > mark) break;
                __syncthreads();
            }
        }
    } else if (writer) {
        a.token[b] = -1;
    }
    if (cl > 1) cluster_sync();  // a peer may still read this CTA's shared memory
}

}  // namespace

int tree_verify_launch(const sgmv_tree_verify_args &a, int nsm, int *err, cudaStream_t stream) {
    // CTAs per sequence: up to eight, each with 2048 tokens of the vocabulary at
    // least.  Sequences differ in their rejections, so spreading every one of them
    // wins over filling the SMs once (128 chains over 100277 tokens: 63, 51, 47 and 49 us
    // with 1, 2, 4 and 8 CTAs each; 32 trees over 32000: 39, 31, 26 and 24 us).
    int cl = 1;
    while (cl < kVerifyMaxCluster && (int64_t)a.B * cl * 2 <= 4 * std::max(1, nsm) && a.V >= cl * 2 * 2048) cl *= 2;
    return spec_launch(sgmv_verify_kernel, dim3((unsigned)a.B * (unsigned)cl), kVerifyThreads, 0, cl, stream, a, err);
}

}  // namespace sgmv
