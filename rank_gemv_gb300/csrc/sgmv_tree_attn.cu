// sgmv_tree_attn.cu -- attention of every sequence's drafted tokens over the
// paged cache: o = softmax(scale * q K^T) V over the context, the row's
// ancestors in the tree and itself.
//
// This file: heads of more than 128 columns, on the CUDA cores.  One CTA per (row,
// head): its warps take the tokens in turn, keep a running maximum and sum each, and join at
// the end.  K and V are read for every row and query head, and the context is not
// split, so it is the chain of tokens (a reduction over the warp and two exponentials each)
// that bounds it, far from the bytes: 32 sequences of one row, up to 4096 tokens, 32
// heads of 256: 1330 us (1.6 TB/s of algorithmic bytes); with trees of up to 16 rows 4700; one row over 32768
// tokens, 32 heads on 8: 10200.
#include <math.h>

#include "sgmv_device.cuh"
#include "sgmv_spec.h"

namespace sgmv {
namespace {

constexpr int kRowThreads = 128;
constexpr int kRowWarps = kRowThreads / 32;
constexpr int kNodeWords = SGMV_TREE_MAX_NODES / 32;

// Sequence of row t: the last b with tree_ptr[b] <= t (B >= 1).
__device__ __forceinline__ int sequence_of(const int32_t *tree_ptr, int B, int t) {
    int lo = 0, hi = B - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (tree_ptr[mid] <= t) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

template <typename T>
__global__ void __launch_bounds__(kRowThreads)
    sgmv_tree_row_kernel(const __grid_constant__ sgmv_tree_attention_args a, int *err) {
    __shared__ uint32_t s_anc[kNodeWords];
    __shared__ int s_seen;  // 0: a padding row
    __shared__ float s_m[kRowWarps], s_l[kRowWarps], s_o[kRowWarps][kSpecMaxD];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int t = blockIdx.x, h = blockIdx.y;
    pdl_wait();
    pdl_trigger();
    if (t == 0 && h == 0)  // one CTA looks the whole of tree_ptr over
        for (int s = tid; s < a.B; s += kRowThreads)
            if (a.tree_ptr[s] < 0 || a.tree_ptr[s + 1] < a.tree_ptr[s] || a.tree_ptr[s + 1] > a.T)
                set_error(err, kErrBadSegments);
    const int b = sequence_of(a.tree_ptr, a.B, t);
    const int t0 = a.tree_ptr[b], t1 = a.tree_ptr[b + 1], n = t1 - t0;
    if (t < t0 || t >= t1) return;
    const int64_t prefix = a.prefix_lens[b];
    const int i = t - t0;
    const bool report = tid == 0 && h == 0;
    if (t0 < 0 || n > SGMV_TREE_MAX_NODES || t1 > a.T || prefix < 0 ||
        prefix + n > (int64_t)a.max_blocks * a.block_size) {
        if (report) set_error(err, kErrBadSegments);
        return;
    }
    if (tid < kNodeWords) s_anc[tid] = 0;
    __syncthreads();
    if (tid == 0) {
        int seen = 1;
        for (int j = i; j >= 0;) {
            const int par = a.parents ? a.parents[t0 + j] : j - 1;
            if (par < -2 || par >= j) set_error(err, kErrBadIndex);
            if (par < -1 || par >= j) {  // padding, or a parent that cannot be one
                if (j == i) seen = 0;
                break;
            }
            s_anc[j >> 5] |= 1u << (j & 31);
            j = par;
        }
        s_seen = seen;
    }
    __syncthreads();
    const bool seen = s_seen != 0;
    const int D = a.D, col = lane * 8;
    const int64_t kvh = h / (a.Hq / a.Hkv);
    float q[8] = {}, o[8] = {};
    if (col < D) load8<T>(static_cast<const T *>(a.q) + t * a.q_token + h * a.q_head + col, q);
#pragma unroll
    for (int e = 0; e < 8; ++e) q[e] *= a.scale;
    float m = -INFINITY, l = 0.f;
    const int64_t total = seen ? prefix + n : 0;
    for (int64_t j = warp; j < total; j += kRowWarps) {
        if (j >= prefix && !(s_anc[(j - prefix) >> 5] >> ((j - prefix) & 31) & 1)) continue;
        const int64_t pg = j / a.block_size;
        const int32_t block = a.block_table[b * a.table_row + pg];
        if (block < 0 || block >= a.num_blocks) {
            if (lane == 0) set_error(err, kErrBadIndex);
            continue;
        }
        const int64_t off = block * a.cache_block + (j - pg * a.block_size) * a.cache_token +
                            kvh * a.cache_head + col;
        float x[8] = {}, s = 0.f;
        if (col < D) load8<T>(static_cast<const T *>(a.k_cache) + off, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) s = fmaf(q[e], x[e], s);
#pragma unroll
        for (int w = 16; w > 0; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
        if (s == -INFINITY) continue;
        const float mn = fmaxf(m, s);
        const float f = m == -INFINITY ? 0.f : expf(m - mn), p = expf(s - mn);
        m = mn;
        l = l * f + p;
        if (col < D) load8<T>(static_cast<const T *>(a.v_cache) + off, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = o[e] * f + p * x[e];
    }
    if (lane == 0) s_m[warp] = m, s_l[warp] = l;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (col < D) s_o[warp][col + e] = o[e];
    __syncthreads();
    float M = -INFINITY, L = 0.f;
    for (int w = 0; w < kRowWarps; ++w) M = fmaxf(M, s_m[w]);
    float f[kRowWarps];
    for (int w = 0; w < kRowWarps; ++w) {
        f[w] = s_m[w] == -INFINITY ? 0.f : expf(s_m[w] - M);
        L += s_l[w] * f[w];
    }
    for (int c = tid; c < D; c += kRowThreads) {
        float x = 0.f;
        for (int w = 0; w < kRowWarps; ++w)
            if (f[w] != 0.f) x += s_o[w][c] * f[w];
        static_cast<T *>(a.out)[t * a.out_token + h * a.out_head + c] = from_f<T>(L == 0.f ? 0.f : x / L);
    }
    if (a.lse && tid == 0) a.lse[(int64_t)t * a.Hq + h] = L == 0.f ? -INFINITY : M + logf(L);
}

}  // namespace

size_t tree_attention_workspace(int32_t T, int32_t Hq, int32_t Hkv, int32_t D) {
    return D <= kMmaMaxD ? tree_mma_workspace(T, Hq / Hkv) : 256;
}

int tree_attention_launch(const sgmv_tree_attention_args &a, int nsm, int *err,
                          cudaStream_t stream) {
    if (a.D <= kMmaMaxD) return tree_mma_launch(a, nsm, err, stream);
    const dim3 grid((unsigned)a.T, (unsigned)a.Hq, 1);
    return a.dtype == SGMV_F16
               ? spec_launch(sgmv_tree_row_kernel<__half>, grid, kRowThreads, 0, 1, stream, a, err)
               : spec_launch(sgmv_tree_row_kernel<__nv_bfloat16>, grid, kRowThreads, 0, 1, stream, a,
                             err);
}

}  // namespace sgmv
