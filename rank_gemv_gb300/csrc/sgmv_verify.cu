// sgmv_verify.cu -- verification of drafted tokens: the walk down each
// sequence's tree, and the token drawn where it ends.
//
// Probabilities become whole multiples of 2^-38, so that a distribution's sum
// is exact in 64 bits whatever the order of summation, and the drawn token is
// the same for any division of the vocabulary among threads.  The products
// q * W are single fp32 multiplications of each element.  An accepted child
// costs two lookups; only a rejected one needs a pass over the vocabulary, for
// the sum of what is left.  The rest of a distribution after k rejections
// is recomputed from p, q and the k earlier sums instead of being stored.
#include "sgmv_device.cuh"
#include "sgmv_spec.h"

namespace sgmv {
namespace {

constexpr int kVerifyThreads = 1024;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int64_t kOne = 1ll << 38;

__device__ __forceinline__ float prob(float p) { return fminf(fmaxf(p, 0.f), 1.f); }  // NaN -> 0
__device__ __forceinline__ int64_t weight(float p) { return (int64_t)(prob(p) * 0x1p38f); }

struct VerifyShared {
    float W[SGMV_TREE_MAX_NODES];      // W before each rejection at this node
    int32_t out[SGMV_TREE_MAX_NODES];  // rejected tokens (without a draft)
    int64_t part[kVerifyWarps];
    int64_t total;
    int32_t token;
};

// w(token j) after `k` rejections at a node with distributions p and q
__device__ __forceinline__ int64_t rest(const float *p, const float *q, int j, int k,
                                        const VerifyShared &s) {
    int64_t w = weight(p[j]);
    if (q) {
        const float qj = k > 0 ? prob(q[j]) : 0.f;
        for (int i = 0; i < k; ++i) {
            w -= (int64_t)__fmul_rn(qj, s.W[i]);
            w = w < 0 ? 0 : w;
        }
    } else {
        for (int i = 0; i < k; ++i)
            if (s.out[i] == j) w = 0;
    }
    return w;
}

// One CTA per sequence.  Warp w holds vocabulary range [w c, (w + 1) c).
__global__ void __launch_bounds__(kVerifyThreads)
    sgmv_verify_kernel(const __grid_constant__ sgmv_tree_verify_args a, int *err) {
    __shared__ VerifyShared s;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int b = blockIdx.x;
    pdl_wait();
    pdl_trigger();
    const int t0 = a.tree_ptr[b], n = a.tree_ptr[b + 1] - t0;
    int32_t *path = a.path + (int64_t)b * a.max_path;
    const bool bad = t0 < 0 || n < 0 || n > SGMV_TREE_MAX_NODES || (int64_t)t0 + n > a.T;
    if (bad && tid == 0) set_error(err, kErrBadSegments);
    if (bad || n == 0) {
        for (int i = tid; i < a.max_path; i += kVerifyThreads) path[i] = -1;
        if (tid == 0) a.count[b] = 0, a.token[b] = -1;
        return;
    }
    const int chunk = (a.V + kVerifyWarps - 1) / kVerifyWarps;
    const int v0 = min(a.V, warp * chunk), v1 = min(a.V, v0 + chunk);
    // sums of the rest after k rejections: part[] per warp, total
    auto sum_pass = [&](const float *p, const float *q, int k) {
        int64_t sum = 0;
        for (int j = v0 + lane; j < v1; j += 32) sum += rest(p, q, j, k, s);
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        __syncthreads();  // earlier readers of part and total are done
        if (lane == 0) s.part[warp] = sum;
        __syncthreads();
        if (tid == 0) {
            int64_t t = 0;
            for (int w = 0; w < kVerifyWarps; ++w) t += s.part[w];
            s.total = t;
        }
        __syncthreads();
    };
    int cur = 0, count = 1, k = 0;  // last accepted node, nodes accepted, rejections at it
    int64_t total = kOne;
    const float *p = a.target + (int64_t)t0 * a.target_row;
    const float *q = a.draft ? a.draft + (int64_t)t0 * a.draft_row : nullptr;
    if (tid == 0 && a.max_path > 0) path[0] = 0;
    for (int i = 1; i < n && count < a.max_path; ++i) {  // every thread walks alike
        const int par = a.parents ? a.parents[t0 + i] : i - 1;
        if (par >= i || par < -2) {
            if (tid == 0) set_error(err, kErrBadIndex);
            continue;
        }
        if (par != cur) continue;
        const int tok = a.tokens[t0 + i];
        if (tok < 0 || tok >= a.V) {
            if (tid == 0) set_error(err, kErrBadIndex);
            continue;
        }
        const float have = __ll2float_rn(rest(p, q, tok, k, s));
        const float qt = q ? prob(q[tok]) : 1.f;
        if (__fmul_rn(__fmul_rn(a.u_accept[t0 + i], qt), __ll2float_rn(total)) < have) {
            if (tid == 0) path[count] = i;
            ++count;
            cur = i;
            k = 0;
            total = kOne;
            p = a.target + (int64_t)(t0 + i) * a.target_row;
            if (q) q = a.draft + (int64_t)(t0 + i) * a.draft_row;
            __syncthreads();  // s.W is rewritten by the next rejection
        } else {
            __syncthreads();
            if (tid == 0) s.W[k] = __ll2float_rn(total), s.out[k] = tok;
            __syncthreads();
            ++k;
            sum_pass(p, q, k);
            total = s.total;
        }
    }
    for (int i = count + tid; i < a.max_path; i += kVerifyThreads) path[i] = -1;
    // the rest's sums (of the last rejection, or of the target itself)
    if (k == 0) sum_pass(p, q, 0);
    if (s.total == 0 && k > 0) {
        k = 0;
        sum_pass(p, q, 0);
    }
    total = s.total;
    if (tid == 0) a.count[b] = count;
    if (total == 0) {
        if (tid == 0) a.token[b] = -1;
        return;
    }
    const int64_t unit = 1ll << 24;
    const float u = a.u_sample[b];
    int64_t m = (int64_t)__fmul_rn(u, 0x1p24f);
    m = m < 0 ? 0 : m >= unit ? unit - 1 : m;
    const int64_t mark = (total >> 24) * m + (((total & (unit - 1)) * m) >> 24);
    // the warp whose range holds the mark finds the first token beyond it
    int64_t before = 0;
    for (int w = 0; w < warp; ++w) before += s.part[w];
    if (before <= mark && mark < before + s.part[warp]) {
        for (int j0 = v0; j0 < v1; j0 += 32) {
            int64_t run = j0 + lane < v1 ? rest(p, q, j0 + lane, k, s) : 0;
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t up = __shfl_up_sync(0xffffffffu, run, o);
                if (lane >= o) run += up;
            }
            const unsigned over = __ballot_sync(0xffffffffu, before + run > mark);
            if (over) {
                if (lane == 0) a.token[b] = j0 + __ffs(over) - 1;
                break;
            }
            before += __shfl_sync(0xffffffffu, run, 31);
        }
    }
}

}  // namespace

int tree_verify_launch(const sgmv_tree_verify_args &a, int nsm, int *err, cudaStream_t stream) {
    return spec_launch(sgmv_verify_kernel, dim3((unsigned)a.B), kVerifyThreads, 0, 1, stream, a, err);
}

}  // namespace sgmv
