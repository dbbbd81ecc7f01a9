// sgmv_commit.cu -- the accepted tokens' k and v to their final places in the
// paged cache, in place.
//
// A thread owns one 16-byte piece of a head in one layer of k or v and moves it
// for every accepted node in ascending order.  The node of depth d sits at
// position >= d, and later nodes at still later ones, so a destination is
// never the source of a later move; within a batch of moves all sources are
// read before the first destination is written.  The moves' places are
// looked up once per CTA.
#include "sgmv_device.cuh"
#include "sgmv_spec.h"

namespace sgmv {
namespace {

constexpr int kCommitThreads = 256;
constexpr int kCommitBatch = 4;  // moves whose loads are in flight together
static_assert(kCommitThreads >= SGMV_TREE_MAX_NODES, "one path entry per thread");

// Grid: x = pieces of all layers of k and v, y = sequence.
__global__ void __launch_bounds__(kCommitThreads, 6)
    sgmv_commit_kernel(const __grid_constant__ sgmv_cache_commit_args a, int *err) {
    __shared__ int64_t s_from[SGMV_TREE_MAX_NODES], s_to[SGMV_TREE_MAX_NODES];
    __shared__ int s_first_bad;
    pdl_wait();
    pdl_trigger();
    const int tid = threadIdx.x, pieces = a.Hkv * (a.D / 8);
    const int64_t u = (int64_t)blockIdx.x * kCommitThreads + tid, kv = u / pieces;
    const int piece = (int)(u - kv * pieces), head = piece / (a.D / 8);
    const bool mine = kv < 2 * (int64_t)a.layers;
    uint16_t *const base = static_cast<uint16_t *>((kv & 1) ? a.v_cache : a.k_cache) + (kv >> 1) * a.cache_layer +
                           head * a.cache_head + (piece - head * (a.D / 8)) * 8;
    for (int b = blockIdx.y; b < a.B; b += gridDim.y) {
        const int32_t *path = a.path + (int64_t)b * a.max_path, *table = a.block_table + b * a.table_row;
        // the first entries of the path are read beside its length
        const int early = tid < a.max_path ? path[tid] : 0, early_before = tid > 0 && tid < a.max_path ? path[tid - 1] : -1;
        const int64_t prefix = a.prefix_lens[b];
        const int n = a.count[b];
        const bool report = tid == 0 && blockIdx.x == 0;
        if (n < 0 || n > a.max_path || n > SGMV_TREE_MAX_NODES || prefix < 0) {
            if (report) set_error(err, kErrBadIndex);
            continue;
        }
        // element offset of token position j, or -1
        auto place = [&](int64_t j) -> int64_t {
            const int64_t pg = j / a.block_size;
            if (pg >= a.max_blocks) return -1;
            const int32_t block = table[pg];
            if (block < 0 || block >= a.num_blocks) return -1;
            return block * a.cache_block + (j - pg * a.block_size) * a.cache_token;
        };
        if (tid == 0) s_first_bad = n;
        __syncthreads();
        if (const int d = tid; d < n) {
            const int node = early, before = early_before;
            int64_t from = -1, to = -1;
            bool good = node > before && node < SGMV_TREE_MAX_NODES;  // an ascending path
            if (good && node != d) {
                from = place(prefix + node);
                to = place(prefix + d);
                good = from >= 0 && to >= 0;
            }
            s_from[d] = from;
            s_to[d] = to;
            if (!good) atomicMin(&s_first_bad, d);
        }
        __syncthreads();
        const int moves = s_first_bad;  // the path up to its first bad entry
        if (moves < n && report) set_error(err, kErrBadIndex);
        if (mine) {
            for (int d0 = 0; d0 < moves; d0 += kCommitBatch) {
                uint4 val[kCommitBatch];
#pragma unroll
                for (int e = 0; e < kCommitBatch; ++e)
                    if (d0 + e < moves && s_from[d0 + e] >= 0)
                        val[e] = *reinterpret_cast<const uint4 *>(base + s_from[d0 + e]);
#pragma unroll
                for (int e = 0; e < kCommitBatch; ++e)
                    if (d0 + e < moves && s_from[d0 + e] >= 0)
                        *reinterpret_cast<uint4 *>(base + s_to[d0 + e]) = val[e];
            }
        }
        __syncthreads();
    }
}

}  // namespace

int cache_commit_launch(const sgmv_cache_commit_args &a, int *err, cudaStream_t stream) {
    const int64_t units = 2 * (int64_t)a.layers * a.Hkv * (a.D / 8);
    const dim3 grid((unsigned)((units + kCommitThreads - 1) / kCommitThreads), (unsigned)(a.B < 65535 ? a.B : 65535));
    return spec_launch(sgmv_commit_kernel, grid, kCommitThreads, 0, 1, stream, a, err);
}

}  // namespace sgmv
