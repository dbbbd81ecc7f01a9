// sgmv_commit.cu -- the accepted tokens' k and v to their final places in the
// paged cache, in place.
//
// A thread owns one 16-byte piece of a head in one layer of one sequence and
// moves it for every accepted node in ascending order.  The node of depth d
// sits at position >= d, and later nodes at still later ones, so a
// destination is never the source of a later move; within a batch of moves
// all sources are read before the first destination is written.
#include "sgmv_device.cuh"
#include "sgmv_spec.h"

namespace sgmv {
namespace {

constexpr int kCommitThreads = 256;
constexpr int kCommitBatch = 8;  // moves whose loads are in flight together

// Grid: x = pieces of one token's heads, y = 2 * layers (k, v), z = sequence.
__global__ void __launch_bounds__(kCommitThreads)
    sgmv_commit_kernel(const __grid_constant__ sgmv_cache_commit_args a, int *err) {
    pdl_wait();
    pdl_trigger();
    const bool report = threadIdx.x == 0 && blockIdx.x == 0 && blockIdx.y == 0;
    const int pieces = a.Hkv * (a.D / 8);
    const int u = blockIdx.x * kCommitThreads + threadIdx.x;
    for (int b = blockIdx.z; b < a.B; b += gridDim.z) {
        const int64_t prefix = a.prefix_lens[b];
        const int32_t *path = a.path + (int64_t)b * a.max_path;
        const int32_t *table = a.block_table + b * a.table_row;
        int n = a.count[b];
        if (n < 0 || n > a.max_path || prefix < 0) {
            if (report) set_error(err, kErrBadIndex);
            continue;
        }
        if (u >= pieces) continue;
        uint16_t *base = static_cast<uint16_t *>((blockIdx.y & 1) ? a.v_cache : a.k_cache) +
                         (int64_t)(blockIdx.y >> 1) * a.cache_layer +
                         (int64_t)(u / (a.D / 8)) * a.cache_head + (u % (a.D / 8)) * 8;
        // slot of token position j, or null
        auto slot = [&](int64_t j) -> uint4 * {
            const int64_t pg = j / a.block_size;
            if (pg >= a.max_blocks) return nullptr;
            const int32_t block = table[pg];
            if (block < 0 || block >= a.num_blocks) return nullptr;
            return reinterpret_cast<uint4 *>(base + block * a.cache_block +
                                             (j - pg * a.block_size) * a.cache_token);
        };
        int last = -1;
        bool bad = false;
        for (int d0 = 0; d0 < n && !bad; d0 += kCommitBatch) {
            uint4 val[kCommitBatch];
            uint4 *to[kCommitBatch];
#pragma unroll
            for (int e = 0; e < kCommitBatch; ++e) {
                to[e] = nullptr;
                const int d = d0 + e;
                if (d >= n || bad) continue;
                const int node = path[d];
                if (node <= last || node >= SGMV_TREE_MAX_NODES) {  // not an ascending path
                    bad = true;
                    continue;
                }
                last = node;
                if (node == d) continue;
                const uint4 *from = slot(prefix + node);
                uint4 *dst = slot(prefix + d);
                if (!from || !dst) {
                    bad = true;
                    continue;
                }
                val[e] = *from;
                to[e] = dst;
            }
#pragma unroll
            for (int e = 0; e < kCommitBatch; ++e)
                if (to[e]) *to[e] = val[e];
        }
        if (bad && report) set_error(err, kErrBadIndex);
    }
}

}  // namespace

int cache_commit_launch(const sgmv_cache_commit_args &a, int nsm, int *err, cudaStream_t stream) {
    const int pieces = a.Hkv * (a.D / 8);
    const dim3 grid((unsigned)((pieces + kCommitThreads - 1) / kCommitThreads),
                    (unsigned)(2 * a.layers), (unsigned)(a.B < 65535 ? a.B : 65535));
    return spec_launch(sgmv_commit_kernel, grid, kCommitThreads, 0, 1, stream, a, err);
}

}  // namespace sgmv
