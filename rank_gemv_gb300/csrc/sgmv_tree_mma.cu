// sgmv_tree_mma.cu -- the tensor-core tree attention over caches of the queries'
// own type: K and V by TMA where pages allow, else by cp.async.
#include "sgmv_tree_mma.cuh"

namespace sgmv {

// For the batch and every smaller one: fewer sequences or rows may make higher row
// tiles, up to those of a single sequence with all the rows.
size_t tree_mma_workspace(int32_t T, int32_t group) {
    size_t most = 0;
    for (int rt = 8, last = row_tile(T, 1, group); rt <= last; rt *= 2)
        most = std::max(most, kHeadBytes + (size_t)max_ctas(rt) * (sizeof(Cut) + 2u * (size_t)rt * 130u * 4u));
    return most;
}

int tree_mma_launch(const sgmv_tree_attention_args &a, int nsm, int *err, cudaStream_t stream) {
    int rt, ctas;
    MmaParams p = plan_launch(a, nsm, err, &rt, &ctas);
    map_cache(p, a.dtype == SGMV_BF16, a.D, 64, 2, true);
    return launch_row_tile<false>(p, rt, ctas, stream);
}

}  // namespace sgmv
