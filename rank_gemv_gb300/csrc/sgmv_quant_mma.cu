// sgmv_quant_mma.cu -- the tensor-core tree attention over caches of e4m3, one
// scale per KV head for K and one for V.
//
// The scale of K goes into the factor of the scores, that of V into the rows'
// last factor, so the stored values themselves are the tensor cores' operands.
#include "sgmv_tree_mma.cuh"

namespace sgmv {

int quant_mma_launch(const sgmv_quant_attention_args &q, int nsm, int *err, cudaStream_t stream) {
    int rt, ctas;
    MmaParams p = plan_launch(q.attention, nsm, err, &rt, &ctas);
    // as half as many 16-bit columns
    map_cache(p, false, p.a.D / 2, p.a.D / 2, 1, false);
    p.k_scale = q.k_scale;
    p.v_scale = q.v_scale;
    return launch_row_tile<true>(p, rt, ctas, stream);
}

}  // namespace sgmv
