// sgmv_quant_mma.cu -- the tensor-core tree attention over caches of e4m3, one
// scale per KV head for K and one for V.
//
// The scale of K goes into the factor of the scores, that of V into the rows'
// last factor, so the stored values themselves are the tensor cores' operands.
//
// 32 trees of up to 16 over up to 4096 tokens, 32 heads of 128: 140 us, 4.1 TB/s of an
// 8-bit cache (a 16-bit one takes 182).  Bounded by a tile's chain, conversion, product,
// softmax and product, in the two stages that each of an SM's two CTAs has room for; the
// conversions themselves, two values in an instruction that 16 lanes per clock and SM
// make, are 60 us of that.  Where the softmax bounds a 16-bit cache, that is quicker: 8
// trees of 64 over up to 32768 tokens, 64 heads on 8, 434 us against 260 (the conversion
// takes issue slots and a stage); and 128 x 3 rows over up to 2100, 20 heads of 80 on 4, 69
// against 50 (the chain again, where 16-bit tiles have three stages).  One token each of 128
// sequences of up to 8192, 32 heads of 128 on 8: 277 us, 4.5 TB/s (a 16-bit cache 377).
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
