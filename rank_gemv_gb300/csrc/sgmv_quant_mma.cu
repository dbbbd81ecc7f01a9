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
    const sgmv_tree_attention_args &a = p.a;
    // Boxes as high as pages and a loading warp's tokens allow, of pairs of columns
    const int own = rt > 64 ? 64 : 32;
    p.box = std::gcd(a.block_size, own);
    if (p.box >= 8) {
        const cuuint64_t dims[4] = {(cuuint64_t)a.D / 2, (cuuint64_t)a.block_size, (cuuint64_t)a.Hkv,
                                    (cuuint64_t)a.num_blocks};
        const cuuint64_t strides[3] = {(cuuint64_t)a.cache_token, (cuuint64_t)a.cache_head, (cuuint64_t)a.cache_block};
        const cuuint32_t box[4] = {(cuuint32_t)a.D / 2, (cuuint32_t)p.box, 1, 1};
        // (L2 fetches as for a 16-bit cache: no wider than a head's rows)
        const CUtensorMapL2promotion fetch = a.cache_token == a.D ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B
                                             : a.D % 128 == 0     ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B
                                             : a.D % 64 == 0      ? CU_TENSOR_MAP_L2_PROMOTION_L2_64B
                                                                  : CU_TENSOR_MAP_L2_PROMOTION_NONE;
        if (!tmap_encode(&p.map_k, false, 4, a.k_cache, dims, strides, box, false, fetch) ||
            !tmap_encode(&p.map_v, false, 4, a.v_cache, dims, strides, box, false, fetch))
            p.box = 0;  // strides that a tensor map cannot hold
    } else {
        p.box = 0;
    }
    p.k_scale = q.k_scale;
    p.v_scale = q.v_scale;
    return launch_row_tile<true>(p, rt, ctas, stream);
}

}  // namespace sgmv
