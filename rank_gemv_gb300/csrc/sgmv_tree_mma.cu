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
    const bool bf16 = a.dtype == SGMV_BF16;
    // Boxes are as high as pages allow, for TMA's cost here is per box: at pages of
    // 24 tokens, boxes of 8 filling every tile took 115 us, boxes of 24 and tiles of
    // 120 tokens 109 us (128 sequences of up to 2100 tokens, 4 heads of 80).
    p.tok = tree_tile(a.block_size);
    p.box = p.tok < kTok ? a.block_size : std::gcd(a.block_size, kTok);
    if (p.box >= 8) {
        const cuuint64_t dims[4] = {(cuuint64_t)a.D, (cuuint64_t)a.block_size, (cuuint64_t)a.Hkv,
                                    (cuuint64_t)a.num_blocks};
        const cuuint64_t strides[3] = {(cuuint64_t)a.cache_token * 2u, (cuuint64_t)a.cache_head * 2u,
                                       (cuuint64_t)a.cache_block * 2u};
        const cuuint32_t box[4] = {64, (cuuint32_t)p.box, 1, 1};
        // What L2 fetches around a row of a box is this head's only if the rows of
        // a head are contiguous or as wide; else it is another CTA's (32 x 4 rows over up
        // to 4096 tokens, 32 heads side by side: of 64 columns 142 us with 256 bytes,
        // 122 with 128; of 96 columns 220 with 256, 167 with 64)
        const int row = a.D * 2;
        const CUtensorMapL2promotion fetch =
            a.cache_token == a.D || row % 256 == 0 ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B
            : row % 128 == 0                       ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B
            : row % 64 == 0                        ? CU_TENSOR_MAP_L2_PROMOTION_L2_64B
                                                   : CU_TENSOR_MAP_L2_PROMOTION_NONE;
        if (!tmap_encode(&p.map_k, bf16, 4, a.k_cache, dims, strides, box, true, fetch) ||
            !tmap_encode(&p.map_v, bf16, 4, a.v_cache, dims, strides, box, true, fetch))
            p.box = 0, p.tok = kTok;  // strides that a tensor map cannot hold
    } else {
        p.box = 0;
    }
    return launch_row_tile<false>(p, rt, ctas, stream);
}

}  // namespace sgmv
