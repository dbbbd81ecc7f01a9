// sgmv_spec.h -- the decoding operators (rotary positions with or without head
// norms, tree attention over 16-bit and e4m3 caches, sampling, verification,
// commit): launchers behind the C ABI and the device helpers they share.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "sgmv.h"
#include "sgmv_device.cuh"

namespace sgmv {

#ifdef __CUDACC__
// Two fp32 values rounded to a 16-bit pair, in one instruction.
template <typename T> __device__ __forceinline__ uint32_t pack2(float a, float b);
template <> __device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
template <> __device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
// Cosine and sine of the angle of a pair at a position; turns: its turns per position,
// modulo one, times 2^64 (the product wraps modulo one turn by itself).
__device__ __forceinline__ float2 rotary_angle(uint64_t turns, int32_t position) {
    const uint64_t turn = (uint64_t)(int64_t)position * turns;
    const float half_turns = (float)(int32_t)(turn >> 32) * 0x1p-31f;
    float sn, cs;
    sincospif(half_turns, &sn, &cs);
    return make_float2(cs, sn);
}
#endif

constexpr int kSpecMaxD = 256;               // widest head
constexpr int kRopeMaxPairs = kSpecMaxD / 2;

// Every launcher returns a cudaError_t value.
// turns[i]: turns per position of pair i, modulo one, times 2^64.
int rope_launch(const sgmv_rope_args &a, const uint64_t *turns, int nsm, int *err,
                cudaStream_t stream);
int tree_attention_launch(const sgmv_tree_attention_args &a, int nsm, int *err,
                          cudaStream_t stream);
// The tensor-core form, for D <= kMmaMaxD.
constexpr int kMmaMaxD = 128;
// Its tokens per tile: 128, or as many whole pages of a multiple of 8 tokens as fit.
inline int32_t tree_tile(int32_t block_size) {
    return block_size > 0 && block_size < 128 && block_size % 8 == 0 ? 128 / block_size * block_size : 128;
}
size_t tree_mma_workspace(int32_t T, int32_t group);
int tree_mma_launch(const sgmv_tree_attention_args &a, int nsm, int *err, cudaStream_t stream);
size_t tree_attention_workspace(int32_t T, int32_t Hq, int32_t Hkv, int32_t D);
int tree_verify_launch(const sgmv_tree_verify_args &a, int nsm, int *err, cudaStream_t stream);
int cache_commit_launch(const sgmv_cache_commit_args &a, int *err, cudaStream_t stream);
int norm_rope_launch(const sgmv_norm_rope_args &a, const uint64_t *turns, int nsm, int *err,
                     cudaStream_t stream);
constexpr int kGradMaxSms = 152;  // of which the gradient's workspace holds sums
size_t norm_rope_grad_workspace(int32_t D);
int norm_rope_grad_launch(const sgmv_norm_rope_grad_args &a, const uint64_t *turns, int nsm,
                          cudaStream_t stream);
int quant_mma_launch(const sgmv_quant_attention_args &a, int nsm, int *err, cudaStream_t stream);
int sample_launch(const sgmv_sample_args &a, int nsm, cudaStream_t stream);

// Records how many kernels the calling thread's last call launched.
void set_launch_count(int n);
// What sgmv_debug_inject_wait_timeout was last given on the calling thread.
int injected_timeout();
// Streaming multiprocessors of the current device.
int device_sms();

// Launches a kernel that may start while its predecessor on the stream ends
// (every kernel here waits for it, griddepcontrol.wait, before its first access).
template <typename... P, typename... A>
int spec_launch(void (*kernel)(P...), dim3 grid, int threads, size_t smem, int cluster,
                cudaStream_t stream, A &&...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attrs[2];
    attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[0].val.programmaticStreamSerializationAllowed = 1;
    int na = 1;
    if (cluster > 1) {
        attrs[na].id = cudaLaunchAttributeClusterDimension;
        attrs[na].val.clusterDim.x = (unsigned)cluster;
        attrs[na].val.clusterDim.y = 1;
        attrs[na].val.clusterDim.z = 1;
        ++na;
    }
    cfg.attrs = attrs;
    cfg.numAttrs = (unsigned)na;
    return (int)cudaLaunchKernelEx(&cfg, kernel, static_cast<A &&>(args)...);
}

}  // namespace sgmv
