// sgmv_rope.cu -- rotary positions of q and k, and the append of k and v to
// the paged cache.
//
// One CTA per token (several along y when there are few tokens): the sines
// and cosines of the token's pairs are computed once, into shared memory, and
// used by all of its heads.  The angle position * inv_freq is a fraction of a
// turn in 64-bit fixed point, so the product wraps modulo one turn by itself
// and keeps 32 bits of the fraction at any position; in fp32 the product
// alone would lose 2^-24 of the angle, 0.008 rad at position 131072.
#include "sgmv_device.cuh"
#include "sgmv_spec.h"

namespace sgmv {
namespace {

constexpr int kRopeThreads = 256;

struct RopePhases {
    uint64_t f[kRopeMaxPairs];
};

// Work items of a token: units of 16 bytes (scalar half pairs: of one pair or
// one copied element), q's heads first, then k's, then v's (copied).
template <typename T>
__global__ void __launch_bounds__(kRopeThreads)
    sgmv_rope_kernel(const __grid_constant__ sgmv_rope_args a, const __grid_constant__ RopePhases ph,
                     int *err) {
    __shared__ float s_cos[kRopeMaxPairs], s_sin[kRopeMaxPairs];
    const int tid = threadIdx.x, t = blockIdx.x;
    pdl_wait();
    pdl_trigger();
    const int pairs = a.pairs, D = a.D;
    const int32_t pos = a.positions[t];
    if (tid < pairs) {
        const uint64_t turn = (uint64_t)(int64_t)pos * ph.f[tid];  // modulo one turn
        const float half_turns = (float)(int32_t)(turn >> 32) * 0x1p-31f;
        float sn, cs;
        sincospif(half_turns, &sn, &cs);
        s_cos[tid] = cs * a.scale;
        s_sin[tid] = (a.inverse ? -sn : sn) * a.scale;
    }
    int64_t slot_off = -1;
    if (a.k_cache) {
        const int32_t slot = a.slots[t];
        if (slot >= 0 && (int64_t)slot < (int64_t)a.num_blocks * a.block_size)
            slot_off = (int64_t)(slot / a.block_size) * a.cache_block +
                       (int64_t)(slot % a.block_size) * a.cache_token;
        else if (slot != -1 && tid == 0 && blockIdx.y == 0)
            set_error(err, kErrBadIndex);
    }
    __syncthreads();
    const int mode = a.interleaved ? 1 : pairs % 8 == 0 ? 0 : 2;
    // units per rotated head: half pairs in 16-byte vectors, then the copied
    // columns; interleaved: every 16-byte vector; scalar: pairs, then columns
    const int rot = mode == 0 ? pairs / 8 : mode == 1 ? D / 8 : pairs;
    const int uph = mode == 0 ? rot + (D - 2 * pairs) / 8 : mode == 1 ? rot : rot + (D - 2 * pairs);
    const int nqk = (a.Hq + a.Hk) * uph;
    const int nv = slot_off >= 0 ? a.Hk * (D / 8) : 0;
    for (int u = blockIdx.y * kRopeThreads + tid; u < nqk + nv; u += gridDim.y * kRopeThreads) {
        if (u >= nqk) {
            const int h = (u - nqk) / (D / 8), c = (u - nqk) % (D / 8) * 8;
            const T *src = static_cast<const T *>(a.v) + t * a.v_token + h * a.v_head + c;
            *reinterpret_cast<uint4 *>(static_cast<T *>(a.v_cache) + slot_off + h * a.cache_head + c) =
                *reinterpret_cast<const uint4 *>(src);
            continue;
        }
        int h = u / uph;
        const int w = u - h * uph;
        const T *src;
        T *dst, *dst2 = nullptr;
        if (h < a.Hq) {
            src = static_cast<const T *>(a.q) + t * a.q_token + h * a.q_head;
            dst = static_cast<T *>(a.q_out) + t * a.q_out_token + h * a.q_out_head;
        } else {
            h -= a.Hq;
            src = static_cast<const T *>(a.k) + t * a.k_token + h * a.k_head;
            dst = a.k_out ? static_cast<T *>(a.k_out) + t * a.k_out_token + h * a.k_out_head : nullptr;
            if (slot_off >= 0) dst2 = static_cast<T *>(a.k_cache) + slot_off + h * a.cache_head;
        }
        if (mode == 2) {
            if (w < pairs) {
                const float x = to_f<T>(src[w]), y = to_f<T>(src[w + pairs]);
                const T p = from_f<T>(x * s_cos[w] - y * s_sin[w]);
                const T q = from_f<T>(x * s_sin[w] + y * s_cos[w]);
                if (dst) dst[w] = p, dst[w + pairs] = q;
                if (dst2) dst2[w] = p, dst2[w + pairs] = q;
            } else {
                const int c = w + pairs;
                const T p = src[c];
                if (dst) dst[c] = p;
                if (dst2) dst2[c] = p;
            }
        } else if (mode == 0 && w < rot) {
            const int c = w * 8;
            float x[8], y[8], p[8], q[8];
            load8<T>(src + c, x);
            load8<T>(src + c + pairs, y);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                p[e] = x[e] * s_cos[c + e] - y[e] * s_sin[c + e];
                q[e] = x[e] * s_sin[c + e] + y[e] * s_cos[c + e];
            }
            if (dst) store8<T>(dst + c, p), store8<T>(dst + c + pairs, q);
            if (dst2) store8<T>(dst2 + c, p), store8<T>(dst2 + c + pairs, q);
        } else {
            const int c = mode == 0 ? (w - rot) * 8 + 2 * pairs : w * 8;
            uint4 r = *reinterpret_cast<const uint4 *>(src + c);
            if (mode == 1 && c < 2 * pairs) {
                T *x = reinterpret_cast<T *>(&r);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int i = c / 2 + e;
                    if (i < pairs) {
                        const float p = to_f<T>(x[2 * e]), q = to_f<T>(x[2 * e + 1]);
                        x[2 * e] = from_f<T>(p * s_cos[i] - q * s_sin[i]);
                        x[2 * e + 1] = from_f<T>(p * s_sin[i] + q * s_cos[i]);
                    }
                }
            }
            if (dst) *reinterpret_cast<uint4 *>(dst + c) = r;
            if (dst2) *reinterpret_cast<uint4 *>(dst2 + c) = r;
        }
    }
}

}  // namespace

int rope_launch(const sgmv_rope_args &a, const uint64_t *phase, int nsm, int *err,
                cudaStream_t stream) {
    RopePhases ph;
    for (int i = 0; i < a.pairs; ++i) ph.f[i] = phase[i];
    const dim3 grid((unsigned)a.T, 1, 1);
    return a.dtype == SGMV_F16
               ? spec_launch(sgmv_rope_kernel<__half>, grid, kRopeThreads, 0, 1, stream, a, ph, err)
               : spec_launch(sgmv_rope_kernel<__nv_bfloat16>, grid, kRopeThreads, 0, 1, stream, a,
                             ph, err);
}

}  // namespace sgmv
