// sgmv_rope.cu -- rotary positions of q and k, and the append of k and v to
// the paged cache.
//
// One CTA per token: the sines and cosines of the token's pairs are computed
// once, into shared memory, and used by all of its heads.  The angle position *
// inv_freq is a fraction of a turn in 64-bit fixed point, so the product wraps
// modulo one turn by itself and keeps 32 bits of the fraction at any position;
// in fp32 the product alone would lose 2^-24 of the angle, 0.008 rad at
// position 131072.
//
// Bound by memory for many tokens and by the chain position -> sine -> store
// for few: the first rows are requested before the angles are computed, four
// 16- or 32-byte pieces per thread at once.
#include "sgmv_device.cuh"
#include "sgmv_spec.h"

namespace sgmv {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeBatch = 4;  // pieces in flight per thread

enum RopeMode : int {
    kHalves = 0,       // pairs (i, i + pairs), pairs a multiple of 8: 16-byte vectors
    kInterleaved = 1,  // pairs (2i, 2i + 1): 16-byte vectors
    kScalar = 2,       // pairs (i, i + pairs) of any number: one pair or column at a time
};

struct RopeParams {
    sgmv_rope_args a;
    uint64_t turns[kRopeMaxPairs];  // turns per position of every pair, times 2^64
    int32_t rot, uph;               // pieces that rotate, pieces in all, per head
    uint32_t by_uph, by_vec;        // 2^32 / uph and 2^32 / (D / 8), rounded up; 0: divide by one
};

// u / n for u * n < 2^32, by = 2^32 / n rounded up (0 for n = 1)
__device__ __forceinline__ int quotient(int u, uint32_t by) {
    return by ? (int)__umulhi((uint32_t)u, by) : u;
}

// Pieces of a token: q's heads, then k's, then v's (copied, D / 8 per head).
template <typename T, int MODE>
__global__ void __launch_bounds__(kRopeThreads, 4)
    sgmv_rope_kernel(const __grid_constant__ RopeParams P, int *err) {
    const sgmv_rope_args &a = P.a;
    __shared__ float s_cos[kRopeMaxPairs], s_sin[kRopeMaxPairs];
    const int tid = threadIdx.x, pairs = a.pairs, D = a.D, uph = P.uph, rot = P.rot;
    const int64_t t = blockIdx.x;
    pdl_wait();
    pdl_trigger();
    const int32_t pos = a.positions[t], slot = a.k_cache ? a.slots[t] : -1;
    const int nqk = (a.Hq + a.Hk) * uph;
    const int units = nqk + (a.k_cache ? a.Hk * (D / 8) : 0);

    uint4 x[kRopeBatch], y[kRopeBatch];
    auto load = [&](int u, uint4 &x, uint4 &y) {
        if (u >= nqk) {
            const int h = quotient(u - nqk, P.by_vec), c = (u - nqk - h * (D / 8)) * 8;
            x = *reinterpret_cast<const uint4 *>(static_cast<const T *>(a.v) + t * a.v_token + h * a.v_head + c);
            return;
        }
        const int h = quotient(u, P.by_uph), w = u - h * uph;
        const T *src = h < a.Hq ? static_cast<const T *>(a.q) + t * a.q_token + h * a.q_head
                                : static_cast<const T *>(a.k) + t * a.k_token + (h - a.Hq) * a.k_head;
        if (MODE == kScalar) {
            x.x = *reinterpret_cast<const uint16_t *>(src + (w < rot ? w : w + pairs));
            if (w < rot) y.x = *reinterpret_cast<const uint16_t *>(src + w + pairs);
        } else if (MODE == kHalves && w < rot) {
            x = *reinterpret_cast<const uint4 *>(src + w * 8);
            y = *reinterpret_cast<const uint4 *>(src + w * 8 + pairs);
        } else {
            x = *reinterpret_cast<const uint4 *>(src + (MODE == kHalves ? (w - rot) * 8 + 2 * pairs : w * 8));
        }
    };
#pragma unroll
    for (int e = 0; e < kRopeBatch; ++e)
        if (tid + e * kRopeThreads < units) load(tid + e * kRopeThreads, x[e], y[e]);

    if (tid < pairs) {
        const uint64_t turn = (uint64_t)(int64_t)pos * P.turns[tid];  // modulo one turn
        const float half_turns = (float)(int32_t)(turn >> 32) * 0x1p-31f;
        float sn, cs;
        sincospif(half_turns, &sn, &cs);
        s_cos[tid] = cs * a.scale;
        s_sin[tid] = (a.inverse ? -sn : sn) * a.scale;
    }
    int64_t slot_off = -1;
    if (slot >= 0 && (int64_t)slot < (int64_t)a.num_blocks * a.block_size)
        slot_off = (int64_t)(slot / a.block_size) * a.cache_block + (int64_t)(slot % a.block_size) * a.cache_token;
    else if (slot != -1 && tid == 0)
        set_error(err, kErrBadIndex);
    __syncthreads();

    auto store = [&](int u, uint4 x, uint4 y) {
        if (u >= nqk) {
            const int h = quotient(u - nqk, P.by_vec), c = (u - nqk - h * (D / 8)) * 8;
            if (slot_off >= 0)
                *reinterpret_cast<uint4 *>(static_cast<T *>(a.v_cache) + slot_off + h * a.cache_head + c) = x;
            return;
        }
        int h = quotient(u, P.by_uph);
        const int w = u - h * uph;
        T *dst, *dst2 = nullptr;
        if (h < a.Hq) {
            dst = static_cast<T *>(a.q_out) + t * a.q_out_token + h * a.q_out_head;
        } else {
            h -= a.Hq;
            dst = a.k_out ? static_cast<T *>(a.k_out) + t * a.k_out_token + h * a.k_out_head : nullptr;
            if (slot_off >= 0) dst2 = static_cast<T *>(a.k_cache) + slot_off + h * a.cache_head;
        }
        if (MODE == kScalar) {
            const T xs = *reinterpret_cast<const T *>(&x.x), ys = *reinterpret_cast<const T *>(&y.x);
            if (w < rot) {
                const float p = to_f<T>(xs), q = to_f<T>(ys);
                const T r = from_f<T>(p * s_cos[w] - q * s_sin[w]), s = from_f<T>(p * s_sin[w] + q * s_cos[w]);
                if (dst) dst[w] = r, dst[w + pairs] = s;
                if (dst2) dst2[w] = r, dst2[w + pairs] = s;
            } else {
                if (dst) dst[w + pairs] = xs;
                if (dst2) dst2[w + pairs] = xs;
            }
            return;
        }
        int c = w * 8;
        if (MODE == kHalves && w < rot) {
            T *xs = reinterpret_cast<T *>(&x), *ys = reinterpret_cast<T *>(&y);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float p = to_f<T>(xs[e]), q = to_f<T>(ys[e]);
                xs[e] = from_f<T>(p * s_cos[c + e] - q * s_sin[c + e]);
                ys[e] = from_f<T>(p * s_sin[c + e] + q * s_cos[c + e]);
            }
            if (dst) *reinterpret_cast<uint4 *>(dst + c + pairs) = y;
            if (dst2) *reinterpret_cast<uint4 *>(dst2 + c + pairs) = y;
        } else if (MODE == kHalves) {
            c = (w - rot) * 8 + 2 * pairs;
        } else {
            T *xs = reinterpret_cast<T *>(&x);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = w * 4 + e;
                if (i < pairs) {
                    const float p = to_f<T>(xs[2 * e]), q = to_f<T>(xs[2 * e + 1]);
                    xs[2 * e] = from_f<T>(p * s_cos[i] - q * s_sin[i]);
                    xs[2 * e + 1] = from_f<T>(p * s_sin[i] + q * s_cos[i]);
                }
            }
        }
        if (dst) *reinterpret_cast<uint4 *>(dst + c) = x;
        if (dst2) *reinterpret_cast<uint4 *>(dst2 + c) = x;
    };
    for (int u0 = 0;;) {
#pragma unroll
        for (int e = 0; e < kRopeBatch; ++e)
            if (u0 + tid + e * kRopeThreads < units) store(u0 + tid + e * kRopeThreads, x[e], y[e]);
        u0 += kRopeBatch * kRopeThreads;
        if (u0 >= units) break;
#pragma unroll
        for (int e = 0; e < kRopeBatch; ++e)
            if (u0 + tid + e * kRopeThreads < units) load(u0 + tid + e * kRopeThreads, x[e], y[e]);
    }
}

uint32_t inverse_of(int n) { return n > 1 ? (uint32_t)(((1ull << 32) + n - 1) / n) : 0; }

template <typename T> int launch(const RopeParams &p, int mode, int *err, cudaStream_t stream) {
    const dim3 grid((unsigned)p.a.T);
    switch (mode) {
        case kHalves: return spec_launch(sgmv_rope_kernel<T, kHalves>, grid, kRopeThreads, 0, 1, stream, p, err);
        case kInterleaved:
            return spec_launch(sgmv_rope_kernel<T, kInterleaved>, grid, kRopeThreads, 0, 1, stream, p, err);
        default: return spec_launch(sgmv_rope_kernel<T, kScalar>, grid, kRopeThreads, 0, 1, stream, p, err);
    }
}

}  // namespace

int rope_launch(const sgmv_rope_args &a, const uint64_t *turns, int *err, cudaStream_t stream) {
    RopeParams p;
    p.a = a;
    for (int i = 0; i < a.pairs; ++i) p.turns[i] = turns[i];
    const int mode = a.interleaved ? kInterleaved : a.pairs % 8 == 0 ? kHalves : kScalar, rest = a.D - 2 * a.pairs;
    p.rot = mode == kHalves ? a.pairs / 8 : mode == kInterleaved ? a.D / 8 : a.pairs;
    p.uph = mode == kHalves ? p.rot + rest / 8 : mode == kInterleaved ? p.rot : p.rot + rest;
    p.by_uph = inverse_of(p.uph);
    p.by_vec = inverse_of(a.D / 8);
    return a.dtype == SGMV_F16 ? launch<__half>(p, mode, err, stream) : launch<__nv_bfloat16>(p, mode, err, stream);
}

}  // namespace sgmv
