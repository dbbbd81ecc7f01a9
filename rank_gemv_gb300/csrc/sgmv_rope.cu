// sgmv_rope.cu -- rotary positions of q and k, and the append of k and v to
// the paged cache.
//
// A CTA takes one token after another: the sines and cosines of the token's
// pairs are computed once, into shared memory, and used by all of its heads.  The angle position *
// inv_freq is a fraction of a turn in 64-bit fixed point, so the product wraps
// modulo one turn by itself and keeps 32 bits of the fraction at any position;
// in fp32 the product alone would lose 2^-24 of the angle, 0.008 rad at
// position 131072.
//
// A thread keeps one place in the head and steps over the heads, so that its
// sines and cosines stay in registers.  The rows are requested before the
// angles are computed, two 16- or 32-byte pieces per thread at once.
#include <algorithm>

#include "sgmv_device.cuh"
#include "sgmv_spec.h"

namespace sgmv {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeCtas = 4;   // per SM
constexpr int kRopeBatch = 2;  // pieces of q or k, and of v, in flight per thread

enum RopeMode : int {
    kHalves = 0,       // pairs (i, i + pairs), pairs a multiple of 8: 16-byte vectors
    kInterleaved = 1,  // pairs (2i, 2i + 1), pairs a multiple of 4: 16-byte vectors
    kScalar = 2,       // pairs (i, i + pairs) of any number: one pair or column at a time
    // kInterleaved with a last pair inside a vector, whose other columns are copied (a
    // mode of its own: looking in every vector cost 8192 rows 0.6 of 42 us)
    kInterleavedPart = 3,
};

struct RopeParams {
    sgmv_rope_args a;
    uint64_t turns[kRopeMaxPairs];  // turns per position of every pair, times 2^64
    int32_t rot, uph;               // pieces that rotate, pieces in all, per head
};

// Pieces of a head: the rotating ones, then the copied columns.  Piece w of
// heads h0, h0 + step, ... (q's heads, then k's) is one thread's.
template <typename T, int MODE>
__global__ void __launch_bounds__(kRopeThreads, kRopeCtas)
    sgmv_rope_kernel(const __grid_constant__ RopeParams P, int *err) {
    const sgmv_rope_args &a = P.a;
    constexpr bool kAdjacent = MODE == kInterleaved || MODE == kInterleavedPart;
    constexpr int kAngles = MODE == kHalves ? 8 : kAdjacent ? 4 : 1;  // per piece
    __shared__ __align__(16) float2 s_angles[2][kRopeMaxPairs];  // cosine, sine
    const int tid = threadIdx.x, pairs = a.pairs, D = a.D, uph = P.uph;
    pdl_wait();
    pdl_trigger();
    const int heads = a.Hq + a.Hk, step = kRopeThreads / uph, h0 = tid / uph, w = tid - h0 * uph;
    const bool turns = w < P.rot && (!kAdjacent || w * 4 < pairs);
    // first column of the piece, and of its partners
    const int c = MODE == kScalar ? (w < P.rot ? w : w + pairs)
                                  : (MODE == kHalves && w >= P.rot ? (w - P.rot) * 8 + 2 * pairs : w * 8);
    // v: whole vectors, copied
    const int vph = D / 8, vstep = kRopeThreads / vph, vh0 = tid / vph, vc = (tid - vh0 * vph) * 8;
    const uint64_t per_position = tid < pairs ? P.turns[tid] : 0;
    int32_t next_pos = a.positions[blockIdx.x], next_slot = a.k_cache ? a.slots[blockIdx.x] : -1;
    for (int64_t t = blockIdx.x, buf = 0; t < a.T; t += gridDim.x, buf ^= 1) {
    const int32_t pos = next_pos, slot = next_slot;
    if (t + gridDim.x < a.T) {
        next_pos = a.positions[t + gridDim.x];
        if (a.k_cache) next_slot = a.slots[t + gridDim.x];
    }
    float2 *const s_angle = s_angles[buf];
    const T *const q = static_cast<const T *>(a.q) + t * a.q_token + c;
    const T *const k = static_cast<const T *>(a.k) + t * a.k_token + c;
    const T *const vs = static_cast<const T *>(a.v) + t * a.v_token + vc;

    uint4 x[kRopeBatch], y[kRopeBatch], z[kRopeBatch];
    auto load = [&](int hb, int vb) {
#pragma unroll
        for (int e = 0; e < kRopeBatch; ++e) {
            const int h = hb + e * step;
            if (h0 < step && h < heads) {
                const T *src = h < a.Hq ? q + h * a.q_head : k + (h - a.Hq) * a.k_head;
                if (MODE == kScalar) {
                    x[e].x = *reinterpret_cast<const uint16_t *>(src);
                    if (turns) y[e].x = *reinterpret_cast<const uint16_t *>(src + pairs);
                } else {
                    x[e] = *reinterpret_cast<const uint4 *>(src);
                    if (MODE == kHalves && turns) y[e] = *reinterpret_cast<const uint4 *>(src + pairs);
                }
            }
            const int v = vb + e * vstep;
            if (a.k_cache && vh0 < vstep && v < a.Hk)
                z[e] = *reinterpret_cast<const uint4 *>(vs + v * a.v_head);
        }
    };
    load(h0, vh0);

    if (tid < pairs) {
        const float2 u = rotary_angle(per_position, pos);
        s_angle[tid] = make_float2(u.x * a.scale, (a.inverse ? -u.y : u.y) * a.scale);
    }
    int64_t slot_off = -1;
    if (slot >= 0 && (int64_t)slot < (int64_t)a.num_blocks * a.block_size)
        slot_off = (int64_t)(slot / a.block_size) * a.cache_block + (int64_t)(slot % a.block_size) * a.cache_token;
    else if (slot != -1 && tid == 0)
        set_error(err, kErrBadIndex);
    __syncthreads();
    // this piece's angles (an interleaved vector may hold columns past the last
    // pair: those are left as they are below, and their angles are not used)
    float2 r[kAngles];
    if (turns) {
#pragma unroll
        for (int e = 0; e < kAngles; ++e) r[e] = s_angle[w * kAngles + e];
    }
    T *const qo = static_cast<T *>(a.q_out) + t * a.q_out_token + c;
    T *const ko = a.k_out ? static_cast<T *>(a.k_out) + t * a.k_out_token + c : nullptr;
    T *const kc = slot_off >= 0 ? static_cast<T *>(a.k_cache) + slot_off + c : nullptr;
    T *const vo = slot_off >= 0 ? static_cast<T *>(a.v_cache) + slot_off + vc : nullptr;
    auto put = [&](T *dst, const uint4 &x, const uint4 &y) {
        if (MODE == kScalar) {
            *reinterpret_cast<uint16_t *>(dst) = (uint16_t)x.x;
            if (turns) *reinterpret_cast<uint16_t *>(dst + pairs) = (uint16_t)y.x;
        } else {
            *reinterpret_cast<uint4 *>(dst) = x;
            if (MODE == kHalves && turns) *reinterpret_cast<uint4 *>(dst + pairs) = y;
        }
    };
    auto store = [&](int hb, int vb) {
#pragma unroll
        for (int e = 0; e < kRopeBatch; ++e) {
            const int h = hb + e * step;
            if (h0 < step && h < heads) {
                if (turns) {
                    uint32_t *const xs = reinterpret_cast<uint32_t *>(&x[e]), *const ys = reinterpret_cast<uint32_t *>(&y[e]);
                    if (MODE == kScalar) {
                        const float p = to_f<T>(*reinterpret_cast<const T *>(xs)), q = to_f<T>(*reinterpret_cast<const T *>(ys));
                        xs[0] = pack2<T>(p * r[0].x - q * r[0].y, 0.f);
                        ys[0] = pack2<T>(p * r[0].y + q * r[0].x, 0.f);
                    } else if (kAdjacent) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            float p, q;
                            unpack2<T>(xs[i], p, q);
                            const uint32_t turned = pack2<T>(p * r[i % kAngles].x - q * r[i % kAngles].y,
                                                             p * r[i % kAngles].y + q * r[i % kAngles].x);
                            // (a select: cosine 1 and sine 0 would make NaN of an infinity's neighbour)
                            if (MODE == kInterleaved || w * 4 + i < pairs) xs[i] = turned;
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float2 r0 = r[2 * i % kAngles], r1 = r[(2 * i + 1) % kAngles];
                            float p0, p1, q0, q1;
                            unpack2<T>(xs[i], p0, p1);
                            unpack2<T>(ys[i], q0, q1);
                            xs[i] = pack2<T>(p0 * r0.x - q0 * r0.y, p1 * r1.x - q1 * r1.y);
                            ys[i] = pack2<T>(p0 * r0.y + q0 * r0.x, p1 * r1.y + q1 * r1.x);
                        }
                    }
                }
                if (h < a.Hq) {
                    put(qo + h * a.q_out_head, x[e], y[e]);
                } else {
                    if (ko) put(ko + (h - a.Hq) * a.k_out_head, x[e], y[e]);
                    if (kc) put(kc + (h - a.Hq) * a.cache_head, x[e], y[e]);
                }
            }
            const int v = vb + e * vstep;
            if (vo && vh0 < vstep && v < a.Hk) *reinterpret_cast<uint4 *>(vo + v * a.cache_head) = z[e];
        }
    };
    for (int hb = h0, vb = vh0;;) {
        store(hb, vb);
        hb += kRopeBatch * step;
        vb += kRopeBatch * vstep;
        if (hb >= heads && vb >= a.Hk) break;
        load(hb, vb);
    }
    }  // the next token's angles go to the other buffer: one barrier per token
}

template <typename T> int launch(const RopeParams &p, int mode, int nsm, int *err, cudaStream_t stream) {
    // as many CTAs as fit at once (8192 rows of 48 heads: a CTA per row, with its
    // set-up each time, took 44 us)
    const dim3 grid((unsigned)std::min(p.a.T, kRopeCtas * std::max(1, nsm)));
    switch (mode) {
        case kHalves: return spec_launch(sgmv_rope_kernel<T, kHalves>, grid, kRopeThreads, 0, 1, stream, p, err);
        case kInterleaved:
            return spec_launch(sgmv_rope_kernel<T, kInterleaved>, grid, kRopeThreads, 0, 1, stream, p, err);
        case kInterleavedPart:
            return spec_launch(sgmv_rope_kernel<T, kInterleavedPart>, grid, kRopeThreads, 0, 1, stream, p, err);
        default: return spec_launch(sgmv_rope_kernel<T, kScalar>, grid, kRopeThreads, 0, 1, stream, p, err);
    }
}

}  // namespace

int rope_launch(const sgmv_rope_args &a, const uint64_t *turns, int nsm, int *err, cudaStream_t stream) {
    RopeParams p;
    p.a = a;
    for (int i = 0; i < a.pairs; ++i) p.turns[i] = turns[i];
    const int mode = a.interleaved ? (a.pairs % 4 == 0 ? kInterleaved : kInterleavedPart)
                     : a.pairs % 8 == 0 ? kHalves : kScalar;
    const int rest = a.D - 2 * a.pairs;
    p.rot = a.interleaved ? a.D / 8 : mode == kHalves ? a.pairs / 8 : a.pairs;
    p.uph = a.interleaved ? p.rot : mode == kHalves ? p.rot + rest / 8 : p.rot + rest;
    return a.dtype == SGMV_F16 ? launch<__half>(p, mode, nsm, err, stream)
                                 : launch<__nv_bfloat16>(p, mode, nsm, err, stream);
}

}  // namespace sgmv
