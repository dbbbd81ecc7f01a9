// sgmv_norm_rope.cu -- norms of queries and keys for each head, the rotary
// positions and the append to the cache (16-bit or e4m3) in one pass; and the
// gradient of norms and rotation.
//
// One (token, head) is an item, its columns one group of G lanes': with
//   r = (mean x^2 + eps)^-1/2,  y = scale R(pos) (w * x * r),
// a lane holds the pairs that turn together, so that a row is read once, summed
// over the group by shuffles, turned in registers and written once to each of its
// places.  Items of q, k and v lie on one line, t * (Hq + 2 Hk) + head, of which
// every CTA takes an equal contiguous part; the angles of kChunk tokens at a time
// are computed into shared memory and used by all their heads.  8192 rows of 32 + 8 heads of 128 to an
// e4m3 cache: 47 us, 184 MB at 3.9 TB/s; bounded by the instructions (some 370 per warp and
// 512 columns, the issue slots 68 % busy) in front of the memory: a plain copy of as many
// bytes takes 35 us.  (Loads under a condition, one vector per lane: 69 us; fp32 operations
// one at a time: 50.)
//
// Gradient: with g = scale R^T dy, xh = r x, h = w * g,
//   dx = r (h - xh mean(h * xh)),   dw = sum over rows of g * xh.
// A lane adds up its columns of dw in registers over all its items, a CTA then its
// groups' in shared memory, in order; a second kernel adds the CTAs' sums, in order
// too, so the result is the same in every run.  A CTA has rows of q or of k only.  8192
// rows of 32 + 8 heads of 128: 72 us, 252 MB at 3.5 TB/s (a plain copy: 45); bounded by
// latency, as the sums' registers leave room for 512 threads on an SM, with 32 KB of rows
// under way.  With few KV heads k's CTAs set the time, whose chunks of 8 tokens leave groups
// idle: 32 + 2 heads 120 us, 32 + 1 heads 209.
#include <cuda_fp8.h>

#include <algorithm>

#include "sgmv_device.cuh"
#include "sgmv_spec.h"

namespace sgmv {
namespace {

constexpr int kNormThreads = 256;
constexpr int kNormCtas = 3;  // per SM
constexpr int kGradCtas = 2;  // the gradient's, which holds more
constexpr int kChunk = 8;     // tokens whose angles are held

enum NormMode : int {
    kHalves = 0,       // pairs (i, i + pairs), pairs a multiple of 8: a lane has two vectors
    kInterleaved = 1,  // pairs (2i, 2i + 1): a lane has two vectors side by side
    kGather = 2,       // pairs (i, i + pairs) of any number: one vector, partners read singly
};

struct NormParams {
    sgmv_norm_rope_args a;
    uint64_t turns[kRopeMaxPairs];
    int32_t rot, uph;  // lanes of a group whose columns turn, lanes with columns
    float inv_d;
};
struct GradParams {
    sgmv_norm_rope_grad_args a;
    uint64_t turns[kRopeMaxPairs];
    int32_t rot, uph;
    float inv_d;
    int32_t ctas_q;  // CTAs with rows of q; the others have rows of k
    float *part;     // [CTA][D]
};

// Where a lane's columns are: [c, c + 8), and [d, d + 8) if it has a second vector.
template <int MODE> struct Columns {
    int c, d;
    bool here, turns, second;
    __device__ __forceinline__ Columns(int w, int rot, int uph, int pairs, int D) {
        here = w < uph;
        turns = w < rot;
        c = MODE == kInterleaved ? w * 16 : MODE == kHalves && !turns ? (w - rot) * 8 + 2 * pairs : w * 8;
        d = MODE == kInterleaved ? c + 8 : c + pairs;
        second = here && (MODE == kInterleaved ? d < D : MODE == kHalves && turns);
    }
    // What was read as the second vector: zeros, if an interleaved lane has none.
    __device__ __forceinline__ uint4 rest(const uint4 &v) const {
        return MODE == kInterleaved && !second ? make_uint4(0, 0, 0, 0) : v;
    }
    // The sum of the lane's own columns, from those of x and y (see Lane).
    __device__ __forceinline__ float own(float2 x, float2 y) const {
        return !here ? 0.f : MODE == kInterleaved || second ? (x.x + x.y) + (y.x + y.y) : x.x + x.y;
    }
};

// Token and head of an item, and of the one `by` items on, without a division each time.
struct Walk {
    int t, h, heads, dt, dh;
    __device__ __forceinline__ Walk(int i, int heads_, int by) : heads(heads_) {
        dt = by / heads;
        dh = by - dt * heads;
        to(i);
    }
    __device__ __forceinline__ void to(int i) {
        t = i / heads;
        h = i - t * heads;
    }
    __device__ __forceinline__ void step() {
        t += dt;
        h += dh;
        if (h >= heads) h -= heads, ++t;
    }
};

template <int G> __device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Two fp32 operations in one instruction, each rounded as alone: these kernels are bound by
// their instructions as much as by memory.
__device__ __forceinline__ uint64_t bits2(float2 a) {
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a.x), "f"(a.y));
    return v;
}
__device__ __forceinline__ float2 floats2(uint64_t v) {
    float2 a;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a.x), "=f"(a.y) : "l"(v));
    return a;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    uint64_t v;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(bits2(a)), "l"(bits2(b)));
    return floats2(v);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    uint64_t v;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(v) : "l"(bits2(a)), "l"(bits2(b)), "l"(bits2(c)));
    return floats2(v);
}
__device__ __forceinline__ float2 both(float a) { return make_float2(a, a); }
__device__ __forceinline__ float2 minus(float2 a) { return make_float2(-a.x, -a.y); }

// A lane's columns in fp32: x and y are partners.  kHalves: its two vectors; kInterleaved: the
// first and the second columns of its eight pairs; kGather: its vector, and the partners.
struct Lane {
    float2 x[4], y[4];
};
template <typename T, int MODE> __device__ __forceinline__ void spread(const uint4 &u, const uint4 &v, Lane &l) {
    const uint32_t w[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (MODE == kInterleaved) {
            unpack2<T>(w[2 * i], l.x[i].x, l.y[i].x);
            unpack2<T>(w[2 * i + 1], l.x[i].y, l.y[i].y);
        } else {
            unpack2<T>(w[i], l.x[i].x, l.x[i].y);
            unpack2<T>(w[4 + i], l.y[i].x, l.y[i].y);
        }
    }
}
// Values j of the two vectors, in the columns' order.
template <int MODE> __device__ __forceinline__ float2 two_of(const Lane &l, int j) {
    if (MODE != kInterleaved) return j < 4 ? l.x[j] : l.y[j - 4];
    return j & 1 ? make_float2(l.x[j / 2].y, l.y[j / 2].y) : make_float2(l.x[j / 2].x, l.y[j / 2].x);
}
template <typename T, int MODE> __device__ __forceinline__ uint4 vector_of(const Lane &l, int which) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 v = two_of<MODE>(l, 4 * which + j);
        w[j] = pack2<T>(v.x, v.y);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
// Eight values of e4m3: beyond 448 the largest, NaN as NaN.
template <int MODE> __device__ __forceinline__ uint2 bytes_of(const Lane &l, int which) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = __nv_cvt_float2_to_fp8x2(two_of<MODE>(l, 4 * which + j), __NV_SATFINITE, __NV_E4M3);
    return make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
}

// The angles of kChunk tokens, scale included.
struct Angles {
    float c[kChunk][kRopeMaxPairs], s[kChunk][kRopeMaxPairs];
};
__device__ __forceinline__ void chunk_angles(Angles &to, const int32_t *positions, const uint64_t *turns, int64_t t0,
                                             int n, int pairs, float scale) {
    for (int e = threadIdx.x; e < n * pairs; e += kNormThreads) {
        const int k = e / pairs, i = e - k * pairs;
        const float2 cs = rotary_angle(turns[i], positions[t0 + k]);
        to.c[k][i] = cs.x * scale;
        to.s[k][i] = cs.y * scale;
    }
}

// Turns the lane's columns by the angles of its token, or back.
template <int MODE, bool BACK>
__device__ __forceinline__ void turn(const Columns<MODE> &col, const Angles &angles, int token, int pairs, Lane &l) {
    const float *const c = angles.c[token], *const s = angles.s[token];
    if (MODE == kGather) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int j = col.c + i;
            if (j >= 2 * pairs) break;
            const bool second = j >= pairs;
            const int k = second ? j - pairs : j;
            float &x = i & 1 ? l.x[i / 2].y : l.x[i / 2].x;
            const float y = i & 1 ? l.y[i / 2].y : l.y[i / 2].x;
            x = x * c[k] + y * (BACK != second ? s[k] : -s[k]);
        }
        return;
    }
    const int first = MODE == kInterleaved ? col.c / 2 : col.c;  // of the lane's pairs
    if (MODE == kHalves ? !col.turns : first + 8 > pairs) {
        // (columns behind the last pair stay: the angle zero would make NaN of an infinity's partner)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (MODE == kInterleaved && first + i < pairs) {
                float &x = i & 1 ? l.x[i / 2].y : l.x[i / 2].x, &y = i & 1 ? l.y[i / 2].y : l.y[i / 2].x;
                const float cc = c[first + i], ss = BACK ? -s[first + i] : s[first + i], a = x;
                x = a * cc - y * ss;
                y = a * ss + y * cc;
            }
        return;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float4 cc = *reinterpret_cast<const float4 *>(c + first + 4 * i);
        const float4 ss = *reinterpret_cast<const float4 *>(s + first + 4 * i);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float2 c2 = e ? make_float2(cc.z, cc.w) : make_float2(cc.x, cc.y);
            const float2 s0 = e ? make_float2(ss.z, ss.w) : make_float2(ss.x, ss.y);
            const float2 s2 = BACK ? minus(s0) : s0;
            const float2 a = l.x[2 * i + e], b = l.y[2 * i + e];
            l.x[2 * i + e] = fma2(a, c2, minus(mul2(b, s2)));
            l.y[2 * i + e] = fma2(a, s2, mul2(b, c2));
        }
    }
}
// Column of the partner of column j, or j itself.
__device__ __forceinline__ int partner_of(int j, int pairs) {
    return j < pairs ? j + pairs : j < 2 * pairs ? j - pairs : j;
}

template <typename T, int MODE, int G, bool Q8>
__global__ void __launch_bounds__(kNormThreads, kNormCtas)
    sgmv_norm_rope_kernel(const __grid_constant__ NormParams P, int *err) {
    const sgmv_rope_args &a = P.a.rope;
    constexpr int kGroups = kNormThreads / G;
    constexpr bool kTwo = MODE != kGather;
    __shared__ __align__(16) Angles s_angles[2];
    const int g = threadIdx.x / G, pairs = a.pairs;
    const Columns<MODE> col(threadIdx.x % G, P.rot, P.uph, pairs, a.D);
    const bool append = a.k_cache != nullptr;
    const int heads = a.Hq + a.Hk + (append ? a.Hk : 0);
    pdl_wait();
    pdl_trigger();
    const int all = a.T * heads, own = (all + (int)gridDim.x - 1) / (int)gridDim.x;
    const int i0 = min(all, own * (int)blockIdx.x), i1 = min(all, i0 + own);
    // An item's rows, and what is read of them.  No load stands under a condition (behind the
    // last item its rows are read again, lanes without columns read others'): its
    // answer would be waited for where the branches meet.
    struct Item {
        int64_t t;
        int h;
        uint4 x, y;
        int32_t slot;
    };
    const int c_at = col.here ? col.c : 0, d_at = col.second ? col.d : c_at;
    const int32_t *const slots = append ? a.slots : a.positions;
    Walk walk(i0 + g, heads, kGroups), end(i1 - 1, heads, kGroups);
    auto fetch = [&](int i, Item &m) {
        m.t = i < i1 ? walk.t : end.t;
        m.h = i < i1 ? walk.h : end.h;
        const bool is_q = m.h < a.Hq, is_v = m.h >= a.Hq + a.Hk;
        const int h = m.h - (is_q ? 0 : is_v ? a.Hq + a.Hk : a.Hq);
        const T *const src = static_cast<const T *>(is_q ? a.q : is_v ? a.v : a.k) +
                             m.t * (is_q ? a.q_token : is_v ? a.v_token : a.k_token) +
                             h * (is_q ? a.q_head : is_v ? a.v_head : a.k_head);
        m.x = *reinterpret_cast<const uint4 *>(src + c_at);
        if (kTwo) m.y = *reinterpret_cast<const uint4 *>(src + d_at);
        if (MODE == kGather) {
            uint16_t p[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) p[e] = reinterpret_cast<const uint16_t *>(src)[partner_of(c_at + e, pairs)];
            m.y = make_uint4(p[0] | p[1] << 16, p[2] | p[3] << 16, p[4] | p[5] << 16, p[6] | p[7] << 16);
        }
        m.slot = slots[m.t];
    };
    // the weights of this lane's columns
    uint4 wq[2] = {}, wk[2] = {};
    auto weights = [&](const void *w, uint4 (&to)[2]) {
        if (!w || !col.here) return;
        const T *const src = static_cast<const T *>(w);
        to[0] = *reinterpret_cast<const uint4 *>(src + col.c);
        if (col.second) to[1] = *reinterpret_cast<const uint4 *>(src + col.d);
        if (MODE == kGather)
            for (int e = 0; e < 8; ++e)
                reinterpret_cast<T *>(&to[1])[e] = src[partner_of(col.c + e, pairs)];
    };
    if (i0 >= i1) return;
    Item next;
    fetch(i0 + g, next);
    weights(P.a.q_weight, wq);
    weights(P.a.k_weight, wk);
    int buf = 0;
    for (int c0 = i0; c0 < i1; buf ^= 1) {
        const int t0 = c0 / heads, c1 = min((int64_t)i1, ((int64_t)t0 + kChunk) * heads);
        chunk_angles(s_angles[buf], a.positions, P.turns, t0, (c1 - 1) / heads - t0 + 1, pairs, a.scale);
        __syncthreads();
        // (whole warps together: the sums are shuffled)
        for (int ib = c0; ib < c1; ib += kGroups) {
            const bool mine = ib + g < c1;
            const Item m = next;
            // the group's next item, in this chunk or the next one
            const int after = ib + g + kGroups;
            if (after < c1) walk.step();
            else walk.to(c1 + g);
            fetch(after < c1 ? after : c1 + g, next);
            if (!__any_sync(0xffffffffu, mine)) continue;
            const bool is_v = mine && m.h >= a.Hq + a.Hk, is_k = mine && m.h >= a.Hq && !is_v;
            Lane l;
            spread<T, MODE>(m.x, col.rest(m.y), l);
            const bool normed = mine && !is_v && (is_k ? P.a.k_weight : P.a.q_weight) != nullptr;
            float2 s2 = both(0.f), t2 = both(0.f);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                s2 = fma2(l.x[e], l.x[e], s2);
                if (kTwo) t2 = fma2(l.y[e], l.y[e], t2);
            }
            const float ss = group_sum<G>(col.own(s2, t2));
            if (MODE == kGather) __syncwarp();  // in place: partners are read before any is written
            if (!mine || !col.here) continue;
            if (normed) {
                const float2 r = both(rsqrtf(ss * P.inv_d + P.a.eps));
                Lane w;
                spread<T, MODE>(is_k ? wk[0] : wq[0], is_k ? wk[1] : wq[1], w);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    l.x[e] = mul2(l.x[e], mul2(r, w.x[e]));
                    l.y[e] = mul2(l.y[e], mul2(r, w.y[e]));
                }
            }
            if (!is_v) turn<MODE, false>(col, s_angles[buf], (int)(m.t - t0), pairs, l);
            auto put16 = [&](T *dst) {
                *reinterpret_cast<uint4 *>(dst + col.c) = vector_of<T, MODE>(l, 0);
                if (col.second) *reinterpret_cast<uint4 *>(dst + col.d) = vector_of<T, MODE>(l, 1);
            };
            if (!is_k && !is_v) {
                put16(static_cast<T *>(a.q_out) + m.t * a.q_out_token + m.h * a.q_out_head);
                continue;
            }
            const int h = m.h - a.Hq - (is_v ? a.Hk : 0);
            if (is_k && a.k_out) put16(static_cast<T *>(a.k_out) + m.t * a.k_out_token + h * a.k_out_head);
            if (!append) continue;
            if (m.slot < 0 || (int64_t)m.slot >= (int64_t)a.num_blocks * a.block_size) {
                if (m.slot != -1) set_error(err, kErrBadIndex);
                continue;
            }
            const int64_t off = (int64_t)(m.slot / a.block_size) * a.cache_block +
                                (int64_t)(m.slot % a.block_size) * a.cache_token + h * a.cache_head;
            if (Q8) {
                uint8_t *const dst = static_cast<uint8_t *>(is_v ? a.v_cache : a.k_cache) + off;
                const float2 f = both(1.f / (is_v ? P.a.v_scale : P.a.k_scale)[h]);
#pragma unroll
                for (int e = 0; e < 4; ++e) l.x[e] = mul2(l.x[e], f), l.y[e] = mul2(l.y[e], f);
                *reinterpret_cast<uint2 *>(dst + col.c) = bytes_of<MODE>(l, 0);
                if (col.second) *reinterpret_cast<uint2 *>(dst + col.d) = bytes_of<MODE>(l, 1);
            } else {
                put16(static_cast<T *>(is_v ? a.v_cache : a.k_cache) + off);
            }
        }
        c0 = c1;
    }  // the next chunk's angles go to the other buffer: one barrier per chunk
}

template <typename T, int MODE, int G>
__global__ void __launch_bounds__(kNormThreads, kGradCtas)
    sgmv_norm_rope_grad_kernel(const __grid_constant__ GradParams P) {
    const sgmv_norm_rope_grad_args &a = P.a;
    constexpr int kGroups = kNormThreads / G;
    constexpr bool kTwo = MODE != kGather;
    __shared__ __align__(16) Angles s_angles[2];
    __shared__ float s_dw[kGroups > 8 ? 8 : kGroups][kSpecMaxD];
    const int g = threadIdx.x / G, pairs = a.pairs;
    const Columns<MODE> col(threadIdx.x % G, P.rot, P.uph, pairs, a.D);
    pdl_wait();
    pdl_trigger();
    const bool is_k = (int)blockIdx.x >= P.ctas_q;
    const int heads = is_k ? a.Hk : a.Hq;
    const int cta = (int)blockIdx.x - (is_k ? P.ctas_q : 0), ctas = is_k ? (int)gridDim.x - P.ctas_q : P.ctas_q;
    const T *const X = static_cast<const T *>(is_k ? a.k : a.q);
    const T *const DY = static_cast<const T *>(is_k ? a.dk_out : a.dq_out);
    T *const DX = static_cast<T *>(is_k ? a.dk : a.dq);
    const T *const W = static_cast<const T *>(is_k ? a.k_weight : a.q_weight);
    const int64_t x_token = is_k ? a.k_token : a.q_token, x_head = is_k ? a.k_head : a.q_head;
    const int64_t dy_token = is_k ? a.dk_out_token : a.dq_out_token, dy_head = is_k ? a.dk_out_head : a.dq_out_head;
    const int64_t dx_token = is_k ? a.dk_token : a.dq_token, dx_head = is_k ? a.dk_head : a.dq_head;
    const int all = a.T * heads, own = (all + ctas - 1) / ctas;
    const int i0 = min(all, own * cta), i1 = min(all, i0 + own);
    struct Item {
        int t, h;
        uint4 x, y, gx, gy;
    };
    // (no load under a condition, as above)
    const int c_at = col.here ? col.c : 0, d_at = col.second ? col.d : c_at;
    const T *const X0 = W ? X : DY;  // x is not read without its weight
    const int64_t x0_token = W ? x_token : dy_token, x0_head = W ? x_head : dy_head;
    Walk walk(i0 + g, heads, kGroups), end(max(i1 - 1, 0), heads, kGroups);
    auto fetch = [&](int i, Item &m) {
        m.t = i < i1 ? walk.t : end.t;
        m.h = i < i1 ? walk.h : end.h;
        const T *const dy = DY + m.t * dy_token + m.h * dy_head, *const x = X0 + m.t * x0_token + m.h * x0_head;
        m.gx = *reinterpret_cast<const uint4 *>(dy + c_at);
        m.x = *reinterpret_cast<const uint4 *>(x + c_at);
        if (kTwo) {
            m.gy = *reinterpret_cast<const uint4 *>(dy + d_at);
            m.y = *reinterpret_cast<const uint4 *>(x + d_at);
        }
        if (MODE == kGather) {
            uint16_t p[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) p[e] = reinterpret_cast<const uint16_t *>(dy)[partner_of(c_at + e, pairs)];
            m.gy = make_uint4(p[0] | p[1] << 16, p[2] | p[3] << 16, p[4] | p[5] << 16, p[6] | p[7] << 16);
        }
    };
    Lane w, dw;  // weights of the lane's columns, and their gradients
#pragma unroll
    for (int e = 0; e < 4; ++e) w.x[e] = w.y[e] = both(1.f), dw.x[e] = dw.y[e] = both(0.f);
    if (W)
        spread<T, MODE>(*reinterpret_cast<const uint4 *>(W + c_at), *reinterpret_cast<const uint4 *>(W + d_at), w);
    Item next = {};
    if (i0 < i1) fetch(i0 + g, next);
    int buf = 0;
    for (int c0 = i0; c0 < i1; buf ^= 1) {
        const int t0 = c0 / heads, c1 = min((int64_t)i1, ((int64_t)t0 + kChunk) * heads);
        chunk_angles(s_angles[buf], a.positions, P.turns, t0, (c1 - 1) / heads - t0 + 1, pairs, a.scale);
        __syncthreads();
        for (int ib = c0; ib < c1; ib += kGroups) {
            const int i = ib + g;
            const bool mine = i < c1;
            const Item m = next;
            if (i + kGroups < c1) walk.step();
            else walk.to(c1 + g);
            fetch(i + kGroups < c1 ? i + kGroups : c1 + g, next);
            if (!__any_sync(0xffffffffu, mine)) continue;
            const bool on = mine && col.here, second = col.second;
            Lane g, x;
            spread<T, MODE>(m.gx, col.rest(m.gy), g);
            spread<T, MODE>(m.x, col.rest(m.y), x);
            const int64_t t = mine ? m.t : t0, h = mine ? m.h : 0;
            if (on) turn<MODE, true>(col, s_angles[buf], (int)(t - t0), pairs, g);
            if (W) {
                // sum x^2, and sum of w g x: then mean(h * xh) = r / D times it
                float2 s2 = both(0.f), d2 = both(0.f), t2 = both(0.f), e2 = both(0.f);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    s2 = fma2(x.x[e], x.x[e], s2);
                    d2 = fma2(mul2(w.x[e], g.x[e]), x.x[e], d2);
                    if (kTwo) {
                        t2 = fma2(x.y[e], x.y[e], t2);
                        e2 = fma2(mul2(w.y[e], g.y[e]), x.y[e], e2);
                    }
                }
                const float ss = group_sum<G>(col.own(s2, t2)), dot = group_sum<G>(col.own(d2, e2));
                const float r = rsqrtf(ss * P.inv_d + a.eps), f = dot * r * P.inv_d * r;
                if (on) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        dw.x[e] = fma2(g.x[e], mul2(x.x[e], both(r)), dw.x[e]);
                        g.x[e] = mul2(both(r), fma2(x.x[e], both(-f), mul2(w.x[e], g.x[e])));
                        if (kTwo) {
                            dw.y[e] = fma2(g.y[e], mul2(x.y[e], both(r)), dw.y[e]);
                            g.y[e] = mul2(both(r), fma2(x.y[e], both(-f), mul2(w.y[e], g.y[e])));
                        }
                    }
                }
            }
            if (on) {
                T *const dx = DX + t * dx_token + h * dx_head;
                *reinterpret_cast<uint4 *>(dx + col.c) = vector_of<T, MODE>(g, 0);
                if (second) *reinterpret_cast<uint4 *>(dx + col.d) = vector_of<T, MODE>(g, 1);
            }
        }
        c0 = c1;
    }
    if (!W) return;
    // the groups' sums, in order: over the warp, then over the eight warps
    float sums[16];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float2 v = two_of<MODE>(dw, j);
        sums[2 * j] = v.x;
        sums[2 * j + 1] = v.y;
    }
#pragma unroll
    for (int e = 0; e < (kTwo ? 16 : 8); ++e)
#pragma unroll
        for (int o = G; o < 32; o <<= 1) sums[e] += __shfl_xor_sync(0xffffffffu, sums[e], o);
    const int warp = threadIdx.x / 32;
    static_assert(kNormThreads / 32 <= 8 && kGroups >= 8, "a row of sums per warp");
    if ((threadIdx.x & 31) < G && col.here) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            s_dw[warp][col.c + e] = sums[e];
            if (col.second) s_dw[warp][col.d + e] = sums[8 + e];
        }
    }
    __syncthreads();
    for (int d = threadIdx.x; d < a.D; d += kNormThreads) {
        float sum = 0.f;
        for (int i = 0; i < kNormThreads / 32; ++i) sum += s_dw[i][d];
        P.part[(int64_t)blockIdx.x * a.D + d] = sum;
    }
}

// dw of a column of q (blockIdx.y 0) or k: the CTAs' sums added up, 32 columns and
// 32 strands a CTA.
__global__ void __launch_bounds__(1024) sgmv_norm_rope_dw_kernel(const float *part, float *dwq, float *dwk, int D,
                                                                 int ctas_q, int ctas) {
    __shared__ double s_sum[32][33];
    pdl_wait();
    pdl_trigger();
    const int d = blockIdx.x * 32 + (threadIdx.x & 31), strand = threadIdx.x >> 5;
    float *const dw = blockIdx.y ? dwk : dwq;
    if (!dw) return;
    double sum = 0.0;
    if (d < D)
        for (int i = (blockIdx.y ? ctas_q : 0) + strand; i < (blockIdx.y ? ctas : ctas_q); i += 32)
            sum += (double)part[(int64_t)i * D + d];
    s_sum[strand][threadIdx.x & 31] = sum;
    __syncthreads();
    if (strand == 0 && d < D) {
        for (int i = 1; i < 32; ++i) sum += s_sum[i][threadIdx.x];
        dw[d] = (float)sum;
    }
}

// Lanes of a group: a power of two that holds the columns.
int lanes(int uph) { return uph <= 4 ? 4 : uph <= 8 ? 8 : uph <= 16 ? 16 : 32; }
int mode_of(int interleaved, int pairs) {
    return interleaved ? kInterleaved : pairs % 8 == 0 ? kHalves : kGather;
}
void places(int mode, int D, int pairs, int32_t *rot, int32_t *uph) {
    *uph = mode == kHalves ? pairs / 8 + (D - 2 * pairs) / 8 : mode == kInterleaved ? (D + 15) / 16 : D / 8;
    *rot = mode == kHalves ? pairs / 8 : *uph;
}

template <typename T, int MODE, int G> int launch(const NormParams &p, int nsm, int *err, cudaStream_t stream) {
    const sgmv_rope_args &a = p.a.rope;
    const int64_t items = (int64_t)a.T * (a.Hq + a.Hk + (a.k_cache ? a.Hk : 0)), groups = kNormThreads / G;
    const dim3 grid((unsigned)std::min<int64_t>((items + groups - 1) / groups, (int64_t)kNormCtas * std::max(1, nsm)));
    return p.a.k_scale
               ? spec_launch(sgmv_norm_rope_kernel<T, MODE, G, true>, grid, kNormThreads, 0, 1, stream, p, err)
               : spec_launch(sgmv_norm_rope_kernel<T, MODE, G, false>, grid, kNormThreads, 0, 1, stream, p, err);
}
template <typename T, int MODE> int launch_lanes(const NormParams &p, int nsm, int *err, cudaStream_t stream) {
    switch (lanes(p.uph)) {
        case 4: return launch<T, MODE, 4>(p, nsm, err, stream);
        case 8: return launch<T, MODE, 8>(p, nsm, err, stream);
        case 16: return launch<T, MODE, 16>(p, nsm, err, stream);
        default: return launch<T, MODE, 32>(p, nsm, err, stream);
    }
}
template <typename T> int launch_mode(const NormParams &p, int mode, int nsm, int *err, cudaStream_t stream) {
    switch (mode) {
        case kHalves: return launch_lanes<T, kHalves>(p, nsm, err, stream);
        case kInterleaved: return launch_lanes<T, kInterleaved>(p, nsm, err, stream);
        default: return launch_lanes<T, kGather>(p, nsm, err, stream);
    }
}

template <typename T, int MODE, int G> int launch_grad(GradParams p, int nsm, cudaStream_t stream) {
    const sgmv_norm_rope_grad_args &a = p.a;
    // CTAs to q and k by their rows
    const int64_t most = (int64_t)kGradCtas * std::min(std::max(1, nsm), kGradMaxSms), groups = kNormThreads / G;
    const int64_t q = ((int64_t)a.T * a.Hq + groups - 1) / groups, k = ((int64_t)a.T * a.Hk + groups - 1) / groups;
    int64_t nq = q, nk = k;
    if (q + k > most) {
        nq = q == 0 ? 0 : std::min(q, std::max<int64_t>(1, most * q / (q + k)));
        nk = k == 0 ? 0 : std::max<int64_t>(1, most - nq);
        if (nq + nk > most) nq = most - nk;
    }
    p.ctas_q = (int)nq;
    if (nq + nk > 0) {  // (no rows: the weights' gradients are zero)
        const int r = spec_launch(sgmv_norm_rope_grad_kernel<T, MODE, G>, dim3((unsigned)(nq + nk)), kNormThreads, 0,
                                  1, stream, p);
        if (r != (int)cudaSuccess) return r;
    }
    if (!a.dq_weight && !a.dk_weight) return (int)cudaSuccess;
    return spec_launch(sgmv_norm_rope_dw_kernel, dim3((unsigned)((a.D + 31) / 32), 2), 1024, 0, 1, stream, p.part,
                       a.dq_weight, a.dk_weight, (int)a.D, (int)nq, (int)(nq + nk));
}
template <typename T, int MODE> int launch_grad_lanes(const GradParams &p, int nsm, cudaStream_t stream) {
    switch (lanes(p.uph)) {
        case 4: return launch_grad<T, MODE, 4>(p, nsm, stream);
        case 8: return launch_grad<T, MODE, 8>(p, nsm, stream);
        case 16: return launch_grad<T, MODE, 16>(p, nsm, stream);
        default: return launch_grad<T, MODE, 32>(p, nsm, stream);
    }
}
template <typename T> int launch_grad_mode(const GradParams &p, int mode, int nsm, cudaStream_t stream) {
    switch (mode) {
        case kHalves: return launch_grad_lanes<T, kHalves>(p, nsm, stream);
        case kInterleaved: return launch_grad_lanes<T, kInterleaved>(p, nsm, stream);
        default: return launch_grad_lanes<T, kGather>(p, nsm, stream);
    }
}

}  // namespace

int norm_rope_launch(const sgmv_norm_rope_args &a, const uint64_t *turns, int nsm, int *err, cudaStream_t stream) {
    NormParams p;
    p.a = a;
    p.inv_d = 1.f / (float)a.rope.D;
    for (int i = 0; i < a.rope.pairs; ++i) p.turns[i] = turns[i];
    const int mode = mode_of(a.rope.interleaved, a.rope.pairs);
    places(mode, a.rope.D, a.rope.pairs, &p.rot, &p.uph);
    return a.rope.dtype == SGMV_F16 ? launch_mode<__half>(p, mode, nsm, err, stream)
                                    : launch_mode<__nv_bfloat16>(p, mode, nsm, err, stream);
}

size_t norm_rope_grad_workspace(int32_t D) { return (size_t)kGradCtas * kGradMaxSms * (size_t)D * 4u; }

int norm_rope_grad_launch(const sgmv_norm_rope_grad_args &a, const uint64_t *turns, int nsm, cudaStream_t stream) {
    GradParams p;
    p.a = a;
    p.part = static_cast<float *>(a.workspace);
    p.inv_d = 1.f / (float)a.D;
    for (int i = 0; i < a.pairs; ++i) p.turns[i] = turns[i];
    const int mode = mode_of(a.interleaved, a.pairs);
    places(mode, a.D, a.pairs, &p.rot, &p.uph);
    return a.dtype == SGMV_F16 ? launch_grad_mode<__half>(p, mode, nsm, stream)
                               : launch_grad_mode<__nv_bfloat16>(p, mode, nsm, stream);
}

}  // namespace sgmv
