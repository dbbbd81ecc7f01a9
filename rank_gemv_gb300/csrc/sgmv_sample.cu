// sgmv_sample.cu -- the next token from logits: temperature, top-k, top-p and
// min-p, drawn from given random numbers; and the filtered distribution itself.
//
// Weights are whole numbers, w = floor(2^38 exp((l - max) / temperature)), so sums
// are exact in 64 bits, the same in any order, and the drawn token does not depend
// on how the vocabulary is divided.  exp is made in integers, to a few units of 2^-38
// (a division of the exponent into 128ths with a table, then three terms of the series).
//
// A cluster of CTAs has a row, each warp one contiguous range of it, staged in
// shared memory as fp32 once; everything else happens on chip.  The filters keep
// the first tokens in order of (logit, index), and what cuts there is found without a
// sort: a histogram of 2048 bins over the logits counts the tokens; the bin where the
// k-th falls, or the bins where the running weight can pass p of the total (the
// weights at a bin's edges bound it from both sides), are looked at again, finer,
// until few tokens are left, which are ranked one against all, or one value, whose
// tokens are counted off by index.  Sums above the cut are exact at every step.
#include <algorithm>

#include "sgmv_device.cuh"
#include "sgmv_spec.h"

namespace sgmv {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kBins = 4 * kThreads;
constexpr int kFew = 256;               // tokens that are ranked one against all
constexpr float kOctaves = 39.f;        // weights below 2^-39 of the largest are zero
constexpr float kSlack = 3e-5f;         // rounding of the weights at bins' edges and of their sums
constexpr int64_t kOne = 1ll << 38, kUnit = 1ll << 24;

// 2^38 2^(j / 128), j = -64 ... 64
__device__ const int64_t kExp2[129] = {
    194368031998ll, 195423431192ll, 196484561098ll, 197551452835ll, 198624137689ll, 199702647115ll,
    200787012741ll, 201877266365ll, 202973439958ll, 204075565666ll, 205183675807ll, 206297802876ll,
    207417979546ll, 208544238664ll, 209676613257ll, 210815136533ll, 211959841877ll, 213110762859ll,
    214267933227ll, 215431386916ll, 216601158044ll, 217777280913ll, 218959790013ll, 220148720020ll,
    221344105800ll, 222545982406ll, 223754385084ll, 224969349268ll, 226190910588ll, 227419104865ll,
    228653968116ll, 229895536552ll, 231143846582ll, 232398934811ll, 233660838046ll, 234929593291ll,
    236205237751ll, 237487808834ll, 238777344152ll, 240073881518ll, 241377458955ll, 242688114688ll,
    244005887152ll, 245330814990ll, 246662937055ll, 248002292412ll, 249348920335ll, 250702860315ll,
    252064152055ll, 253432835475ll, 254808950710ll, 256192538115ll, 257583638263ll, 258982291947ll,
    260388540182ll, 261802424207ll, 263223985481ll, 264653265693ll, 266090306755ll, 267535150807ll,
    268987840221ll, 270448417593ll, 271916925757ll, 273393407775ll, 274877906944ll, 276370466797ll,
    277871131102ll, 279379943866ll, 280896949334ll, 282422191992ll, 283955716566ll, 285497568028ll,
    287047791590ll, 288606432713ll, 290173537103ll, 291749150715ll, 293333319753ll, 294926090673ll,
    296527510181ll, 298137625238ll, 299756483061ll, 301384131122ll, 303020617151ll, 304665989137ll,
    306320295331ll, 307983584243ll, 309655904650ll, 311337305591ll, 313027836374ll, 314727546571ll,
    316436486026ll, 318154704854ll, 319882253439ll, 321619182443ll, 323365542800ll, 325121385721ll,
    326886762695ll, 328661725491ll, 330446326160ll, 332240617034ll, 334044650731ll, 335858480151ll,
    337682158486ll, 339515739215ll, 341359276105ll, 343212823218ll, 345076434909ll, 346950165827ll,
    348834070918ll, 350728205428ll, 352632624901ll, 354547385183ll, 356472542425ll, 358408153079ll,
    360354273909ll, 362310961982ll, 364278274677ll, 366256269686ll, 368245005013ll, 370244538975ll,
    372254930209ll, 374276237669ll, 376308520629ll, 378351838683ll, 380406251753ll, 382471820083ll,
    384548604245ll, 386636665139ll, 388736063997ll,
};

struct SampleShared {
    uint32_t hist[kBins];
    int64_t exp2[129];
    int64_t part[2][3][kWarps], mine[2][3];
    int64_t scan[kWarps];
    float scan_lo[kWarps], scan_hi[kWarps];
    uint32_t scan_n[kWarps];
    float list_l[kFew];
    int32_t list_v[kFew];
    int64_t list_w[kFew];
    uint32_t listed;
    int bin0, bin1;
    uint32_t rank, count;
    float cut_l;
    int32_t cut_v, found;
};

struct SampleParams {
    sgmv_sample_args a;
    int32_t share;   // entries of a warp's range
    int32_t staged;  // the ranges are in shared memory
};

// One zero; finite logits and +inf within +-2^126, so that differences are finite; NaN as -inf.
__device__ __forceinline__ float canonical(float l) {
    return l > -INFINITY ? fminf(fmaxf(l, -0x1p126f), 0x1p126f) + 0.f : -INFINITY;
}
__device__ __forceinline__ void st_peer32(uint32_t addr, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// What a row's weights are made with.
struct Weigh {
    float m, ch, cl;  // largest logit; log2(e) / temperature, in two parts
    const int64_t *table;

    // fp32 exponent, never above zero, descending with l
    __device__ __forceinline__ float rough(float l) const { return (l - m) * ch; }
    __device__ __forceinline__ int64_t operator()(float l) const {
        // l - m = d + e exactly; times log2(e) / temperature: p + q
        const float d = l - m, b = d - l, e = (l - (d - b)) + (-m - b);
        const float p = d * ch;
        if (!(p > -kOctaves)) return 0;
        const float q = fmaf(d, ch, -p) + fmaf(d, cl, e * ch);
        // p = n + j / 128 + g; the magic sums leave whole numbers in the low bits
        const float nm = p + 12582912.f, f = p - (nm - 12582912.f);
        const int n = __float_as_int(nm) - 0x4B400000;
        const float jm = fmaf(f, 128.f, 12582912.f), g = fmaf(jm - 12582912.f, -0.0078125f, f);
        const int j = __float_as_int(jm) - 0x4B400000;
        // in units of 2^-38: z = (g + q) ln 2, then z + z^2 / 2 + z^3 / 6
        const int x = __float2int_rn(g * 0x1p38f) + __float2int_rn(q * 0x1p38f);
        const int z = (int)(((int64_t)x * 1488522236ll) >> 31);
        const int zz = __mulhi(z, z);                          // 2^-44
        const int z3 = (int)(((__mulhi(zz, z) >> 8) * 10923) >> 20);  // z^3 / 6 from 2^-50
        const int s = z + (zz >> 7) + z3;
        const int64_t t = table[j + 64];
        const int64_t w = t + (((int64_t)(int)(t >> 8) * s) >> 30);
        return w >> min(63, -n);
    }
};

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) sgmv_sample_kernel(const __grid_constant__ SampleParams P) {
    const sgmv_sample_args &a = P.a;
    extern __shared__ __align__(16) float staged[];
    __shared__ SampleShared s;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cl = (int)cluster_size(), rank = (int)cluster_rank(), share = P.share;
    const int64_t t = (int64_t)(blockIdx.x / (unsigned)cl);
    pdl_wait();
    pdl_trigger();
    const T *const row = static_cast<const T *>(a.logits) + t * a.logits_row;
    // Entries u = token + skew: vectors at whole multiples are aligned in memory.
    constexpr int kVec = 16 / (int)sizeof(T);
    const int skew = (int)((reinterpret_cast<uintptr_t>(row) / sizeof(T)) % kVec);
    const int u_end = a.V + skew;
    const int u0 = (rank * kWarps + warp) * share;  // this warp's first
    float *const mine = staged + warp * share;
    auto read1 = [&](int u) { return u >= skew && u < u_end ? canonical(to_f<T>(row[u - skew])) : -INFINITY; };
    // four entries of warp w's range
    auto get4 = [&](int i) {
        if (P.staged) {
            const uint4 x = lds128(mine + i);
            return make_float4(__uint_as_float(x.x), __uint_as_float(x.y), __uint_as_float(x.z), __uint_as_float(x.w));
        }
        return make_float4(read1(u0 + i), read1(u0 + i + 1), read1(u0 + i + 2), read1(u0 + i + 3));
    };
    auto get1 = [&](int w, int i) {
        return P.staged ? ldsf(staged + w * share + i) : read1((rank * kWarps + w) * share + i);
    };
    // every entry of this warp, f(logit, token)
    auto each = [&](auto f) {
        for (int i = lane * 4; i < share; i += 128) {
            const float4 x = get4(i);
            const int v = u0 + i - skew;
            f(x.x, v);
            f(x.y, v + 1);
            f(x.z, v + 2);
            f(x.w, v + 3);
        }
    };

    // ---- the cluster's sums ----------------------------------------------------
    int turn = 0;
    // Joins N values of all threads by op(n, x, y); everyone gets the result.  The warps'
    // values stay in part[], the CTAs' in mine[], of the turn before.
    auto join = [&](auto &v, auto op) {
        constexpr int N = sizeof(v) / sizeof(v[0]);
        const int at = turn;
        turn ^= 1;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            for (int o = 16; o > 0; o >>= 1) v[n] = op(n, v[n], (int64_t)__shfl_xor_sync(0xffffffffu, v[n], o));
            if (lane == 0) s.part[at][n][warp] = v[n];
        }
        __syncthreads();
#pragma unroll
        for (int n = 0; n < N; ++n) {
            v[n] = s.part[at][n][0];
            for (int w = 1; w < kWarps; ++w) v[n] = op(n, v[n], s.part[at][n][w]);
            if (tid == 0) s.mine[at][n] = v[n];
        }
        if (cl > 1) {
            cluster_sync();
#pragma unroll
            for (int n = 0; n < N; ++n)
                for (int r = 0; r < cl; ++r) {
                    uint64_t x;
                    asm volatile("ld.shared::cluster.u64 %0, [%1];"
                                 : "=l"(x)
                                 : "r"(peer_addr(&s.mine[at][n], (uint32_t)r))
                                 : "memory");
                    v[n] = r == 0 ? (int64_t)x : op(n, v[n], (int64_t)x);
                }
        }
    };
    auto plus = [](int, int64_t x, int64_t y) { return x + y; };
    // The token where the running sum of f in index order passes `mark`, after a join of
    // f's sums alone (found: it, in every CTA).
    auto locate = [&](auto f, int64_t mark) {
        const int at = turn ^ 1;
        int64_t before = 0, all = 0;
        if (cl > 1) {
            for (int r = 0; r <= rank; ++r) {
                uint64_t x;
                asm volatile("ld.shared::cluster.u64 %0, [%1];"
                             : "=l"(x)
                             : "r"(peer_addr(&s.mine[at][0], (uint32_t)r))
                             : "memory");
                if (r < rank) before += (int64_t)x;
                else all = (int64_t)x;
            }
        } else {
            for (int w = 0; w < kWarps; ++w) all += s.part[at][0][w];
        }
        if (before <= mark && mark < before + all) {  // it is this CTA's
            int w = 0;
            while (w < kWarps - 1 && mark >= before + s.part[at][0][w]) before += s.part[at][0][w++];
            for (int i0 = 0; i0 < share; i0 += kThreads) {
                const int i = i0 + tid, v = (rank * kWarps + w) * share + i - skew;
                int64_t run = i < share ? f(get1(w, i), v) : 0;
                for (int o = 1; o < 32; o <<= 1) {
                    const int64_t up = __shfl_up_sync(0xffffffffu, run, o);
                    if (lane >= o) run += up;
                }
                if (lane == 31) s.scan[warp] = run;
                __syncthreads();
                int64_t here = before, sum = 0;
                for (int e = 0; e < kWarps; ++e) {
                    if (e < warp) here += s.scan[e];
                    sum += s.scan[e];
                }
                const unsigned over = __ballot_sync(0xffffffffu, here + run > mark);
                if (here <= mark && over && lane == __ffs(over) - 1)
                    for (int r = 0; r < cl; ++r) st_peer32(peer_addr(&s.found, (uint32_t)r), (uint32_t)v);
                before += sum;
                if (before > mark) break;
                __syncthreads();
            }
        }
        if (cl > 1) cluster_sync();
        else __syncthreads();
        return s.found;
    };

    // ---- the row, and its largest logit -------------------------------------------
    const float tau = a.temperature ? a.temperature[t] : a.temperature_all;
    int k = a.top_k ? a.top_k[t] : a.top_k_all;
    const float top_p = a.top_p ? a.top_p[t] : a.top_p_all, min_p = a.min_p ? a.min_p[t] : a.min_p_all;
    float m = -INFINITY;
    if (P.staged) {
        for (int i = lane * kVec; i < share; i += 32 * kVec) {
            const int u = u0 + i;
            float x[kVec];
            if (u >= skew && u + kVec <= u_end) {
                const uint4 raw = __ldcs(reinterpret_cast<const uint4 *>(row + (u - skew)));
#pragma unroll
                for (int e = 0; e < kVec; ++e) x[e] = canonical(to_f<T>(reinterpret_cast<const T *>(&raw)[e]));
            } else {
#pragma unroll
                for (int e = 0; e < kVec; ++e) x[e] = read1(u + e);
            }
#pragma unroll
            for (int e = 0; e < kVec; e += 4) {
                sts128(mine + i + e, make_uint4(__float_as_uint(x[e]), __float_as_uint(x[e + 1]),
                                                __float_as_uint(x[e + 2]), __float_as_uint(x[e + 3])));
                m = fmaxf(m, fmaxf(fmaxf(x[e], x[e + 1]), fmaxf(x[e + 2], x[e + 3])));
            }
        }
        __syncwarp();
    } else {
        each([&](float l, int) { m = fmaxf(m, l); });
    }
    for (int i = tid; i < 129; i += kThreads) s.exp2[i] = kExp2[i];
    for (int i = tid; i < kBins; i += kThreads) s.hist[i] = 0;
    if (tid == 0) s.listed = 0;
    {
        // (floats in the order of whole numbers)
        auto key = [](float x) { return (int64_t)(__float_as_int(x) ^ (__float_as_int(x) < 0 ? 0x7fffffff : 0)); };
        int64_t v[1] = {key(m)};
        join(v, [](int, int64_t x, int64_t y) { return x > y ? x : y; });
        m = __int_as_float((int)v[0] ^ ((int)v[0] < 0 ? 0x7fffffff : 0));
    }
    float *const probs = a.probs ? a.probs + t * a.probs_row : nullptr;
    // f(logit, token): a probability
    auto write_probs = [&](auto f) {
        for (int i = lane; i < share; i += 32) {
            const int v = u0 + i - skew;
            if (v >= 0 && v < a.V) __stcs(probs + v, f(get1(warp, i), v));
        }
    };
    if (m == -INFINITY) {  // nothing to draw
        if (a.token && rank == 0 && tid == 0) a.token[t] = -1;
        if (probs) write_probs([](float, int) { return 0.f; });
        if (cl > 1) cluster_sync();
        return;
    }
    const int64_t part_p = (int64_t)(fminf(fmaxf(top_p, 0.f), 1.f) * 0x1p24f);
    // of a total, by a fraction of 24 bits
    auto part = [](int64_t total, int64_t f) { return (total >> 24) * f + (((total & (kUnit - 1)) * f) >> 24); };
    if (!(tau > 0.f) || k == 1 || part_p == 0) {  // the likeliest token alone
        auto top = [&](float l, int) { return (int64_t)(l == m); };
        int64_t v[1] = {0};
        each([&](float l, int) { v[0] += l == m; });
        join(v, plus);
        const int token = locate(top, 0);
        if (a.token && rank == 0 && tid == 0) a.token[t] = token;
        if (probs) write_probs([&](float, int v) { return v == token ? 1.f : 0.f; });
        if (cl > 1) cluster_sync();
        return;
    }
    Weigh weigh;
    {
        // log2(e) = 1.44269502 + 1.925963e-8, by a division and its remainder
        const float c = 1.44269502162933349609375f / tau;
        weigh.m = m;
        weigh.ch = fminf(c, 3e38f);
        weigh.cl = c <= 3e38f ? (fmaf(-c, tau, 1.44269502162933349609375f) + 1.92596299112661746887e-8f) / tau : 0.f;
        weigh.table = s.exp2;
    }
    // what the filters keep: logits above cut_l, and at cut_l tokens up to cut_v
    float cut_l = -INFINITY;
    int cut_v = INT32_MAX;
    auto kept = [&](float l, int v) { return l > cut_l || (l == cut_l && v <= cut_v); };

    // ---- bins ------------------------------------------------------------------------
    // of the first histogram by exponent, of finer ones evenly between two logits
    bool first = true;
    float hi = 0.f, lo = 0.f;
    auto bin_of = [&](float l) {  // kBins or more, or negative: in none
        if (first) {
            const float p = weigh.rough(l);
            return p > -kOctaves ? (int)(p * (-kBins / kOctaves)) : kBins;
        }
        return l > hi ? -1 : l < lo ? kBins : (int)((hi - l) / (hi - lo) * (kBins - 1));
    };
    uint32_t n4[4];  // tokens in this thread's bins
    uint32_t n_before, n_all;
    // Counts the kept tokens; the whole cluster's counts in n4, those before them in n_before.
    auto count_bins = [&]() {
        __syncthreads();
        each([&](float l, int v) {
            const int b = bin_of(l);
            if (b >= 0 && b < kBins && kept(l, v)) atomicAdd(&s.hist[b], 1u);
        });
        if (cl > 1) cluster_sync();
        else __syncthreads();
        n4[0] = n4[1] = n4[2] = n4[3] = 0;
        for (int r = 0; r < cl; ++r) {
            uint32_t x, y, z, w;
            asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(x), "=r"(y), "=r"(z), "=r"(w)
                         : "r"(peer_addr(&s.hist[4 * tid], (uint32_t)r))
                         : "memory");
            n4[0] += x, n4[1] += y, n4[2] += z, n4[3] += w;
        }
        uint32_t run = n4[0] + n4[1] + n4[2] + n4[3];
        const uint32_t own = run;
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t up = __shfl_up_sync(0xffffffffu, run, o);
            if (lane >= o) run += up;
        }
        if (lane == 31) s.scan_n[warp] = run;
        __syncthreads();
        n_before = run - own;
        n_all = 0;
        for (int e = 0; e < kWarps; ++e) {
            if (e < warp) n_before += s.scan_n[e];
            n_all += s.scan_n[e];
        }
    };
    // (after a join: every CTA has read the counts)
    auto clear_bins = [&]() {
        for (int i = tid; i < kBins; i += kThreads) s.hist[i] = 0;
    };
    // The kept tokens of bins b0 ... b1 to the first CTA's list.
    auto collect = [&](int b0, int b1) {
        if (tid == 0) s.cut_l = cut_l, s.cut_v = cut_v;
        each([&](float l, int v) {
            const int b = bin_of(l);
            if (b >= b0 && b <= b1 && kept(l, v)) {
                uint32_t at;
                asm volatile("atom.shared::cluster.add.u32 %0, [%1], 1;"
                             : "=r"(at)
                             : "r"(peer_addr(&s.listed, 0))
                             : "memory");
                if (at < kFew) {
                    st_peer(peer_addr(&s.list_l[at], 0), l);
                    st_peer32(peer_addr(&s.list_v[at], 0), (uint32_t)v);
                }
            }
        });
        if (cl > 1) cluster_sync();
        else __syncthreads();
    };
    // Ranks the list; where yes(rank, weight before, weight, last), the cut is.
    auto rank_list = [&](bool weights, auto yes) {
        if (rank == 0) {
            const int n = min((int)s.listed, kFew);
            if (weights) {
                if (tid < n) s.list_w[tid] = weigh(s.list_l[tid]);
                __syncthreads();
            }
            if (tid < n) {
                const float l = s.list_l[tid];
                const int v = s.list_v[tid];
                int place = 0;
                int64_t before = 0;
                for (int i = 0; i < n; ++i) {
                    const float x = s.list_l[i];
                    if (x > l || (x == l && s.list_v[i] < v)) {
                        ++place;
                        if (weights) before += s.list_w[i];
                    }
                }
                if (yes(place, before, weights ? s.list_w[tid] : 0, place == n - 1))
                    for (int r = 0; r < cl; ++r) {
                        st_peer(peer_addr(&s.cut_l, (uint32_t)r), l);
                        st_peer32(peer_addr(&s.cut_v, (uint32_t)r), (uint32_t)v);
                    }
            }
            __syncthreads();
            if (tid == 0) s.listed = 0;
        }
        if (cl > 1) cluster_sync();
        else __syncthreads();
        cut_l = s.cut_l;
        cut_v = s.cut_v;
    };
    // The cut at the count-th token of logit l, by index.
    auto cut_ties = [&](float l, int64_t count) {
        int64_t v[1] = {0};
        each([&](float x, int) { v[0] += x == l; });
        join(v, plus);
        cut_v = locate([&](float x, int) { return (int64_t)(x == l); }, count - 1);
        cut_l = l;
    };
    // Logits of the kept tokens in bins b0 ... b1, and the sums before them.
    struct Span {
        int64_t above, count;
        float lo, hi;
    };
    auto span = [&](int b0, int b1, bool weights) {
        int64_t v[3] = {0, 0, 0};
        float small = INFINITY, large = -INFINITY;
        each([&](float l, int i) {
            const int b = bin_of(l);
            if (b < 0 || b > b1 || !kept(l, i)) return;
            if (b >= b0) {
                ++v[1];
                small = fminf(small, l);
                large = fmaxf(large, l);
            } else if (weights) {
                v[0] += weigh(l);
            }
        });
        // both ends as one: order-preserving whole numbers, each 32 bits
        auto key = [](float x) { return (int64_t)(__float_as_int(x) ^ (__float_as_int(x) < 0 ? 0x7fffffff : 0)); };
        auto back = [](int64_t x) { return __int_as_float((int)x ^ ((int)x < 0 ? 0x7fffffff : 0)); };
        join(v, plus);
        int64_t e[2] = {key(small), key(large)};
        join(e, [](int n, int64_t x, int64_t y) { return (n == 0) == (x < y) ? x : y; });
        return Span{v[0], v[1], back(e[0]), back(e[1])};
    };

    const bool by_k = k > 0 && k < a.V, by_p = part_p < kUnit;
    int64_t total = 0;  // of the tokens that top-k keeps
    if (by_k || by_p) count_bins();
    if (by_k && n_all > (uint32_t)k) {
        // ---- the k-th token ---------------------------------------------------------
        uint32_t want = (uint32_t)k;
        uint32_t kn[4], kb = n_before;
        for (int e = 0; e < 4; ++e) kn[e] = n4[e];
        for (;;) {
            uint32_t run = kb;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (run < want && want <= run + kn[e]) {
                    s.bin0 = 4 * tid + e;
                    s.rank = want - run;
                    s.count = kn[e];
                }
                run += kn[e];
            }
            __syncthreads();
            const int b = s.bin0;
            want = s.rank;
            if (s.count <= kFew) {
                collect(b, b);
                rank_list(false, [&](int place, int64_t, int64_t, bool) { return place == (int)want - 1; });
                break;
            }
            const Span e = span(b, b, false);
            if (e.lo == e.hi) {
                cut_ties(e.lo, want);
                break;
            }
            first = false;
            hi = e.hi;
            lo = e.lo;
            clear_bins();
            count_bins();
            for (int i = 0; i < 4; ++i) kn[i] = n4[i];
            kb = n_before;
        }
    }
    if (by_p) {
        // ---- where the running weight reaches p of the total ------------------------------
        {
            int64_t v[1] = {0};
            each([&](float l, int i) {
                if (kept(l, i)) v[0] += weigh(l);
            });
            join(v, plus);
            total = v[0];
        }
        const int64_t target = part(total, part_p);
        int64_t above = 0;
        // the first histogram again, of the tokens that are left
        if (!first || cut_l > -INFINITY) {
            first = true;
            clear_bins();
            count_bins();
        }
        for (;;) {
            // bounds of the running weight behind each of this thread's bins
            float wl[4], wh[4], sl = 0.f, sh = 0.f;
            auto edge = [&](int b) {
                return first ? b * (-kOctaves / kBins) : (hi - (hi - lo) * ((float)b / (kBins - 1)) - m) * weigh.ch;
            };
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                wh[e] = sh += (float)n4[e] * exp2f(edge(4 * tid + e) + 38.f);
                wl[e] = sl += (float)n4[e] * exp2f(edge(4 * tid + e + 1) + 38.f);
            }
            const float own_l = sl, own_h = sh;
            for (int o = 1; o < 32; o <<= 1) {
                const float ul = __shfl_up_sync(0xffffffffu, sl, o), uh = __shfl_up_sync(0xffffffffu, sh, o);
                if (lane >= o) sl += ul, sh += uh;
            }
            if (lane == 31) s.scan_lo[warp] = sl, s.scan_hi[warp] = sh;
            if (tid == 0) s.bin0 = s.bin1 = kBins - 1;
            __syncthreads();
            sl -= own_l, sh -= own_h;
            for (int e = 0; e < warp; ++e) sl += s.scan_lo[e], sh += s.scan_hi[e];
            const float need = (float)(target - above);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if ((sh + wh[e]) * (1.f + kSlack) >= need) atomicMin(&s.bin0, 4 * tid + e);
                if ((sl + wl[e]) * (1.f - kSlack) >= need) atomicMin(&s.bin1, 4 * tid + e);
            }
            __syncthreads();
            int b0 = s.bin0, b1 = s.bin1;
            Span e = span(b0, b1, true);
            if (!first && e.count > kFew && e.lo < e.hi && e.lo == lo && e.hi == hi) {
                // as wide as before, so near is the cut to a bin's end: exactly, then
                const Span f = span(b0 + 1, b1, true);
                if (above + f.above >= target) {
                    b1 = b0;
                    e = span(b0, b0, true);
                } else {
                    ++b0;
                    e = f;
                }
            }
            above += e.above;
            if (e.count <= kFew) {
                collect(b0, b1);
                rank_list(true, [&](int, int64_t before, int64_t w, bool last) {
                    return above + before < target && (above + before + w >= target || last);
                });
                break;
            }
            if (e.lo == e.hi) {
                const int64_t w = weigh(e.lo), n = w > 0 ? (target - above + w - 1) / w : 1;
                cut_ties(e.lo, n < 1 ? 1 : n > e.count ? e.count : n);
                break;
            }
            first = false;
            hi = e.hi;
            lo = e.lo;
            clear_bins();
            count_bins();
        }
    }

    // ---- the token ---------------------------------------------------------------------
    const int64_t least = (int64_t)(fminf(fmaxf(min_p, 0.f), 1.f) * 0x1p38f);
    auto final_weight = [&](float l, int v) -> int64_t {
        if (!kept(l, v)) return 0;
        const int64_t w = weigh(l);
        return w >= least ? w : 0;
    };
    int64_t v[1] = {0};
    each([&](float l, int i) { v[0] += final_weight(l, i); });
    join(v, plus);
    if (a.token) {
        int64_t u = (int64_t)(a.u[t] * 0x1p24f);
        u = u < 0 ? 0 : u >= kUnit ? kUnit - 1 : u;
        const int token = locate(final_weight, part(v[0], u));
        if (rank == 0 && tid == 0) a.token[t] = token;
    }
    if (probs) {
        const float f = 1.f / (float)v[0];
        write_probs([&](float l, int i) { return (float)final_weight(l, i) * f; });
    }
    if (cl > 1) cluster_sync();  // a peer may still read this CTA's shared memory
}

template <typename T> int launch(const SampleParams &p, int cl, size_t smem, cudaStream_t stream) {
    const cudaError_t e =
        cudaFuncSetAttribute(sgmv_sample_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, 200 * 1024);
    if (e != cudaSuccess) return (int)e;
    return spec_launch(sgmv_sample_kernel<T>, dim3((unsigned)p.a.T * (unsigned)cl), kThreads, smem, cl, stream, p);
}

}  // namespace

int sample_launch(const sgmv_sample_args &a, int nsm, cudaStream_t stream) {
    // CTAs per row: as many as leave two CTAs' ranges room on an SM; more where there
    // are few rows.
    int cl = 1;
    while (cl < kMaxCluster && ((int64_t)a.V * 4 > (int64_t)cl * 100 * 1024 ||
                                ((int64_t)a.T * cl * 2 <= 2 * std::max(1, nsm) && a.V >= cl * 2 * 2048)))
        cl *= 2;
    SampleParams p;
    p.a = a;
    // (7: entries before the first token, so that vectors are aligned)
    p.share = ((a.V + 7 + cl * kWarps - 1) / (cl * kWarps) + 7) / 8 * 8;
    const size_t bytes = (size_t)p.share * kWarps * 4;
    p.staged = bytes <= 200 * 1024;
    const size_t smem = p.staged ? bytes : 0;
    switch (a.dtype) {
        case SGMV_F16: return launch<__half>(p, cl, smem, stream);
        case SGMV_BF16: return launch<__nv_bfloat16>(p, cl, smem, stream);
        default: return launch<float>(p, cl, smem, stream);
    }
}

}  // namespace sgmv
