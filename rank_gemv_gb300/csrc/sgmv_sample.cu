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
// sort.  A histogram over the logits counts the tokens; top-k bounds the bins that can
// matter, or top-p does (the weights at a bin's edges bound the running weight from both
// sides).  If they hold few tokens, as they mostly do, one CTA collects them, ranks them
// one against all and draws.  If not, each thread notes which of its tokens they are,
// and only those are looked at again: the bins around the cut are divided finer, until
// few tokens are left, or one value, whose tokens are counted off by index; the sums
// above the cut are exact at every step.
//
// 128 rows of 100277 fp32 logits, all filters, no two rows alike: 63 to 82 us for eight sets of
// rows and settings (51 MB at 0.6 to 0.8 TB/s; a plain copy of them takes 16; without filters
// 62).  Bounded by the rows that have many candidates: one row takes 10 us greedy, 12 to 25
// with a top-k of up to 256, 30 to 40 of 1000, and 35 to 60 with top-p alone, most of that
// weighing, some 40 instructions for a weight that is not deep.  Each token is weighed once
// for the total and once above the cut, at most: what a thread has weighed above is its part
// of the kept weights too, where min-p drops nothing (a third time: 64 to 94 us, top-p alone
// 133 against 107).  One row of 32000, top-p: 12 to 30 us by the number of candidates, a
// chain of passes with a cluster barrier after each; the host needs 9.
//
// Slower: a cut among weights of a few units, where the bounds are wide and each pass narrows
// less (one large logit over 128255 others 24 nats below, top_p 1 - 2^-20: 128 rows 583 us, 75
// with 0.9999); and vocabularies from 262138 tokens on, whose ranges are too long for a bit per
// entry of a thread (128 rows, top-p alone: of 250000 tokens 404 us, of 262144 963).
#include <algorithm>

#include "sgmv_device.cuh"
#include "sgmv_spec.h"

namespace sgmv {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kBins = 2 * kThreads;
constexpr int kFew = 256;               // tokens that are ranked one against all
constexpr int kLong = 512;              // entries of a warp's range from which on its threads' largest are counted
constexpr float kDeep = 18.f;            // octaves below the largest weight from which on fp32 is exact enough
constexpr float kOctaves = 39.f;        // weights below 2^-39 of the largest are zero
constexpr float kSlack = 3e-5f;         // rounding of the weights at bins' edges and of their sums
constexpr int64_t kUnit = 1ll << 24;

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
    __align__(16) uint32_t hist[kBins];
    __align__(16) uint4 list[kFew];         // logit, token, weight
    int64_t exp2[129];
    int64_t part[2][4][kWarps];         // a sum of every warp,
    int64_t every[2][4][kMaxCluster];   // and of every CTA
    int64_t scan[kWarps];
    float scan_lo[kWarps], scan_hi[kWarps];
    uint32_t scan_n[kWarps];
    uint32_t listed;
    int bin0, bin1;
    uint32_t rank, count;
    float cut_l;
    int32_t cut_v, found;
};
static_assert(kFew * 16 >= kWarps * 64 * 4, "the warps' queues in the list");
static_assert(2 * (sizeof(SampleShared) + 1024 + 100 * 1024) <= 228 * 1024, "two CTAs per SM");

struct SampleParams {
    sgmv_sample_args a;
    int32_t share;   // entries of a warp's range
    int32_t staged;  // the ranges are in shared memory
    int32_t noted;   // a thread's entries of a range have a bit each
    int32_t sorted;  // slow rows first
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
    // 38 above the exponent; of one below -kDeep the weight, which is less than 2^20,
    // so that its rounding is a unit or so
    __device__ __forceinline__ float raised(float l) const { return fmaf(l - m, ch, 38.f); }
    static __device__ __forceinline__ uint32_t deep(float raised) {
        float w;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(w) : "f"(raised));
        return __float2uint_rz(w);
    }
    __device__ __forceinline__ int64_t operator()(float l) const {
        // l - m = d + e exactly; times log2(e) / temperature: p + q
        const float d = l - m;
        const float up = fmaf(d, ch, 38.f);
        if (!(up >= 38.f - kDeep)) return deep(up);
        const float b = d - l, e = (l - (d - b)) + (-m - b);
        const float p = d * ch;
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
    int64_t t = (int64_t)(blockIdx.x / (unsigned)cl);
    if (cl > 1) cluster_arrive_relaxed();  // waited on just before the first peer access
    pdl_wait();
    pdl_trigger();
    if (P.sorted) {
        // More rows than run at once: those whose filters may have to look at many tokens, which
        // take several times as long, come first (128 rows of 100277, one of the sets of mixed
        // settings: 63 us, 77 as they come; 512 rows of 32000 with probabilities, when they were
        // weighed three times: 113, 144).  A thread looks at each row: up to 512 of them.
        bool slow = false;
        if (tid < a.T) {
            const int k = a.top_k ? a.top_k[tid] : a.top_k_all;
            const float p = a.top_p ? a.top_p[tid] : a.top_p_all, tau = a.temperature ? a.temperature[tid] : a.temperature_all;
            slow = tau > 0.f && (k <= 0 || k > kFew) && (p < 1.f || k > kFew) && p > 0.f;
        }
        const unsigned who = __ballot_sync(0xffffffffu, slow);
        if (lane == 0) s.scan_n[warp] = (uint32_t)__popc(who);
        __syncthreads();
        int before = __popc(who & ((1u << lane) - 1)), all = 0;  // slow rows
        for (int e = 0; e < kWarps; ++e) {
            if (e < warp) before += (int)s.scan_n[e];
            all += (int)s.scan_n[e];
        }
        if (tid < a.T && (slow ? before : all + tid - before) == (int)t) s.found = tid;
        __syncthreads();
        t = s.found;
    }
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
    // the entries of this thread that a pass looks at: all of them, or those noted (bit 4 j + e:
    // entry 128 j + 4 lane + e of the warp's range); inside: those that the last span() counted
    uint64_t noted = 0, inside = 0;
    bool by_note = false;
    uint64_t at_bit = 0;  // of the entry that f is given
    // f(logit, token) of them
    auto each = [&](auto f) {
        if (by_note) {
            // (the warp's lanes together: left to themselves they drift apart at f's
            // branches and run one by one, which took four times as long)
            for (uint64_t left = noted; __any_sync(0xffffffffu, left != 0); left &= left - 1) {
                if (left) {
                    const int k = __ffsll((long long)left) - 1, i = (k >> 2) * 128 + lane * 4 + (k & 3);
                    at_bit = left & -left;
                    f(ldsf(mine + i), u0 + i - skew);
                }
                __syncwarp();
            }
            return;
        }
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
    // values stay in part[], the CTAs' in every[], of the turn before.
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
        if (warp < N) {  // warp n joins value n and hands it to every CTA
            int64_t x = s.part[at][warp][lane % kWarps];
            for (int o = kWarps / 2; o > 0; o >>= 1) x = op(warp, x, (int64_t)__shfl_xor_sync(0xffffffffu, x, o));
            if (lane < cl)
                asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(
                                 peer_addr(&s.every[at][warp][rank], (uint32_t)lane)),
                             "l"(x)
                             : "memory");
        }
        if (cl > 1) cluster_sync();
        else __syncthreads();
#pragma unroll
        for (int n = 0; n < N; ++n) {
            v[n] = s.every[at][n][0];
            for (int r = 1; r < cl; ++r) v[n] = op(n, v[n], s.every[at][n][r]);
        }
    };
    auto plus = [](int, int64_t x, int64_t y) { return x + y; };
    // The token where the running sum of f in index order passes `mark`, after a join of
    // f's sums alone (found: it, in every CTA).
    auto locate = [&](auto f, int64_t mark) {
        const int at = turn ^ 1;
        int64_t before = 0;
        const int64_t all = s.every[at][0][rank];
        for (int r = 0; r < rank; ++r) before += s.every[at][0][r];
        if (before <= mark && mark < before + all) {  // it is this CTA's
            int w = 0;
            while (w < kWarps - 1 && mark >= before + s.part[at][0][w]) before += s.part[at][0][w++];
            // each thread's part of the warp's range, then the thread's entries one by one
            const int each_has = (share + kThreads - 1) / kThreads, i0 = min(share, tid * each_has);
            const int i1 = min(share, i0 + each_has), v0 = (rank * kWarps + w) * share - skew;
            int64_t own = 0;
            for (int i = i0; i < i1; ++i) own += f(get1(w, i), v0 + i);
            int64_t run = own;
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t up = __shfl_up_sync(0xffffffffu, run, o);
                if (lane >= o) run += up;
            }
            if (lane == 31) s.scan[warp] = run;
            __syncthreads();
            run += before - own;
            for (int e = 0; e < warp; ++e) run += s.scan[e];
            if (run <= mark && mark < run + own)
                for (int i = i0; i < i1; ++i) {
                    run += f(get1(w, i), v0 + i);
                    if (mark < run) {
                        for (int r = 0; r < cl; ++r) st_peer32(peer_addr(&s.found, (uint32_t)r), (uint32_t)(v0 + i));
                        break;
                    }
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
        // Four vectors under way at a time, none of them under a condition (their answers would be
        // waited for one by one): a vector that is not whole within the row reads another, and
        // its entries singly.
        const int whole0 = (skew + kVec - 1) / kVec * kVec, whole1 = u_end / kVec * kVec - kVec;
        for (int i0 = lane * kVec; i0 < share; i0 += 4 * 32 * kVec) {
            uint4 raw[4];
            if (whole0 <= whole1) {
#pragma unroll
                for (int b = 0; b < 4; ++b)
                    raw[b] = __ldcs(reinterpret_cast<const uint4 *>(
                        row + (max(whole0, min(whole1, u0 + i0 + b * 32 * kVec)) - skew)));
            }
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const int i = i0 + b * 32 * kVec, u = u0 + i;
                if (i >= share) break;
                float x[kVec];
#pragma unroll
                for (int e = 0; e < kVec; ++e) x[e] = canonical(to_f<T>(reinterpret_cast<const T *>(&raw[b])[e]));
                if (u < whole0 || u > whole1) {
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
        }
        __syncwarp();
    } else {
        each([&](float l, int) { m = fmaxf(m, l); });
    }
    for (int i = tid; i < 129; i += kThreads) s.exp2[i] = kExp2[i];
    for (int i = tid; i < kBins; i += kThreads) s.hist[i] = 0;
    if (tid == 0) s.listed = 0;
    const float largest = m;  // this thread's
    {
        // (floats in the order of whole numbers)
        auto key = [](float x) { return (int64_t)(__float_as_int(x) ^ (__float_as_int(x) < 0 ? 0x7fffffff : 0)); };
        int64_t v[1] = {key(m)};
        if (cl > 1) cluster_wait();  // every CTA of the cluster has started
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
    uint32_t n2[2];  // tokens in this thread's bins
    uint32_t n_before, n_all;
    auto count = [&](float l) {
        const int b = bin_of(l);
        if (b >= 0 && b < kBins) atomicAdd(&s.hist[b], 1u);
    };
    // The sum of the weights of entries with on(logit, token, bit), with take(logit) for those
    // that are not deep.
    // Deep ones, mostly the most, are done at once; the others, whose weights take ten times the
    // instructions, wait in a queue of the warp's until all of its lanes have one.
    auto sum_weights = [&](auto on, auto take, int64_t &deep_sum) {
        float *const queue = reinterpret_cast<float *>(s.list) + warp * 64;
        int64_t sum = 0;
        int waiting = 0;
        auto weigh_one = [&](float l) {
            sum += weigh(l);
            take(l);
        };
        for (int j = 0; 128 * j < share; ++j) {
            const int i = 128 * j + lane * 4;
            const float4 x4 = i < share ? get4(i) : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
            const float x[4] = {x4.x, x4.y, x4.z, x4.w};
            uint32_t w = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float up = weigh.raised(x[e]);
                const bool yes = on(x[e], u0 + i + e - skew, 4 * j + e), full = yes && up >= 38.f - kDeep;
                if (yes && !full) w += Weigh::deep(up);
                const unsigned who = __ballot_sync(0xffffffffu, full);
                if (full) queue[waiting + __popc(who & ((1u << lane) - 1))] = x[e];
                waiting += __popc(who);
                if (waiting >= 32) {
                    __syncwarp();
                    weigh_one(queue[lane]);
                    waiting -= 32;
                    const float rest = queue[32 + lane];
                    __syncwarp();
                    queue[lane] = rest;
                    __syncwarp();
                }
            }
            deep_sum += w;
        }
        __syncwarp();
        if (lane < waiting) weigh_one(queue[lane]);
        __syncwarp();
        return sum + deep_sum;
    };
    // Counts what the pass counts; the whole cluster's counts in n2, those before them in n_before.
    auto count_bins = [&](auto pass) {
        __syncthreads();
        pass();
        if (cl > 1) cluster_sync();
        else __syncthreads();
        uint32_t x[kMaxCluster], y[kMaxCluster];
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r)  // all under way at once
            asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];"
                         : "=r"(x[r]), "=r"(y[r])
                         : "r"(peer_addr(&s.hist[2 * tid], (uint32_t)min(r, cl - 1)))
                         : "memory");
        n2[0] = n2[1] = 0;
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r)
            if (r < cl) n2[0] += x[r], n2[1] += y[r];
        uint32_t run = n2[0] + n2[1];
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
    auto count_kept = [&]() {
        each([&](float l, int v) {
            if (kept(l, v)) count(l);
        });
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
                    st_peer(peer_addr(&s.list[at].x, 0), l);
                    st_peer32(peer_addr(&s.list[at].y, 0), (uint32_t)v);
                }
            }
        });
        if (cl > 1) cluster_sync();
        else __syncthreads();
    };
    // In the first CTA: entry tid (of n) of the list, the number of entries ranked before it
    // and their weight.  Two threads per entry go through half the list each.
    struct Entry {
        float l;
        int v, place;
        int64_t w, before;
    };
    auto entry = [&](int n) {
        Entry x = {};
        const int at = tid % kFew;
        if (at < n) {
            x.l = __uint_as_float(s.list[at].x);
            x.v = (int)s.list[at].y;
            x.w = weigh(x.l);
            if (tid < n) *reinterpret_cast<int64_t *>(&s.list[at].z) = x.w;
        }
        __syncthreads();
        const int e0 = tid < kFew ? 0 : n / 2, e1 = tid < kFew ? n / 2 : n;
#pragma unroll 4
        for (int e = e0; e < e1; ++e) {
            const uint4 y = lds128(&s.list[e]);
            const float l = __uint_as_float(y.x);
            const bool ahead = l > x.l || (l == x.l && (int)y.y < x.v);
            x.place += ahead;
            x.before += ahead ? (int64_t)((uint64_t)y.w << 32 | y.z) : 0;
        }
        static_assert(kThreads == 2 * kFew && sizeof(s.hist) >= kFew * 16, "two halves of the list");
        uint4 *const half = reinterpret_cast<uint4 *>(s.hist);  // (the bins are done with, or cleared before the next use)
        if (tid >= kFew) half[at] = make_uint4((uint32_t)x.place, 0, (uint32_t)x.before, (uint32_t)(x.before >> 32));
        __syncthreads();
        if (tid < kFew) {
            const uint4 y = half[at];
            x.place += (int)y.x;
            x.before += (int64_t)((uint64_t)y.w << 32 | y.z);
        }
        return x;
    };
    // Ranks the list; where yes(entry), the cut is.
    auto rank_list = [&](auto yes) {
        if (rank == 0) {
            const int n = min((int)s.listed, kFew);
            const Entry x = entry(n);
            if (tid < n && yes(x))
                for (int r = 0; r < cl; ++r) {
                    st_peer(peer_addr(&s.cut_l, (uint32_t)r), x.l);
                    st_peer32(peer_addr(&s.cut_v, (uint32_t)r), (uint32_t)x.v);
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
    int64_t own_above = 0;  // this thread's part of the last span's weights
    auto span = [&](int b0, int b1, bool weights) {
        int64_t v[4] = {0, 0, 0, 0};
        float small = INFINITY, large = -INFINITY;
        inside = 0;
        // whether a token is in a bin before b0; those in the bins are counted
        auto before = [&](float l, int i, uint64_t bit) {
            const int b = bin_of(l);
            if (b < 0 || b > b1 || !kept(l, i)) return false;
            if (b < b0) return true;
            ++v[1];
            inside |= bit;
            small = fminf(small, l);
            large = fmaxf(large, l);
            return false;
        };
        if (P.noted && !by_note) {
            int64_t deep = 0;
            v[0] = sum_weights([&](float l, int i, int bit) { return before(l, i, 1ull << bit) && weights; }, [](float) {}, deep);
        } else {
            each([&](float l, int i) {
                if (before(l, i, at_bit) && weights) v[0] += weigh(l);
            });
        }
        own_above = v[0];
        // (floats in the order of whole numbers)
        auto key = [](float x) { return (int64_t)(__float_as_int(x) ^ (__float_as_int(x) < 0 ? 0x7fffffff : 0)); };
        auto back = [](int64_t x) { return __int_as_float((int)x ^ ((int)x < 0 ? 0x7fffffff : 0)); };
        v[2] = -key(small);
        v[3] = key(large);
        join(v, [](int n, int64_t x, int64_t y) { return n < 2 ? x + y : x > y ? x : y; });
        return Span{v[0], v[1], back(-v[2]), back(v[3])};
    };

    const bool by_k = k > 0 && k < a.V, by_p = part_p < kUnit;
    const int64_t least = (int64_t)(fminf(fmaxf(min_p, 0.f), 1.f) * 0x1p38f);
    int64_t target = 0;  // top-p's part of the weights
    // Bounds of the running weight at the ends of this thread's bins, over `above`; then the
    // first bin that can reach the target, and the first that must, to bin0 and bin1.
    // mass: what the counted tokens weigh in all, if known (else 0): then what lies behind a bin
    // bounds it too, which is what finds a cut near the end.  A weight is rounded down to a whole
    // number: at the lower edge it is above 2^x - 2, not 2^x, which counts where the cut is among
    // weights of some thousand units or less.  (What fp32 makes of an edge, x and the weights
    // themselves is 1.5e-5 of a weight at most: kSlack.)
    auto bound_bins = [&](int64_t above, int64_t mass) {
        float wl[2], wh[2], sl = 0.f, sh = 0.f;
        auto edge = [&](int b) {
            return first ? b * (-kOctaves / kBins) : (hi - (hi - lo) * ((float)b / (kBins - 1)) - m) * weigh.ch;
        };
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            wh[e] = sh += (float)n2[e] * exp2f(edge(2 * tid + e) + 38.f);
            wl[e] = sl += (float)n2[e] * fmaxf(exp2f(edge(2 * tid + e + 1) + 38.f) - 2.f, 0.f);
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
        float all_l = 0.f, all_h = 0.f;
        for (int e = 0; e < kWarps; ++e) {
            if (e < warp) sl += s.scan_lo[e], sh += s.scan_hi[e];
            all_l += s.scan_lo[e], all_h += s.scan_hi[e];
        }
        const float need = (float)(target - above), m0 = (float)mass, slack = all_h * kSlack;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float most = (sh + wh[e]) * (1.f + kSlack), least = (sl + wl[e]) * (1.f - kSlack);
            if (mass > 0) {
                most = fminf(most, m0 - (all_l - (sl + wl[e])) + slack);
                least = fmaxf(least, m0 - (all_h - (sh + wh[e])) - slack);
            }
            if (most >= need) atomicMin(&s.bin0, 2 * tid + e);
            if (least >= need) atomicMin(&s.bin1, 2 * tid + e);
        }
        __syncthreads();
    };
    // The bin where the want-th token falls: bin0, with its rank there and the bin's count.
    auto find_bin = [&](uint32_t want) {
        uint32_t run = n_before;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            if (run < want && want <= run + n2[e]) {
                s.bin0 = 2 * tid + e;
                s.rank = want - run;
                s.count = n2[e];
            }
            run += n2[e];
        }
        __syncthreads();
    };
    int64_t total = 0;    // of the tokens that top-k keeps
    int64_t counted = 0;  // and of those in the first bins
    bool cut_k = false, bounds = false;  // bounds: bin0 and bin1 are those of the first bins
    // Notes this thread's tokens in bins up to `last`.
    auto note = [&](int last) {
        noted = 0;
        for (int j = 0; 128 * j + lane * 4 < share; ++j) {
            const float4 x = get4(128 * j + lane * 4);
            const uint32_t bits = (bin_of(x.x) <= last) | (bin_of(x.y) <= last) << 1 | (bin_of(x.z) <= last) << 2 |
                                  (bin_of(x.w) <= last) << 3;
            noted |= (uint64_t)bits << (4 * j);
        }
        by_note = true;
    };
    if (by_k || by_p) {
        // the last bin that matters, and the tokens up to it
        int last = kBins - 1;
        uint32_t few = 0;
        bool bounded = false;
        if (by_k && P.noted && share >= kLong) {
            // In long ranges the threads' largest logits are counted first, which are few:
            // the k-th of them is no larger than the k-th of all.
            count_bins([&]() { count(largest); });
            if (n_all >= (uint32_t)k) {
                find_bin((uint32_t)k);
                last = s.bin0;
                bounded = true;
            }
            note(last);
            int64_t v[1] = {__popcll(noted)};
            join(v, plus);
            few = (uint32_t)v[0];
            cut_k = bounded || few > (uint32_t)k;
            clear_bins();
        }
        if (!by_note || few > kFew) {
            int64_t v[2] = {0, 0};  // the weights, and those of deep ones that are not counted
            const bool sums = by_p && !by_k;
            count_bins([&]() {
                if (sums && P.noted) v[0] = sum_weights([](float, int, int) { return true; }, count, v[1]);
                else each([&](float l, int) {
                    count(l);
                    if (sums) v[0] += weigh(l);
                });
            });
            cut_k = by_k && (bounded || n_all > (uint32_t)k);
            if (cut_k) {
                find_bin((uint32_t)k);
                last = s.bin0;
                few = (uint32_t)k - s.rank + s.count;
            } else {
                few = n_all;
                if (by_p) {
                    if (by_k) each([&](float l, int) { v[0] += weigh(l); });
                    join(v, plus);
                    total = v[0];
                    target = part(total, part_p);
                    counted = total - v[1];
                    bound_bins(0, counted);
                    last = s.bin1;
                    if (sums && P.noted && last >= (int)(kDeep * (kBins / kOctaves)) - 1) {
                        // the cut may be among the deep ones: with them
                        clear_bins();
                        count_bins(count_kept);
                        counted = total;
                        bound_bins(0, counted);
                        last = s.bin1;
                        few = n_all;
                    }
                    bounds = true;
                    if (tid == last / 2) s.count = n_before + n2[0] + (last & 1 ? n2[1] : 0);
                    __syncthreads();
                    few = s.count;
                }
            }
        }
        if (few <= kFew) {
            // ---- one CTA has them all -------------------------------------------------
            collect(0, last);
            if (rank != 0) {
                if (probs) write_probs([](float, int) { return 0.f; });
                if (probs && cl > 1) cluster_sync();
                return;
            }
            const int n = (int)few;
            const Entry x = entry(n);
            int64_t w = tid < n ? x.w : 0;
            // sum over the list, for all
            auto sum = [&](int64_t x) {
                for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
                __syncthreads();
                if (lane == 0) s.scan[warp] = x;
                __syncthreads();
                x = 0;
                for (int e = 0; e < kFew / 32; ++e) x += s.scan[e];
                return x;
            };
            bool on = tid < n && (!cut_k || x.place < k);
            if (by_p) {
                if (target == 0) target = part(sum(on ? w : 0), part_p);  // the list has all that top-k keeps
                on = on && (x.place == 0 || x.before < target);
            }
            if (!on || w < least) w = 0;
            total = sum(w);
            if (tid < n) *reinterpret_cast<int64_t *>(&s.list[tid].z) = w;
            __syncthreads();
            if (a.token) {
                int64_t u = (int64_t)(a.u[t] * 0x1p24f);
                u = u < 0 ? 0 : u >= kUnit ? kUnit - 1 : u;
                const int64_t mark = part(total, u);
                // the weight of kept tokens before this one by index
                int64_t run = 0;
                if (tid < kFew)
#pragma unroll 4
                    for (int e = 0; e < n; ++e) {
                        const uint4 y = lds128(&s.list[e]);
                        run += (int)y.y < x.v ? (int64_t)((uint64_t)y.w << 32 | y.z) : 0;
                    }
                if (w > 0 && run <= mark && mark < run + w) a.token[t] = x.v;
            }
            if (probs) {
                write_probs([](float, int) { return 0.f; });
                if (cl > 1) cluster_sync();
                else __syncthreads();
                if (w > 0) probs[x.v] = (float)w * (1.f / (float)total);
            }
            return;
        }
        // (half of the row: 128 rows with top-k and top-p took 76 us with a sixteenth, 65 so;
        // without, the first span looks at every token, in vectors)
        if (P.noted && few <= (uint32_t)a.V / 2) note(last);
    }
    const uint64_t candidates = noted;
    const bool some = by_note;
    if (cut_k) {
        // ---- the k-th token ---------------------------------------------------------
        const uint32_t n2_0 = n2[0], n2_1 = n2[1], n_before_0 = n_before;
        for (uint32_t want = (uint32_t)k;;) {
            if (!first) find_bin(want);
            const int b = s.bin0;
            want = s.rank;
            if (s.count <= kFew) {
                collect(b, b);
                rank_list([&](const Entry &x) { return x.place == (int)want - 1; });
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
            noted = inside;  // only these are looked at from here on
            by_note = P.noted;
            clear_bins();
            count_bins(count_kept);
        }
        // the first bins' counts of what is left
        first = true;
        noted = candidates;
        by_note = some;
        const uint32_t room = (uint32_t)k > n_before_0 ? (uint32_t)k - n_before_0 : 0;
        n2[0] = min(n2_0, room);
        n2[1] = min(n2_1, room - n2[0]);
        if (by_p) {
            int64_t v[1] = {0};
            each([&](float l, int i) {
                if (kept(l, i)) v[0] += weigh(l);
            });
            join(v, plus);
            counted = total = v[0];
            target = part(total, part_p);
        }
    }
    int64_t own_kept = 0;  // what this thread has weighed above the cut
    if (by_p) {
        // ---- where the running weight reaches p of the total ------------------------------
        int64_t above = 0;
        for (;;) {
            if (!bounds) bound_bins(above, first ? counted : 0);
            bounds = false;
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
            own_kept += own_above;
            noted = inside;  // only these are looked at from here on
            by_note = P.noted;
            if (e.count <= kFew) {
                collect(b0, b1);
                rank_list([&](const Entry &x) {
                    return above + x.before < target && above + x.before + x.w >= target;
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
            count_bins(count_kept);
        }
    }

    // ---- the token ---------------------------------------------------------------------
    // (a logit whose weight cannot reach min_p's needs no weight)
    const float floor_l = least > 0 ? log2f((float)least) - 38.01f : -INFINITY;
    auto final_weight = [&](float l, int v) -> int64_t {
        if (!kept(l, v) || weigh.rough(l) < floor_l) return 0;
        const int64_t w = weigh(l);
        return w >= least ? w : 0;
    };
    int64_t v[1] = {0}, deep = 0;
    if (by_p && P.noted && weigh(cut_l) >= least) {
        // min-p drops nothing that is left: the tokens above have been weighed, those around the
        // cut are noted
        v[0] = own_kept;
        each([&](float l, int i) {
            if (kept(l, i)) v[0] += weigh(l);
        });
    } else {
        noted = candidates;
        by_note = some;
        if (by_note || !P.noted || least > 0) each([&](float l, int i) { v[0] += final_weight(l, i); });
        else v[0] = sum_weights([&](float l, int i, int) { return kept(l, i); }, [](float) {}, deep);
    }
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
    p.noted = p.staged && p.share <= 64 / 4 * 128;
    p.sorted = (a.top_k || a.top_p) && a.T <= kThreads && (int64_t)a.T * cl > 2 * std::max(1, nsm);
    const size_t smem = p.staged ? bytes : 0;
    switch (a.dtype) {
        case SGMV_F16: return launch<__half>(p, cl, smem, stream);
        case SGMV_BF16: return launch<__nv_bfloat16>(p, cl, smem, stream);
        default: return launch<float>(p, cl, smem, stream);
    }
}

}  // namespace sgmv
