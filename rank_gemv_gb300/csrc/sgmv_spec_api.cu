// sgmv_spec_api.cu -- the C ABI of the decoding operators: argument checks and
// launches.
#include <math.h>

#include <climits>

#include "sgmv.h"
#include "sgmv_internal.h"
#include "sgmv_spec.h"

namespace {

using namespace sgmv;

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
// of every array of 32-bit words (those that are not given pass)
template <typename... P> bool aligned4(const P *...p) { return ((reinterpret_cast<uintptr_t>(p) | ... | 0) & 3u) == 0; }
bool half_type(int dt) { return dt == SGMV_F16 || dt == SGMV_BF16; }

// 16-bit data read and written in 16-byte pieces
bool vectors(const void *p, int64_t s0, int64_t s1, int width = 8) {
    return aligned16(p) && s0 % width == 0 && s1 % width == 0;
}

// The stride of a dimension of one entry is never used and may be anything: it
// becomes one that passes the checks here and fits a tensor map.
void settle(int64_t &stride, int32_t entries, int32_t D) {
    if (entries == 1) stride = D;
}

constexpr int32_t kMaxVocabulary = 1 << 24;
constexpr double kMaxRows = 1 << 30;  // heads of all tokens, which the norm kernels count in 32 bits

int check_head(int32_t D) {
    if (D < 1) return SGMV_ERR_INVALID_ARG;
    if (D % 8 != 0) return SGMV_ERR_ALIGNMENT;
    return D > kSpecMaxD ? SGMV_ERR_UNSUPPORTED : SGMV_OK;
}

// Arguments of the rotary calls, a's unused strides settled; width: elements of the
// cache in 16 bytes.  `none`: there is nothing to do.
int check_rope(sgmv_rope_args &a, int width, bool *none) {
    *none = false;
    if (a.T < 0 || a.Hq < 0 || a.Hk < 0 || !half_type(a.dtype)) return SGMV_ERR_INVALID_ARG;
    const int st = check_head(a.D);
    if (st != SGMV_OK) return st;
    if (a.pairs < 0 || 2 * (int64_t)a.pairs > a.D || (a.pairs > 0 && !a.inv_freq))
        return SGMV_ERR_INVALID_ARG;
    const bool append = a.k_cache || a.v_cache || a.slots;
    if (append && (!a.k_cache || !a.v_cache || !a.slots || a.num_blocks < 1 || a.block_size < 1))
        return SGMV_ERR_INVALID_ARG;
    if (a.T == 0 || (a.Hq == 0 && a.Hk == 0)) {
        *none = true;
        return SGMV_OK;
    }
    if (!a.positions || (a.Hq > 0 && (!a.q || !a.q_out))) return SGMV_ERR_INVALID_ARG;
    if (a.Hk > 0 && (!a.k || (!a.k_out && !append) || (append && !a.v))) return SGMV_ERR_INVALID_ARG;
    if (a.Hk == 0 && append) return SGMV_ERR_INVALID_ARG;
    for (int64_t *s : {&a.q_token, &a.q_out_token, &a.k_token, &a.k_out_token, &a.v_token}) settle(*s, a.T, a.D);
    for (int64_t *s : {&a.q_head, &a.q_out_head}) settle(*s, a.Hq, a.D);
    for (int64_t *s : {&a.k_head, &a.k_out_head, &a.v_head, &a.cache_head}) settle(*s, a.Hk, a.D);
    settle(a.cache_block, a.num_blocks, a.D);
    settle(a.cache_token, a.block_size, a.D);
    if (a.Hq > 0 && (!vectors(a.q, a.q_token, a.q_head) || !vectors(a.q_out, a.q_out_token, a.q_out_head)))
        return SGMV_ERR_ALIGNMENT;
    if (a.Hk > 0 && (!vectors(a.k, a.k_token, a.k_head) ||
                     (a.k_out && !vectors(a.k_out, a.k_out_token, a.k_out_head))))
        return SGMV_ERR_ALIGNMENT;
    if (append && (!vectors(a.v, a.v_token, a.v_head) || !vectors(a.k_cache, a.cache_block, a.cache_token, width) ||
                   !vectors(a.v_cache, a.cache_head, 0, width) || a.D % width != 0))
        return SGMV_ERR_ALIGNMENT;
    return aligned4(a.positions, a.slots) ? SGMV_OK : SGMV_ERR_ALIGNMENT;
}

// Turns per position, modulo one turn, as a fraction of 2^64.
int turns_of(const double *inv_freq, int32_t pairs, uint64_t *turns) {
    for (int i = 0; i < pairs; ++i) {
        const double f = inv_freq[i] * 0.15915494309189533577;  // 1 / (2 pi)
        if (!(fabs(f) < 1e15)) return SGMV_ERR_INVALID_ARG;
        const double part = f - floor(f);  // [0, 1]
        turns[i] = part < 1.0 ? (uint64_t)(part * 0x1p64) : 0;
    }
    return SGMV_OK;
}

// Arguments of the attention calls but the workspace's size, as above.
int check_attention(sgmv_tree_attention_args &a, int width, bool *none) {
    *none = false;
    if (a.T < 0 || a.B < 0 || a.Hq < 1 || a.Hkv < 1 || a.Hq % a.Hkv != 0 || !half_type(a.dtype) ||
        !(a.scale == a.scale))
        return SGMV_ERR_INVALID_ARG;
    const int st = check_head(a.D);
    if (st != SGMV_OK) return st;
    if (a.T == 0 || a.B == 0) {
        *none = true;
        return SGMV_OK;
    }
    // a sequence's row tiles (of 8 rows at least) of all heads times its token tiles (and
    // two more, and a part of one) are counted in 32 bits
    if (a.Hq > 65535 || (double)a.Hq * SGMV_TREE_MAX_NODES / 8 *
                                ((double)a.max_blocks * a.block_size / tree_tile(a.block_size) + 3) > 4294967295.0)
        return SGMV_ERR_UNSUPPORTED;
    if (!a.out || !a.q || !a.k_cache || !a.v_cache || !a.block_table || !a.prefix_lens || !a.tree_ptr)
        return SGMV_ERR_INVALID_ARG;
    if (a.num_blocks < 1 || a.block_size < 1 || a.max_blocks < 1 || a.table_row < 0)
        return SGMV_ERR_INVALID_ARG;
    for (int64_t *s : {&a.q_token, &a.out_token}) settle(*s, a.T, a.D);
    for (int64_t *s : {&a.q_head, &a.out_head}) settle(*s, a.Hq, a.D);
    settle(a.cache_block, a.num_blocks, a.D);
    settle(a.cache_token, a.block_size, a.D);
    settle(a.cache_head, a.Hkv, a.D);
    if (!vectors(a.q, a.q_token, a.q_head) || !vectors(a.out, a.out_token, a.out_head) ||
        !vectors(a.k_cache, a.cache_block, a.cache_token, width) || !vectors(a.v_cache, a.cache_head, 0, width) ||
        a.D % width != 0)
        return SGMV_ERR_ALIGNMENT;
    return aligned4(a.lse, a.block_table, a.prefix_lens, a.tree_ptr, a.parents) ? SGMV_OK : SGMV_ERR_ALIGNMENT;
}
int check_workspace(const void *workspace, uint64_t bytes, size_t need, size_t align) {
    if (bytes < need || !workspace) return SGMV_ERR_WORKSPACE;
    return reinterpret_cast<uintptr_t>(workspace) % align != 0 ? SGMV_ERR_ALIGNMENT : SGMV_OK;
}

int finish(const char *what, int e, int launches) {
    if (e == (int)cudaSuccess) {
        set_launch_count(launches);
        return SGMV_OK;
    }
    note_cuda_error(what, (cudaError_t)e);
    return SGMV_ERR_CUDA;
}

}  // namespace

extern "C" {

int sgmv_rope(const sgmv_rope_args *args, void *stream) {
    set_launch_count(0);
    if (!args) return SGMV_ERR_INVALID_ARG;
    sgmv_rope_args a = *args;
    bool none;
    int st = check_rope(a, 8, &none);
    if (st != SGMV_OK || none) return st;
    uint64_t turns[kRopeMaxPairs];
    if ((st = turns_of(a.inv_freq, a.pairs, turns)) != SGMV_OK) return st;
    int *err = device_error_word();
    if (!err) return SGMV_ERR_CUDA;
    return finish("rotary kernel", rope_launch(a, turns, device_sms(), err, static_cast<cudaStream_t>(stream)), 1);
}

int sgmv_rope_frequencies(double *inv_freq, int32_t pairs, double base, double factor,
                          double trained, double slow, double fast) {
    if (!inv_freq || pairs < 1 || !(base > 0) || !(factor > 0)) return SGMV_ERR_INVALID_ARG;
    const bool ramp = factor != 1.0 && isfinite(fast);
    if (ramp && (!(trained > 0) || !(slow < fast))) return SGMV_ERR_INVALID_ARG;
    for (int32_t i = 0; i < pairs; ++i) {
        const double f = pow(base, -(double)i / pairs);
        double keep = factor == 1.0 ? 1.0 : 0.0;
        if (ramp) {
            const double turns = trained * f / 6.283185307179586476925;
            keep = fmin(1.0, fmax(0.0, (turns - slow) / (fast - slow)));
        }
        inv_freq[i] = f * keep + f / factor * (1.0 - keep);
    }
    return SGMV_OK;
}

size_t sgmv_tree_attention_workspace_bytes(int32_t T, int32_t B, int32_t Hq, int32_t Hkv, int32_t D) {
    if (T < 1 || B < 1 || Hq < 1 || Hkv < 1 || D < 1) return 0;
    return tree_attention_workspace(T, Hq, Hkv, D);
}

int sgmv_tree_attention(const sgmv_tree_attention_args *args, void *stream) {
    set_launch_count(0);
    if (!args) return SGMV_ERR_INVALID_ARG;
    sgmv_tree_attention_args a = *args;
    bool none;
    int st = check_attention(a, 8, &none);
    if (st != SGMV_OK || none) return st;
    st = check_workspace(a.workspace, a.workspace_bytes,
                         sgmv_tree_attention_workspace_bytes(a.T, a.B, a.Hq, a.Hkv, a.D), 256);
    if (st != SGMV_OK) return st;
    int *err = device_error_word();
    if (!err) return SGMV_ERR_CUDA;
    return finish("tree attention kernel",
                  tree_attention_launch(a, device_sms(), err, static_cast<cudaStream_t>(stream)),
                  a.D <= kMmaMaxD ? 2 : 1);
}

size_t sgmv_quant_attention_workspace_bytes(int32_t T, int32_t B, int32_t Hq, int32_t Hkv, int32_t D) {
    if (T < 1 || B < 1 || Hq < 1 || Hkv < 1 || D < 1 || D > kMmaMaxD) return 0;
    return tree_mma_workspace(T, Hq / Hkv);
}

int sgmv_quant_attention(const sgmv_quant_attention_args *args, void *stream) {
    set_launch_count(0);
    if (!args) return SGMV_ERR_INVALID_ARG;
    sgmv_quant_attention_args q = *args;
    sgmv_tree_attention_args &a = q.attention;
    bool none;
    int st = check_attention(a, 16, &none);
    if (st != SGMV_OK) return st;
    if (a.D > kMmaMaxD) return SGMV_ERR_UNSUPPORTED;
    if (none) return SGMV_OK;
    if (!q.k_scale || !q.v_scale) return SGMV_ERR_INVALID_ARG;
    if (!aligned4(q.k_scale, q.v_scale)) return SGMV_ERR_ALIGNMENT;
    st = check_workspace(a.workspace, a.workspace_bytes,
                         sgmv_quant_attention_workspace_bytes(a.T, a.B, a.Hq, a.Hkv, a.D), 256);
    if (st != SGMV_OK) return st;
    int *err = device_error_word();
    if (!err) return SGMV_ERR_CUDA;
    return finish("quantised attention kernel",
                  quant_mma_launch(q, device_sms(), err, static_cast<cudaStream_t>(stream)), 2);
}

int sgmv_tree_verify(const sgmv_tree_verify_args *args, void *stream) {
    set_launch_count(0);
    if (!args) return SGMV_ERR_INVALID_ARG;
    const sgmv_tree_verify_args &a = *args;
    if (a.T < 0 || a.B < 0 || a.V < 1 || a.max_path < 1) return SGMV_ERR_INVALID_ARG;
    if (a.V > kMaxVocabulary) return SGMV_ERR_UNSUPPORTED;  // a sum of weights stays below 2^63
    if (a.B == 0) return SGMV_OK;
    if (!a.tree_ptr || !a.count || !a.path || !a.token || !a.u_sample) return SGMV_ERR_INVALID_ARG;
    if (a.T > 0 && (!a.target || !a.tokens || !a.u_accept)) return SGMV_ERR_INVALID_ARG;
    if (!aligned4(a.target, a.draft, a.tokens, a.parents, a.tree_ptr, a.u_accept, a.u_sample, a.count, a.path, a.token))
        return SGMV_ERR_ALIGNMENT;
    int *err = device_error_word();
    if (!err) return SGMV_ERR_CUDA;
    return finish("verification kernel",
                  tree_verify_launch(a, device_sms(), err, static_cast<cudaStream_t>(stream)), 1);
}

int sgmv_cache_commit(const sgmv_cache_commit_args *args, void *stream) {
    set_launch_count(0);
    if (!args) return SGMV_ERR_INVALID_ARG;
    sgmv_cache_commit_args a = *args;
    const bool e4m3 = a.dtype == SGMV_E4M3;
    if (a.layers < 0 || a.B < 0 || a.Hkv < 1 || a.max_path < 0 || (!e4m3 && !half_type(a.dtype)))
        return SGMV_ERR_INVALID_ARG;
    const int st = check_head(a.D);
    if (st != SGMV_OK) return st;
    if (a.layers > 32767) return SGMV_ERR_UNSUPPORTED;
    if (a.layers == 0 || a.B == 0 || a.max_path == 0) return SGMV_OK;
    if (!a.k_cache || !a.v_cache || !a.block_table || !a.prefix_lens || !a.path || !a.count)
        return SGMV_ERR_INVALID_ARG;
    if (a.num_blocks < 1 || a.block_size < 1 || a.max_blocks < 1 || a.table_row < 0)
        return SGMV_ERR_INVALID_ARG;
    settle(a.cache_layer, a.layers, a.D);
    settle(a.cache_block, a.num_blocks, a.D);
    settle(a.cache_token, a.block_size, a.D);
    settle(a.cache_head, a.Hkv, a.D);
    const int width = e4m3 ? 16 : 8;
    if (!vectors(a.k_cache, a.cache_block, a.cache_token, width) ||
        !vectors(a.v_cache, a.cache_head, a.cache_layer, width) || a.D % width != 0 ||
        !aligned4(a.block_table, a.prefix_lens, a.path, a.count))
        return SGMV_ERR_ALIGNMENT;
    if (e4m3) {  // the same bytes as half as many 16-bit values
        for (int64_t *s : {&a.cache_layer, &a.cache_block, &a.cache_token, &a.cache_head}) *s /= 2;
        a.D /= 2;
    }
    int *err = device_error_word();
    if (!err) return SGMV_ERR_CUDA;
    return finish("commit kernel",
                  cache_commit_launch(a, err, static_cast<cudaStream_t>(stream)), 1);
}

int sgmv_norm_rope(const sgmv_norm_rope_args *args, void *stream) {
    set_launch_count(0);
    if (!args) return SGMV_ERR_INVALID_ARG;
    sgmv_norm_rope_args n = *args;
    sgmv_rope_args &a = n.rope;
    const bool e4m3 = n.k_scale || n.v_scale;
    if (!(n.eps > 0.f) || !isfinite(n.eps) || a.inverse) return SGMV_ERR_INVALID_ARG;
    if (e4m3 && (!n.k_scale || !n.v_scale || !a.k_cache)) return SGMV_ERR_INVALID_ARG;
    bool none;
    int st = check_rope(a, e4m3 ? 16 : 8, &none);
    if (st != SGMV_OK) return st;
    if (!aligned16(n.q_weight) || !aligned16(n.k_weight) || !aligned4(n.k_scale, n.v_scale)) return SGMV_ERR_ALIGNMENT;
    if ((double)a.T * ((double)a.Hq + 2.0 * a.Hk) > kMaxRows) return SGMV_ERR_UNSUPPORTED;
    if (none) return SGMV_OK;
    uint64_t turns[kRopeMaxPairs];
    if ((st = turns_of(a.inv_freq, a.pairs, turns)) != SGMV_OK) return st;
    int *err = device_error_word();
    if (!err) return SGMV_ERR_CUDA;
    return finish("norm and rotary kernel",
                  norm_rope_launch(n, turns, device_sms(), err, static_cast<cudaStream_t>(stream)), 1);
}

size_t sgmv_norm_rope_grad_workspace_bytes(int32_t D) {
    return D < 1 || D > kSpecMaxD ? 0 : norm_rope_grad_workspace(D);
}

int sgmv_norm_rope_grad(const sgmv_norm_rope_grad_args *args, void *stream) {
    set_launch_count(0);
    if (!args) return SGMV_ERR_INVALID_ARG;
    sgmv_norm_rope_grad_args a = *args;
    if (a.T < 0 || a.Hq < 0 || a.Hk < 0 || !half_type(a.dtype) || !(a.eps > 0.f) || !isfinite(a.eps))
        return SGMV_ERR_INVALID_ARG;
    int st = check_head(a.D);
    if (st != SGMV_OK) return st;
    if (a.pairs < 0 || 2 * (int64_t)a.pairs > a.D || (a.pairs > 0 && !a.inv_freq)) return SGMV_ERR_INVALID_ARG;
    if (!a.q_weight != !a.dq_weight || !a.k_weight != !a.dk_weight || (a.Hq == 0 && a.q_weight) ||
        (a.Hk == 0 && a.k_weight))
        return SGMV_ERR_INVALID_ARG;
    if ((double)a.T * ((double)a.Hq + a.Hk) > kMaxRows) return SGMV_ERR_UNSUPPORTED;
    if (a.T == 0 && !a.dq_weight && !a.dk_weight) return SGMV_OK;
    if (a.Hq == 0 && a.Hk == 0) return SGMV_OK;
    if (a.T > 0) {
        if (!a.positions) return SGMV_ERR_INVALID_ARG;
        if (a.Hq > 0 && (!a.dq || !a.dq_out || (a.q_weight && !a.q))) return SGMV_ERR_INVALID_ARG;
        if (a.Hk > 0 && (!a.dk || !a.dk_out || (a.k_weight && !a.k))) return SGMV_ERR_INVALID_ARG;
        for (int64_t *s : {&a.dq_token, &a.dk_token, &a.dq_out_token, &a.dk_out_token, &a.q_token, &a.k_token})
            settle(*s, a.T, a.D);
        for (int64_t *s : {&a.dq_head, &a.dq_out_head, &a.q_head}) settle(*s, a.Hq, a.D);
        for (int64_t *s : {&a.dk_head, &a.dk_out_head, &a.k_head}) settle(*s, a.Hk, a.D);
        if (a.Hq > 0 && (!vectors(a.dq, a.dq_token, a.dq_head) || !vectors(a.dq_out, a.dq_out_token, a.dq_out_head) ||
                         (a.q_weight && !vectors(a.q, a.q_token, a.q_head))))
            return SGMV_ERR_ALIGNMENT;
        if (a.Hk > 0 && (!vectors(a.dk, a.dk_token, a.dk_head) || !vectors(a.dk_out, a.dk_out_token, a.dk_out_head) ||
                         (a.k_weight && !vectors(a.k, a.k_token, a.k_head))))
            return SGMV_ERR_ALIGNMENT;
    }
    if (!aligned16(a.q_weight) || !aligned16(a.k_weight) || !aligned4(a.dq_weight, a.dk_weight, a.positions))
        return SGMV_ERR_ALIGNMENT;
    const bool sums = a.dq_weight || a.dk_weight;
    if (sums) {
        st = check_workspace(a.workspace, a.workspace_bytes, norm_rope_grad_workspace(a.D), 16);
        if (st != SGMV_OK) return st;
    }
    // not in place, nor over what the other side reads or writes
    if (a.T > 0) {
        const void *const in[] = {a.Hq > 0 ? a.dq_out : nullptr, a.Hk > 0 ? a.dk_out : nullptr,
                                  a.q_weight ? a.q : nullptr, a.k_weight ? a.k : nullptr};
        for (const void *x : in)
            if (x && ((a.Hq > 0 && x == a.dq) || (a.Hk > 0 && x == a.dk))) return SGMV_ERR_INVALID_ARG;
        if (a.Hq > 0 && a.Hk > 0 && a.dq == a.dk) return SGMV_ERR_INVALID_ARG;
    }
    if (a.dq_weight && a.dq_weight == a.dk_weight) return SGMV_ERR_INVALID_ARG;
    uint64_t turns[kRopeMaxPairs];
    if ((st = turns_of(a.inv_freq, a.pairs, turns)) != SGMV_OK) return st;
    if (!device_error_word()) return SGMV_ERR_CUDA;
    return finish("norm and rotary gradient kernel",
                  norm_rope_grad_launch(a, turns, device_sms(), static_cast<cudaStream_t>(stream)),
                  (a.T > 0) + sums);
}

int sgmv_sample(const sgmv_sample_args *args, void *stream) {
    set_launch_count(0);
    if (!args) return SGMV_ERR_INVALID_ARG;
    const sgmv_sample_args &a = *args;
    if (a.T < 0 || a.V < 1 || !(half_type(a.dtype) || a.dtype == SGMV_F32)) return SGMV_ERR_INVALID_ARG;
    if (a.V > kMaxVocabulary || a.T > (1 << 27)) return SGMV_ERR_UNSUPPORTED;
    if (!a.token != !a.u) return SGMV_ERR_INVALID_ARG;
    if (a.T == 0 || (!a.token && !a.probs)) return SGMV_OK;
    if (!a.logits) return SGMV_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(a.logits) % (a.dtype == SGMV_F32 ? 4 : 2) != 0 ||
        !aligned4(a.u, a.temperature, a.top_k, a.top_p, a.min_p, a.token, a.probs))
        return SGMV_ERR_ALIGNMENT;
    if (a.probs == a.logits) return SGMV_ERR_INVALID_ARG;  // not in place
    return finish("sampling kernel", sample_launch(a, device_sms(), static_cast<cudaStream_t>(stream)), 1);
}

}  // extern "C"
