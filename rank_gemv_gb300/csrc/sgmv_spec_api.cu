// sgmv_spec_api.cu -- the C ABI of the speculative decoding operators:
// argument checks and launches.
#include <math.h>

#include <climits>

#include "sgmv.h"
#include "sgmv_internal.h"
#include "sgmv_spec.h"

namespace {

using namespace sgmv;

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool half_type(int dt) { return dt == SGMV_F16 || dt == SGMV_BF16; }

// 16-bit data read and written in 16-byte pieces
bool vectors(const void *p, int64_t s0, int64_t s1) {
    return aligned16(p) && s0 % 8 == 0 && s1 % 8 == 0;
}

// The stride of a dimension of one entry is never used and may be anything: it
// becomes one that passes the checks here and fits a tensor map.
void settle(int64_t &stride, int32_t entries, int32_t D) {
    if (entries == 1) stride = D;
}

int check_head(int32_t D) {
    if (D < 1) return SGMV_ERR_INVALID_ARG;
    if (D % 8 != 0) return SGMV_ERR_ALIGNMENT;
    return D > kSpecMaxD ? SGMV_ERR_UNSUPPORTED : SGMV_OK;
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
    if (a.T < 0 || a.Hq < 0 || a.Hk < 0 || !half_type(a.dtype)) return SGMV_ERR_INVALID_ARG;
    const int st = check_head(a.D);
    if (st != SGMV_OK) return st;
    if (a.pairs < 0 || 2 * (int64_t)a.pairs > a.D || (a.pairs > 0 && !a.inv_freq))
        return SGMV_ERR_INVALID_ARG;
    const bool append = a.k_cache || a.v_cache || a.slots;
    if (append && (!a.k_cache || !a.v_cache || !a.slots || a.num_blocks < 1 || a.block_size < 1))
        return SGMV_ERR_INVALID_ARG;
    if (a.T == 0 || (a.Hq == 0 && a.Hk == 0)) return SGMV_OK;
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
    if (append && (!vectors(a.v, a.v_token, a.v_head) || !vectors(a.k_cache, a.cache_block, a.cache_token) ||
                   !vectors(a.v_cache, a.cache_head, 0)))
        return SGMV_ERR_ALIGNMENT;
    // turns per position, modulo one turn, as a fraction of 2^64
    uint64_t turns[kRopeMaxPairs];
    for (int i = 0; i < a.pairs; ++i) {
        const double f = a.inv_freq[i] * 0.15915494309189533577;  // 1 / (2 pi)
        if (!(fabs(f) < 1e15)) return SGMV_ERR_INVALID_ARG;
        const double part = f - floor(f);  // [0, 1]
        turns[i] = part < 1.0 ? (uint64_t)(part * 0x1p64) : 0;
    }
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
    if (a.T < 0 || a.B < 0 || a.Hq < 1 || a.Hkv < 1 || a.Hq % a.Hkv != 0 || !half_type(a.dtype) ||
        !(a.scale == a.scale))
        return SGMV_ERR_INVALID_ARG;
    const int st = check_head(a.D);
    if (st != SGMV_OK) return st;
    if (a.T == 0 || a.B == 0) return SGMV_OK;
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
        !vectors(a.k_cache, a.cache_block, a.cache_token) || !vectors(a.v_cache, a.cache_head, 0))
        return SGMV_ERR_ALIGNMENT;
    if (a.workspace_bytes < sgmv_tree_attention_workspace_bytes(a.T, a.B, a.Hq, a.Hkv, a.D) || !a.workspace)
        return SGMV_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(a.workspace) % 256 != 0) return SGMV_ERR_ALIGNMENT;
    int *err = device_error_word();
    if (!err) return SGMV_ERR_CUDA;
    return finish("tree attention kernel",
                  tree_attention_launch(a, device_sms(), err, static_cast<cudaStream_t>(stream)),
                  a.D <= kMmaMaxD ? 2 : 1);
}

int sgmv_tree_verify(const sgmv_tree_verify_args *args, void *stream) {
    set_launch_count(0);
    if (!args) return SGMV_ERR_INVALID_ARG;
    const sgmv_tree_verify_args &a = *args;
    if (a.T < 0 || a.B < 0 || a.V < 1 || a.max_path < 1) return SGMV_ERR_INVALID_ARG;
    if (a.V > (1 << 24)) return SGMV_ERR_UNSUPPORTED;  // a sum of weights stays below 2^63
    if (a.B == 0) return SGMV_OK;
    if (!a.tree_ptr || !a.count || !a.path || !a.token || !a.u_sample) return SGMV_ERR_INVALID_ARG;
    if (a.T > 0 && (!a.target || !a.tokens || !a.u_accept)) return SGMV_ERR_INVALID_ARG;
    if (!aligned4(a.target) || !aligned4(a.draft)) return SGMV_ERR_ALIGNMENT;
    int *err = device_error_word();
    if (!err) return SGMV_ERR_CUDA;
    return finish("verification kernel",
                  tree_verify_launch(a, device_sms(), err, static_cast<cudaStream_t>(stream)), 1);
}

int sgmv_cache_commit(const sgmv_cache_commit_args *args, void *stream) {
    set_launch_count(0);
    if (!args) return SGMV_ERR_INVALID_ARG;
    sgmv_cache_commit_args a = *args;
    if (a.layers < 0 || a.B < 0 || a.Hkv < 1 || a.max_path < 0 || !half_type(a.dtype))
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
    if (!vectors(a.k_cache, a.cache_block, a.cache_token) ||
        !vectors(a.v_cache, a.cache_head, a.cache_layer))
        return SGMV_ERR_ALIGNMENT;
    int *err = device_error_word();
    if (!err) return SGMV_ERR_CUDA;
    return finish("commit kernel",
                  cache_commit_launch(a, err, static_cast<cudaStream_t>(stream)), 1);
}

}  // extern "C"
