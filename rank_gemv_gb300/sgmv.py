"""Thin ctypes binding of libsgmv.so (C ABI in include/sgmv.h).

Argument marshalling only: every step of SGMV runs in the library's CUDA
kernels.  Tensors are torch tensors (PyTorch provides device memory and the
current stream); each function passes their data pointers, sizes and
``torch.cuda.current_stream()`` to the C function of the same name and raises
:class:`SgmvError` on a non-zero status.  If the library has not been built
(``__graft_entry__.build()`` or ``python -m rank_gemv_gb300.build``), loading
it raises: there is no fallback.
"""
from __future__ import annotations

import ctypes
import struct
from pathlib import Path

import torch

LIB_PATH = Path(__file__).resolve().parent / "libsgmv.so"

SGMV_F16, SGMV_BF16, SGMV_F32 = 0, 1, 2
_DTYPES = {torch.float16: SGMV_F16, torch.bfloat16: SGMV_BF16, torch.float32: SGMV_F32}

STATUS = {0: "SGMV_OK", 1: "SGMV_ERR_INVALID_ARG", 2: "SGMV_ERR_UNSUPPORTED",
          3: "SGMV_ERR_ALIGNMENT", 4: "SGMV_ERR_BAD_INDEX", 5: "SGMV_ERR_CUDA",
          6: "SGMV_ERR_WORKSPACE", 7: "SGMV_ERR_TIMEOUT", 8: "SGMV_ERR_BAD_SEGMENTS"}

# Every function include/sgmv.h declares, with its ctypes signature.
_vp, _i32, _i32p = ctypes.c_void_p, ctypes.c_int32, ctypes.POINTER(ctypes.c_int32)
_int, _f32, _sz = ctypes.c_int, ctypes.c_float, ctypes.c_size_t
_f64, _cp = ctypes.c_double, ctypes.c_char_p  # _cp: a packed argument struct
_vpp, _u64p = ctypes.POINTER(ctypes.c_void_p), ctypes.POINTER(ctypes.c_uint64)
SIGNATURES = {
    "sgmv_status_string": (ctypes.c_char_p, [_int]),
    "sgmv_last_error_string": (ctypes.c_char_p, []),
    "sgmv_last_launch_count": (_int, []),
    "sgmv_max_segments": (_i32, [_i32, _i32]),
    "sgmv_build_segments": (_int, [_vp, _i32, _i32, _vp, _vp, _vp, _vp]),
    "sgmv_build_segments_device": (_int, [_vp, _i32, _i32, _vp, _vp, _vp, _vp, _vp]),
    "sgmv_workspace_bytes": (_sz, [_i32, _i32, _i32, _i32]),
    "sgmv_shrink": (_int, [_vp, _vp, _vp, _int, _vp, _vp, _vp, _i32, _vp, _i32, _i32, _i32,
                           _i32, _vp]),
    "sgmv_expand": (_int, [_vp, _int, _vp, _vp, _int, _f32, _vp, _vp, _vp, _i32, _vp, _i32,
                           _i32, _i32, _i32, _vp]),
    "sgmv_apply": (_int, [_vp, _int, _vp, _vp, _vp, _int, _f32, _vp, _vp, _vp, _i32, _vp, _i32,
                          _i32, _i32, _i32, _i32, _vp, _sz, _vp]),
    "sgmv_apply_rows": (_int, [_vp, _int, _vp, _vp, _vp, _int, _f32, _vp, _i32, _i32, _i32, _i32,
                               _i32, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "sgmv_apply_multi": (_int, [_i32, _vpp, _int, _vpp, _vpp, _vpp, _int, _f32, _vp, _vp, _vp,
                                _i32, _vp, _i32, _i32, _i32, _i32, _i32, _vp]),
    "sgmv_apply_noalloc": (_int, [_vp, _int, _vp, _vp, _vp, _int, _f32, _vp, _vp, _vp, _i32, _vp,
                                  _i32, _i32, _i32, _i32, _i32, _vp]),
    "sgmv_fused_workspace_bytes": (_sz, [_i32, _i32, _i32]),
    "sgmv_fused_linear_lora": (_int, [_vp, _int, _vp, _vp, _vp, _vp, _int, _f32, _vp, _vp, _vp,
                                      _i32, _i32, _i32, _i32, _i32, _i32, _vp, _sz, _vp]),
    "sgmv_load_adapter": (_int, [_vp, _vp, _int, _i32, _vp, _vp, _i32, _i32, _i32, _i32, _vp]),
    "sgmv_copy_gather": (_int, [_i32, _vpp, _vpp, _u64p, _i32, _vp]),
    "sgmv_read_floor": (_int, [_vp, _sz, _i32, _i32, _i32, _i32, _i32, _int, _int, _i32p, _i32p,
                               _vp]),
    "sgmv_rope": (_int, [_cp, _vp]),
    "sgmv_rope_frequencies": (_int, [_vp, _i32, _f64, _f64, _f64, _f64, _f64]),
    "sgmv_tree_attention_workspace_bytes": (_sz, [_i32, _i32, _i32, _i32, _i32]),
    "sgmv_tree_attention": (_int, [_cp, _vp]),
    "sgmv_tree_verify": (_int, [_cp, _vp]),
    "sgmv_cache_commit": (_int, [_cp, _vp]),
    "sgmv_debug_inject_wait_timeout": (_int, [_int]),
    "sgmv_get_device_error": (_int, [_vp]),
}

_lib = None


class SgmvError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str = ""):
        self.status = status
        msg = f"{where}: {STATUS.get(status, status)}"
        super().__init__(msg + (f" ({detail})" if detail else ""))


def load_library(path: str | Path | None = None) -> ctypes.CDLL:
    """Load libsgmv.so (once) and declare its signatures."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = Path(path) if path is not None else LIB_PATH
    if not p.exists():
        raise RuntimeError(f"{p} is not built: run __graft_entry__.build() first")
    lib = ctypes.CDLL(str(p))
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    if path is None:
        _lib = lib
    return lib


def _check(rc: int, where: str):
    if rc != 0:
        detail = ""
        if rc == 5:
            detail = (load_library().sgmv_last_error_string() or b"").decode()
        raise SgmvError(rc, where, detail)


def _ptr(t):
    return None if t is None else t.data_ptr()


# pointer-array types for the multi-problem entry (P = 1 .. 4)
_PTR_ARRAYS = [None] + [ctypes.c_void_p * n for n in range(1, 5)]


def _stream(device):
    """Handle of the current stream (without a Stream object, which costs a microsecond).
    A device that is not a GPU is refused: a kernel could not use its addresses."""
    index = device.index
    if index is None:  # not a tensor's on a GPU
        if device.type != "cuda":
            raise ValueError(f"Expected a cuda device, but got: {device}")
        index = torch.cuda.current_device()
    return torch._C._cuda_getCurrentRawStream(index)


def _on_gpu(tensors):
    """Every tensor a kernel is to read or write (None: not given) must be on the GPU."""
    for t in tensors:
        if t is not None and not t.is_cuda:
            raise ValueError(f"Expected a cuda device, but got a tensor on: {t.device}")


def _meta(t, name):
    if t is None:
        return None
    if t.dtype != torch.int32 or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous int32 tensor")
    return t


def _host_i32(a):
    if a is None:
        return None
    t = torch.as_tensor(a, dtype=torch.int32, device="cpu").contiguous()
    return t


def sgmv_status_string(status: int) -> str:
    return load_library().sgmv_status_string(status).decode()


def sgmv_last_launch_count() -> int:
    """Kernels launched by this thread's last launching call."""
    return int(load_library().sgmv_last_launch_count())


def sgmv_max_segments(T: int, L: int) -> int:
    return int(load_library().sgmv_max_segments(T, L))


def sgmv_workspace_bytes(T: int, H1: int, H2: int, r: int) -> int:
    return int(load_library().sgmv_workspace_bytes(T, H1, H2, r))


def sgmv_build_segments(row_adapter, L: int):
    """Host grouping -> (perm, seg_ptr, idx) as CPU int32 tensors."""
    ra = _host_i32(row_adapter).reshape(-1)
    T = ra.numel()
    perm = torch.empty(max(T, 1), dtype=torch.int32)
    seg_ptr = torch.empty(T + 1, dtype=torch.int32)
    idx = torch.empty(max(T, 1), dtype=torch.int32)
    S = ctypes.c_int32(0)
    _check(load_library().sgmv_build_segments(ra.data_ptr(), T, L, perm.data_ptr(),
                                              seg_ptr.data_ptr(), idx.data_ptr(),
                                              ctypes.addressof(S)), "sgmv_build_segments")
    s = S.value
    return perm[:T].clone(), seg_ptr[: s + 1].clone(), idx[:s].clone()


def sgmv_build_segments_device(row_adapter: torch.Tensor, L: int, out=None):
    """Device grouping -> (perm, seg_ptr, idx, S) device int32 tensors, padded to
    sgmv_max_segments(T, L) segments (S holds the real count on the device)."""
    ra = _meta(row_adapter, "row_adapter")
    T = ra.numel()
    smax = sgmv_max_segments(T, L)
    if out is None:
        dev = ra.device
        out = (torch.empty(max(T, 1), dtype=torch.int32, device=dev),
               torch.empty(smax + 1, dtype=torch.int32, device=dev),
               torch.empty(max(smax, 1), dtype=torch.int32, device=dev),
               torch.empty(1, dtype=torch.int32, device=dev))
    perm, seg_ptr, idx, S = out
    _check(load_library().sgmv_build_segments_device(
        ra.data_ptr(), T, L, perm.data_ptr(), seg_ptr.data_ptr(), idx.data_ptr(), S.data_ptr(),
        _stream(ra.device)), "sgmv_build_segments_device")
    return perm, seg_ptr, idx, S


def _nseg(idx, S):
    return idx.numel() if S is None else int(S)


def sgmv_shrink(v, x, A, seg_ptr, idx, perm=None, seg_ptr_host=None, S=None):
    """v[p] = x[row(p)] @ A[idx[s]] (fp32), in place; returns v."""
    T, H1 = x.shape
    L, _, r = A.shape
    sph = _host_i32(seg_ptr_host)
    _check(load_library().sgmv_shrink(
        _ptr(v), _ptr(x), _ptr(A), _DTYPES[x.dtype], _ptr(_meta(perm, "perm")),
        _ptr(_meta(seg_ptr, "seg_ptr")), _ptr(_meta(idx, "idx")), _nseg(idx, S), _ptr(sph),
        T, L, H1, r, _stream(x.device)), "sgmv_shrink")
    return v


def sgmv_expand(y, v, B, seg_ptr, idx, scale=1.0, perm=None, seg_ptr_host=None, S=None):
    """y[row(p)] += scale * v[p] @ B[idx[s]], in place; returns y."""
    T, H2 = y.shape
    L, r, _ = B.shape
    sph = _host_i32(seg_ptr_host)
    _check(load_library().sgmv_expand(
        _ptr(y), _DTYPES[y.dtype], _ptr(v), _ptr(B), _DTYPES[B.dtype], float(scale),
        _ptr(_meta(perm, "perm")), _ptr(_meta(seg_ptr, "seg_ptr")), _ptr(_meta(idx, "idx")),
        _nseg(idx, S), _ptr(sph), T, L, H2, r, _stream(y.device)), "sgmv_expand")
    return y


def sgmv_apply(y, x, A, B, seg_ptr, idx, scale=1.0, perm=None, seg_ptr_host=None,
               workspace=None, S=None):
    """y[row(p)] += scale * (x[row(p)] @ A[idx[s]]) @ B[idx[s]], in place; returns y."""
    T, H1 = x.shape
    L, _, r = A.shape
    H2 = y.shape[1]
    sph = _host_i32(seg_ptr_host)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load_library().sgmv_apply(
        _ptr(y), _DTYPES[y.dtype], _ptr(x), _ptr(A), _ptr(B), _DTYPES[x.dtype], float(scale),
        _ptr(_meta(perm, "perm")), _ptr(_meta(seg_ptr, "seg_ptr")), _ptr(_meta(idx, "idx")),
        _nseg(idx, S), _ptr(sph), T, L, H1, H2, r, _ptr(workspace), ws_bytes,
        _stream(x.device)), "sgmv_apply")
    return y


def sgmv_apply_multi(ys, xs, As, Bs, seg_ptr, idx, scale=1.0, perm=None, seg_ptr_host=None,
                     S=None):
    """sgmv_apply for up to 4 problems with the same rows, segments and
    shapes (e.g. a layer's q / k / v): ys[k][row(p)] += scale * (xs[k][row(p)]
    @ As[k][idx[s]]) @ Bs[k][idx[s]], in place, in one launch when the kernel
    allows (the same bits as separate calls); returns ys."""
    P = len(ys)
    if not (len(xs) == len(As) == len(Bs) == P) or P < 1:
        raise ValueError("ys, xs, As and Bs must hold the same number (>= 1) of tensors")
    x0, y0 = xs[0], ys[0]
    T, H1 = x0.shape
    L, _, r = As[0].shape
    H2 = y0.shape[1]
    xshape, ashape, bshape, yshape = (T, H1), (L, H1, r), (L, r, H2), (T, H2)
    tin, ty = x0.dtype, y0.dtype
    for y, x, A, B in zip(ys, xs, As, Bs):
        if x.shape != xshape or A.shape != ashape or B.shape != bshape or y.shape != yshape:
            raise ValueError("the problems' shapes differ")
        if x.dtype != tin or A.dtype != tin or B.dtype != tin or y.dtype != ty:
            raise TypeError("the problems' types differ")
    arr = _PTR_ARRAYS[P] if P < len(_PTR_ARRAYS) else ctypes.c_void_p * P
    _check(load_library().sgmv_apply_multi(
        P, arr(*[t.data_ptr() for t in ys]), _DTYPES[ty], arr(*[t.data_ptr() for t in xs]),
        arr(*[t.data_ptr() for t in As]), arr(*[t.data_ptr() for t in Bs]), _DTYPES[tin],
        float(scale), _ptr(_meta(perm, "perm")), _ptr(_meta(seg_ptr, "seg_ptr")),
        _ptr(_meta(idx, "idx")), _nseg(idx, S), _ptr(_host_i32(seg_ptr_host)), T, L, H1, H2, r,
        _stream(x0.device)), "sgmv_apply_multi")
    return ys


def sgmv_apply_rows(y, x, A, B, row_adapter, scale=1.0, out=None, workspace=None):
    """Group the rows by adapter and apply SGMV in one call; returns y.

    ``out`` = (perm, seg_ptr, idx, S) device int32 tensors (as returned by
    sgmv_build_segments_device) to receive the grouping, or None.
    """
    T, H1 = x.shape
    L, _, r = A.shape
    H2 = y.shape[1]
    ra = _meta(row_adapter, "row_adapter")
    perm = seg_ptr = idx = S = None
    if out is not None:
        perm, seg_ptr, idx, S = (_meta(t, "out") for t in out)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load_library().sgmv_apply_rows(
        _ptr(y), _DTYPES[y.dtype], _ptr(x), _ptr(A), _ptr(B), _DTYPES[x.dtype], float(scale),
        _ptr(ra), T, L, H1, H2, r, _ptr(perm), _ptr(seg_ptr), _ptr(idx), _ptr(S),
        _ptr(workspace), ws_bytes, _stream(x.device)), "sgmv_apply_rows")
    return y


def sgmv_apply_noalloc(y, x, A, B, seg_ptr, idx, scale=1.0, perm=None, seg_ptr_host=None, S=None):
    """sgmv_apply without a caller-provided workspace: for callers that may not
    allocate device memory, the tensor-core path uses a fixed 4 MiB scratch
    array inside the library (see include/sgmv.h).  Calls that overlap on the
    GPU share that array and race; returns y."""
    T, H1 = x.shape
    L, _, r = A.shape
    H2 = y.shape[1]
    sph = _host_i32(seg_ptr_host)
    _check(load_library().sgmv_apply_noalloc(
        _ptr(y), _DTYPES[y.dtype], _ptr(x), _ptr(A), _ptr(B), _DTYPES[x.dtype], float(scale),
        _ptr(_meta(perm, "perm")), _ptr(_meta(seg_ptr, "seg_ptr")), _ptr(_meta(idx, "idx")),
        _nseg(idx, S), _ptr(sph), T, L, H1, H2, r, _stream(x.device)), "sgmv_apply_noalloc")
    return y


def sgmv_fused_workspace_bytes(T: int, H2: int, r: int) -> int:
    return int(load_library().sgmv_fused_workspace_bytes(T, H2, r))


def sgmv_fused_linear_lora(y, x, W, A, B, seg_ptr, idx, scale=1.0, perm=None, S=None,
                           workspace=None):
    """y = x @ W + scale * SGMV delta (the LoRA layer in one pass), written
    into y; returns y.  ``workspace`` (uint8 device tensor of at least
    sgmv_fused_workspace_bytes(T, H2, r) bytes) holds v, its tiles and the
    partial sums; one is allocated when None."""
    T, H1 = x.shape
    L, _, r = A.shape
    H2 = y.shape[1]
    if tuple(W.shape) != (H1, H2):
        raise ValueError("W must be [H1, H2]")
    if W.dtype != x.dtype:
        raise TypeError("W and x types differ")
    nseg = _nseg(idx, S) if idx is not None else 0
    if workspace is None and T > 0:
        workspace = torch.empty(sgmv_fused_workspace_bytes(T, H2, r), dtype=torch.uint8,
                                device=x.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load_library().sgmv_fused_linear_lora(
        _ptr(y), _DTYPES[y.dtype], _ptr(x), _ptr(W), _ptr(A), _ptr(B), _DTYPES[x.dtype],
        float(scale), _ptr(_meta(perm, "perm")), _ptr(_meta(seg_ptr, "seg_ptr")),
        _ptr(_meta(idx, "idx")), nseg, T, L, H1, H2, r, _ptr(workspace), ws_bytes,
        _stream(x.device)), "sgmv_fused_linear_lora")
    return y


def sgmv_load_adapter(A_pool, B_pool, slot, A_src, B_src, stream=None):
    """Copy one adapter (A_src [H1, r], B_src [r, H2]; host -- ideally pinned --
    or device tensors) into slot `slot` of the pools A_pool [L, H1, r] and
    B_pool [L, r, H2], asynchronously on `stream` (default: the current
    stream of the pools' device)."""
    L, H1, r = A_pool.shape
    H2 = B_pool.shape[2]
    if tuple(A_src.shape) != (H1, r) or tuple(B_src.shape) != (r, H2):
        raise ValueError("adapter shapes do not match the pools")
    if A_src.dtype != A_pool.dtype or B_src.dtype != B_pool.dtype or A_pool.dtype != B_pool.dtype:
        raise TypeError("adapter and pool types differ")
    for t in (A_pool, B_pool, A_src, B_src):
        if not t.is_contiguous():
            raise TypeError("tensors must be contiguous")
    st = (stream if stream is not None else torch.cuda.current_stream(A_pool.device)).cuda_stream
    _check(load_library().sgmv_load_adapter(
        _ptr(A_pool), _ptr(B_pool), _DTYPES[A_pool.dtype], int(slot), _ptr(A_src), _ptr(B_src),
        L, H1, H2, r, st), "sgmv_load_adapter")


GATHER_MAX_COPIES = 512


def sgmv_copy_gather(dsts, srcs, stream=None, max_ctas=0):
    """Copy every srcs[i] into dsts[i] (contiguous tensors of equal byte size;
    host -- ideally page-locked -- or device) on `stream` (default: the
    current stream of the current device): one kernel launch for the pairs
    the device reads directly, one copy-engine transfer for each other pair.
    More than GATHER_MAX_COPIES pairs are issued in groups."""
    if len(dsts) != len(srcs):
        raise ValueError("dsts and srcs differ in length")
    for d, s in zip(dsts, srcs):
        if not d.is_contiguous() or not s.is_contiguous():
            raise TypeError("tensors must be contiguous")
        if d.nbytes != s.nbytes:
            raise ValueError("a destination and its source differ in size")
    st = (stream if stream is not None else torch.cuda.current_stream()).cuda_stream
    lib = load_library()
    for g0 in range(0, len(dsts), GATHER_MAX_COPIES):
        part = range(g0, min(len(dsts), g0 + GATHER_MAX_COPIES))
        n = len(part)
        d = (ctypes.c_void_p * n)(*[dsts[i].data_ptr() for i in part])
        s = (ctypes.c_void_p * n)(*[srcs[i].data_ptr() for i in part])
        b = (ctypes.c_uint64 * n)(*[srcs[i].nbytes for i in part])
        _check(lib.sgmv_copy_gather(n, d, s, b, int(max_ctas), st), "sgmv_copy_gather")


# Argument structs of the speculative decoding calls (include/sgmv.h), packed
# with native sizes and alignment (0q: padded to whole 8-byte words).
_ROPE_ARGS = struct.Struct("@10P13q10if0q")
_ATTENTION_ARGS = struct.Struct("@10PQ8q9if0q")
_VERIFY_ARGS = struct.Struct("@10P2q4i0q")
_COMMIT_ARGS = struct.Struct("@6P5q9i0q")


def _heads(t, name, dtype, shape):
    """(pointer, token stride, head stride) of a [T, H, D] tensor."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {tuple(shape)}")
    s0, s1, s2 = t.stride()
    if s2 != 1 and shape[2] > 1:
        raise TypeError(f"the last dimension of {name} must be contiguous")
    return t.data_ptr(), s0, s1


def _cache(k_cache, v_cache, dtype, ndim):
    """Checked strides and shape of a pair of caches [blocks, block_size, Hkv, D]
    (ndim 5: [layers, blocks, block_size, Hkv, D])."""
    shape, stride = k_cache.shape, k_cache.stride()
    if v_cache.shape != shape or (v_cache.stride() != stride and any(
            n > 1 and a != b for n, a, b in zip(shape, stride, v_cache.stride()))):
        raise ValueError("k_cache and v_cache differ in shape or strides")
    if k_cache.dtype != dtype or v_cache.dtype != dtype:
        raise TypeError(f"the caches must be {dtype}")
    if len(shape) != ndim:
        raise ValueError("the caches must be [blocks, block_size, heads, D]")
    if stride[-1] != 1 and shape[-1] > 1:
        raise TypeError("the last dimension of the caches must be contiguous")
    return shape, stride


_I32, _F32 = torch.int32, torch.float32


def _list(t, name, n):
    """Pointer of a contiguous int32 tensor of n entries (or of None)."""
    if t is None:
        return 0
    if t.dtype != _I32 or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous int32 tensor")
    if t.numel() != n:
        raise ValueError(f"{name} must have {n} entries")
    return t.data_ptr()


def _rows(t, name, shape):
    """(pointer, row stride) of a float32 [T, V] tensor with contiguous rows (or of None)."""
    if t is None:
        return 0, 0
    s0, s1 = t.stride()
    if t.dtype != _F32 or t.shape != shape or (s1 != 1 and shape[1] > 1):
        raise TypeError(f"{name} must be float32 [T, V] with contiguous rows")
    return t.data_ptr(), s0


def _uniform(t, name, n):
    if t.dtype != _F32 or not t.is_contiguous() or t.numel() != n:
        raise TypeError(f"{name} must be a contiguous float32 tensor of {n} entries")
    return t.data_ptr()


def _table(block_table, B):
    if block_table.dtype != torch.int32 or block_table.dim() != 2 or block_table.shape[0] != B or (
            block_table.shape[1] > 1 and block_table.stride(1) != 1):
        raise TypeError("block_table must be int32 [B, max_blocks] with contiguous rows")
    return block_table.data_ptr(), block_table.shape[1], block_table.stride(0)


def sgmv_rope_frequencies(pairs, base=10000.0, factor=1.0, trained=0.0, slow=float("inf"),
                          fast=float("inf")):
    """Inverse frequencies of `pairs` rotary pairs, stretched by `factor` (see
    include/sgmv.h); a float64 CPU tensor to pass to sgmv_rope."""
    out = torch.empty(pairs, dtype=torch.float64)
    _check(load_library().sgmv_rope_frequencies(out.data_ptr(), pairs, base, factor, trained, slow,
                                                fast), "sgmv_rope_frequencies")
    return out


def sgmv_rope(q, k, positions, inv_freq, interleaved=False, scale=1.0, inverse=False, q_out=None,
              k_out=None, v=None, k_cache=None, v_cache=None, slots=None):
    """Rotary positions of q [T, Hq, D] and k [T, Hk, D] (either may be None);
    returns (q_out, k_out).

    Without q_out q is rotated in place; without k_out k is rotated in place,
    unless caches are given: then the rotated k and the unchanged v go to the
    cache slots `slots` only (-1: not appended).  inv_freq: float64 CPU tensor
    of the rotated pairs (sgmv_rope_frequencies); inverse=True turns back, the
    gradient of the rotation."""
    first = q if q is not None else k
    if first is None:
        raise ValueError("q or k must be given")
    shape, dtype = first.shape, first.dtype
    if len(shape) != 3 or dtype not in _DTYPES:
        raise TypeError("q and k must be [T, heads, D] tensors of f16 or bf16")
    T, Hq, D = shape
    if inv_freq.dtype != torch.float64 or inv_freq.is_cuda or not inv_freq.is_contiguous():
        raise TypeError("inv_freq must be a contiguous float64 CPU tensor")
    qi = qo = ki = ko = vi = (0, 0, 0)
    Hk = blocks = bs = kc = vc = 0
    cs = (0, 0, 0, 0)
    if q is not None:
        qi = _heads(q, "q", dtype, shape)
        if q_out is None:
            q_out, qo = q, qi
        else:
            qo = _heads(q_out, "q_out", dtype, shape)
    else:
        Hq = 0
        if q_out is not None:
            raise ValueError("q_out without q")
    if k is not None:
        Hk = k.shape[1]
        kshape = (T, Hk, D)
        ki = _heads(k, "k", dtype, kshape)
        if k_out is not None:
            ko = _heads(k_out, "k_out", dtype, kshape)
        elif k_cache is None:
            k_out, ko = k, ki
    elif k_out is not None:
        raise ValueError("k_out without k")
    if k_cache is None:
        if v_cache is not None or slots is not None:
            raise ValueError("v_cache and slots need k_cache")
    else:
        if k is None or v is None or v_cache is None or slots is None:
            raise ValueError("an append needs k, v, k_cache, v_cache and slots")
        cshape, cs = _cache(k_cache, v_cache, dtype, 4)
        vi = _heads(v, "v", dtype, kshape)
        blocks, bs, ch, cd = cshape
        if ch != Hk or cd != D:
            raise ValueError("the caches do not fit k")
        kc, vc = k_cache.data_ptr(), v_cache.data_ptr()
    args = _ROPE_ARGS.pack(
        qo[0], qi[0], ko[0], ki[0], vi[0], kc, vc, _list(positions, "positions", T),
        _list(slots, "slots", T), inv_freq.data_ptr(), qo[1], qo[2], qi[1], qi[2], ko[1], ko[2],
        ki[1], ki[2], vi[1], vi[2], cs[0], cs[1], cs[2], T, Hq, Hk, D, inv_freq.numel(), blocks, bs,
        _DTYPES[dtype], interleaved, inverse, scale)
    _on_gpu((q, k, q_out, k_out, v, k_cache, v_cache, positions, slots))
    _check(load_library().sgmv_rope(args, _stream(first.device)), "sgmv_rope")
    return q_out, k_out


def sgmv_tree_attention_workspace_bytes(T: int, B: int, Hq: int, Hkv: int, D: int) -> int:
    return int(load_library().sgmv_tree_attention_workspace_bytes(T, B, Hq, Hkv, D))


def sgmv_tree_attention(out, q, k_cache, v_cache, block_table, prefix_lens, tree_ptr, parents=None,
                        scale=None, lse=None, workspace=None):
    """Attention of the drafted rows q [T, Hq, D] over the paged cache [blocks,
    block_size, Hkv, D], into out; returns out.

    Row t of sequence b (tree_ptr[b] <= t < tree_ptr[b + 1]) sees the
    prefix_lens[b] tokens of its context, its ancestors by `parents` (None: a
    chain) and itself.  scale defaults to D ** -0.5; lse (fp32 [T, Hq]) receives
    the log-sum-exp.  workspace: uint8 device tensor of at least
    sgmv_tree_attention_workspace_bytes(T, B, Hq, Hkv, D) bytes (those of the
    largest T and B serve every batch); one is allocated when None."""
    qshape, dtype = q.shape, q.dtype
    if len(qshape) != 3 or dtype not in _DTYPES:
        raise TypeError("q must be a [T, heads, D] tensor of f16 or bf16")
    T, Hq, D = qshape
    B = prefix_lens.numel()
    qi, oo = _heads(q, "q", dtype, qshape), _heads(out, "out", dtype, qshape)
    shape, cs = _cache(k_cache, v_cache, dtype, 4)
    if shape[3] != D:
        raise ValueError("q and the caches differ in head size")
    if lse is not None and (lse.dtype != torch.float32 or lse.shape != (T, Hq) or not lse.is_contiguous()):
        raise TypeError("lse must be a contiguous float32 [T, Hq] tensor")
    table, width, row = _table(block_table, B)
    lib = load_library()
    if workspace is None:
        workspace = torch.empty(lib.sgmv_tree_attention_workspace_bytes(T, B, Hq, shape[2], D),
                                dtype=torch.uint8, device=q.device)
    args = _ATTENTION_ARGS.pack(
        oo[0], qi[0], k_cache.data_ptr(), v_cache.data_ptr(), 0 if lse is None else lse.data_ptr(),
        table, _list(prefix_lens, "prefix_lens", B), _list(tree_ptr, "tree_ptr", B + 1),
        _list(parents, "parents", T), workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), oo[1], oo[2], qi[1], qi[2], cs[0], cs[1],
        cs[2], row, T, B, Hq, shape[2], D, shape[0], shape[1], width, _DTYPES[dtype],
        D ** -0.5 if scale is None else scale)
    _on_gpu((q, out, k_cache, v_cache, lse, block_table, prefix_lens, tree_ptr, parents, workspace))
    _check(lib.sgmv_tree_attention(args, _stream(q.device)), "sgmv_tree_attention")
    return out


def sgmv_tree_verify(target, draft, tokens, parents, tree_ptr, u_accept, u_sample, max_path, out=None):
    """Verify drafted tokens against target [T, V] (fp32 probabilities after each
    node) and draft [T, V] (what each node's children were drawn from, or None)
    with the uniform numbers u_accept [T] and u_sample [B]; returns (count [B],
    path [B, max_path], token [B]), int32 (`out`: such a tuple to write into)."""
    shape = target.shape
    T, V = shape
    B = tree_ptr.numel() - 1
    if out is None:
        dev = target.device
        out = (torch.empty(B, dtype=_I32, device=dev), torch.empty(B, max_path, dtype=_I32, device=dev),
               torch.empty(B, dtype=_I32, device=dev))
        count, path, token = [t.data_ptr() for t in out]
    else:
        count, path, token = (_list(out[0], "count", B), _list(out[1], "path", B * max_path),
                              _list(out[2], "token", B))
    tp, t0 = _rows(target, "target", shape)
    dp, d0 = _rows(draft, "draft", shape)
    args = _VERIFY_ARGS.pack(
        tp, dp, _list(tokens, "tokens", T), _list(parents, "parents", T),
        _list(tree_ptr, "tree_ptr", B + 1), _uniform(u_accept, "u_accept", T),
        _uniform(u_sample, "u_sample", B), count, path, token, t0, d0, T, B, V, max_path)
    _on_gpu((target, draft, tokens, parents, tree_ptr, u_accept, u_sample, *out))
    _check(load_library().sgmv_tree_verify(args, _stream(target.device)), "sgmv_tree_verify")
    return out


def sgmv_cache_commit(k_cache, v_cache, block_table, prefix_lens, path, count):
    """Move the accepted nodes (path [B, max_path], count [B], as
    sgmv_tree_verify returns them) to their final places in the caches
    [blocks, block_size, Hkv, D] or [layers, blocks, block_size, Hkv, D], in place."""
    dtype = k_cache.dtype
    if dtype not in _DTYPES:
        raise TypeError("the caches must be f16 or bf16")
    ndim = 5 if k_cache.dim() == 5 else 4
    shape, cs = _cache(k_cache, v_cache, dtype, ndim)
    layers, layer_stride = (shape[0], cs[0]) if ndim == 5 else (1, 0)
    blocks, bs, Hkv, D = shape[-4:]
    B, width = path.shape
    table, max_blocks, row = _table(block_table, B)
    args = _COMMIT_ARGS.pack(
        k_cache.data_ptr(), v_cache.data_ptr(), table, _list(prefix_lens, "prefix_lens", B),
        _list(path, "path", B * width), _list(count, "count", B), layer_stride, cs[-4], cs[-3],
        cs[-2], row, layers, B, Hkv, D, blocks, bs, max_blocks, width, _DTYPES[dtype])
    _on_gpu((k_cache, v_cache, block_table, prefix_lens, path, count))
    _check(load_library().sgmv_cache_commit(args, _stream(k_cache.device)), "sgmv_cache_commit")


def sgmv_read_floor(src, nbytes, T, L, H1, H2, r, in_dtype=torch.float16, y_dtype=None):
    """Read ``nbytes`` of the device tensor ``src`` with the streaming kernel's
    launch shape for a T-row batch (see include/sgmv.h); returns
    (ctas, cluster) of the grid it launched."""
    y_dtype = in_dtype if y_dtype is None else y_dtype
    if nbytes > src.numel() * src.element_size():
        raise ValueError("nbytes beyond the source tensor")
    ctas, cl = ctypes.c_int32(0), ctypes.c_int32(0)
    _check(load_library().sgmv_read_floor(
        _ptr(src), int(nbytes), T, L, H1, H2, r, _DTYPES[in_dtype], _DTYPES[y_dtype],
        ctypes.byref(ctas), ctypes.byref(cl), _stream(src.device)), "sgmv_read_floor")
    return ctas.value, cl.value


def sgmv_debug_inject_wait_timeout(enable: int) -> None:
    """Make this thread's launches of the streaming kernel, and of the tree attention
    in the role of this number, take the timeout path at their first wait (tests of
    device-side timeout reporting; see include/sgmv.h)."""
    _check(load_library().sgmv_debug_inject_wait_timeout(int(enable)),
           "sgmv_debug_inject_wait_timeout")


def sgmv_get_device_error(device=None) -> int:
    """Synchronise the current stream, read and clear the device error word."""
    dev = torch.device("cuda") if device is None else torch.device(device)
    return int(load_library().sgmv_get_device_error(_stream(dev)))
