"""Python binding of the C ABI in include/*.h (ctypes).

Argument marshalling only: torch tensors are passed as device pointers and
the current CUDA stream as a handle; every step of the computation runs in
the library's CUDA kernels.  Importing fails loudly when the library has not
been built -- there is no fallback path.
"""
from __future__ import annotations

import ctypes
import os

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_lib", "libfpsparse.so")

FP_OK, FP_ERR_ARG, FP_ERR_CUDA, FP_ERR_TIMEOUT, FP_ERR_STATE, FP_ERR_RANGE = 0, 1, 2, 3, 4, 5
FP_QK_BF16, FP_QK_INT8 = 0, 1
FP_PATTERN_VS, FP_PATTERN_QA = 0, 1
FP_DT_BF16, FP_DT_F16, FP_DT_F32, FP_DT_INT8, FP_DT_E4M3 = 0, 1, 2, 3, 4
FP_ROPE_HALF, FP_ROPE_INTERLEAVED = 0, 1
FP_ROPE_NONE, FP_ROPE_LINEAR, FP_ROPE_BASE, FP_ROPE_BANDS, FP_ROPE_RAMP = 0, 1, 2, 3, 4

SYMBOLS = ("fp_index_create", "fp_index_free", "fp_build_index", "fp_sparse_attn", "fp_index_info",
           "fp_index_nnz", "fp_index_export", "fp_get_device_error", "fp_debug_wait_timeout",
           "fp_debug_qk_tile_i8", "fp_debug_capture_i8", "fp_pattern_stats_noalloc", "fp_strerror",
           "fp_index_share", "fp_index_classes", "fp_choose_block_size", "fp_index_csr",
           "fp_index_group_lists",
           "fp_prefill_create", "fp_prefill_free", "fp_prefill_enqueue", "fp_prefill_wait", "fp_prefill_run",
           "fp_prefill_group_index", "fp_varlen_create", "fp_varlen_free", "fp_varlen_build_index",
           "fp_varlen_sparse_attn", "fp_varlen_index", "fp_rope_pool", "fp_build_index_pooled",
           "fp_rope_create", "fp_rope_free", "fp_rope_freqs", "fp_rope_apply",
           "fp_kv_create", "fp_kv_free", "fp_kv_write", "fp_kv_read", "fp_tree_attn_workspace", "fp_tree_attn")


class FpError(RuntimeError):
    def __init__(self, code, where):
        super().__init__(f"{where}: {fp_strerror(code)} (code {code})")
        self.code = code


def _load():
    if not os.path.exists(_LIB_PATH):
        raise ImportError(f"CUDA library not built: {_LIB_PATH} is missing "
                          "(run python -m dynamic_block_sparse_last_b200.build)")
    L = ctypes.CDLL(_LIB_PATH)
    vp, i, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    L.fp_index_create.argtypes = [i, i, i, i, i, ctypes.POINTER(vp)]
    L.fp_index_free.argtypes = [vp]
    L.fp_index_free.restype = None
    L.fp_build_index.argtypes = [vp, vp, i, i, i, i, i, f, f, i, vp, vp, vp, vp]
    L.fp_sparse_attn.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp]
    L.fp_index_info.argtypes = [vp] + [ctypes.POINTER(i)] * 6
    L.fp_index_nnz.argtypes = [vp, ctypes.POINTER(ctypes.c_int64), vp]
    L.fp_index_export.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp]
    L.fp_get_device_error.argtypes = [vp]
    L.fp_debug_wait_timeout.argtypes = [i, vp]
    L.fp_debug_qk_tile_i8.argtypes = [vp, vp, i, i, i, i, i, i, i, vp, vp]
    L.fp_debug_capture_i8.argtypes = [i, i, i, i, vp]
    L.fp_index_share.argtypes = [vp, f, vp]
    L.fp_index_csr.argtypes = [vp, vp, vp, vp]
    L.fp_index_group_lists.argtypes = [vp, vp, vp, vp, vp]
    L.fp_index_classes.argtypes = [vp, vp, vp]
    L.fp_choose_block_size.argtypes = [vp, f, ctypes.POINTER(i), ctypes.POINTER(f), vp]
    L.fp_pattern_stats_noalloc.argtypes = [vp, vp, i, i, i, i, i, f, i, vp, vp, vp, vp, vp, vp, vp, vp]
    L.fp_strerror.argtypes = [i]
    L.fp_strerror.restype = ctypes.c_char_p
    L.fp_prefill_create.argtypes = [i, i, i, i, i, i, i, ctypes.POINTER(vp)]
    L.fp_prefill_free.argtypes = [vp]
    L.fp_prefill_free.restype = None
    L.fp_prefill_run.argtypes = [vp, vp, vp, vp, vp, vp, f, f, vp, vp]
    L.fp_prefill_enqueue.argtypes = [vp, vp, vp, vp, vp, vp, f, f, vp, vp]
    L.fp_prefill_wait.argtypes = [vp, vp]
    L.fp_prefill_group_index.argtypes = [vp, i, ctypes.POINTER(vp)]
    L.fp_rope_pool.argtypes = [vp, vp, vp, vp, i, i, i, i, i, vp, vp, vp, vp, vp]
    L.fp_build_index_pooled.argtypes = [vp, vp, vp, vp, i, i, i, i, i, f, f, vp, vp]
    L.fp_varlen_create.argtypes = [vp, i, i, i, i, i, ctypes.POINTER(vp)]
    L.fp_varlen_free.argtypes = [vp]
    L.fp_varlen_free.restype = None
    L.fp_varlen_build_index.argtypes = [vp, vp, vp, f, f, i, vp, vp, vp]
    L.fp_varlen_sparse_attn.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp]
    L.fp_varlen_index.argtypes = [vp, i, ctypes.POINTER(vp)]
    n, dbl, sz = ctypes.c_int64, ctypes.c_double, ctypes.c_size_t
    L.fp_rope_create.argtypes = [i, i, i, dbl, i, dbl, dbl, dbl, dbl, dbl, ctypes.POINTER(vp)]
    L.fp_rope_freqs.argtypes = [vp, vp]
    L.fp_rope_apply.argtypes = [vp] + [vp, n, n] * 4 + [i, i, i, i, vp, i, vp]
    L.fp_kv_create.argtypes = [vp, vp, vp, vp, i, n, i, i, i, ctypes.POINTER(vp)]
    L.fp_kv_write.argtypes = [vp] + [vp, n, n] * 2 + [i, i, vp, vp]
    L.fp_kv_read.argtypes = [vp, vp, i, vp, vp, i, i] + [vp, n, n] * 2 + [i, vp]
    L.fp_tree_attn_workspace.argtypes = [i] * 5
    L.fp_tree_attn_workspace.restype = sz
    L.fp_tree_attn.argtypes = [vp, vp, n, n, i, i, i, vp, i, vp, vp, i, i, vp, f, vp, n, n, vp, vp, sz, vp]
    for name in ("fp_rope_free", "fp_kv_free"):
        getattr(L, name).argtypes = [vp]
        getattr(L, name).restype = None
    for s in SYMBOLS:
        if s not in ("fp_index_free", "fp_strerror", "fp_prefill_free", "fp_varlen_free", "fp_rope_free", "fp_kv_free",
                     "fp_tree_attn_workspace"):
            getattr(L, s).restype = i
    return L


_lib = _load()


def lib():
    return _lib


def library_path():
    return _LIB_PATH


def _ptr(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream if torch.cuda.is_available() else None
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(rc, where):
    if rc != FP_OK:
        raise FpError(rc, where)


def fp_strerror(code: int) -> str:
    return _lib.fp_strerror(int(code)).decode()


class Index:
    """Owns one fp_index handle (device workspace for one layer shape)."""

    def __init__(self, handle, S, Hq, Hkv, d, b):
        self.handle = handle
        self.S, self.Hq, self.Hkv, self.d, self.b = S, Hq, Hkv, d, b
        self.n = (S + b - 1) // b

    def free(self):
        if self.handle:
            _lib.fp_index_free(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass


def fp_index_create(S, Hq, Hkv, d, b) -> Index:
    h = ctypes.c_void_p()
    _check(_lib.fp_index_create(S, Hq, Hkv, d, b, ctypes.byref(h)), "fp_index_create")
    return Index(h.value, S, Hq, Hkv, d, b)


def fp_index_free(idx: Index):
    idx.free()


def fp_build_index(q, k, S, Hq, Hkv, d, b, gamma, tau, qk_dtype, q_scale, k_scale, idx: Index, stream=None):
    _check(_lib.fp_build_index(_ptr(q), _ptr(k), S, Hq, Hkv, d, b, float(gamma), float(tau), int(qk_dtype),
                               _ptr(q_scale), _ptr(k_scale), idx.handle, _stream(stream)), "fp_build_index")


def fp_sparse_attn(q, k, v, q_scale, k_scale, idx: Index, out, stream=None):
    _check(_lib.fp_sparse_attn(_ptr(q), _ptr(k), _ptr(v), _ptr(q_scale), _ptr(k_scale), idx.handle,
                               _ptr(out), _stream(stream)), "fp_sparse_attn")


def fp_rope_pool(q_in, k_in, rope_cos, rope_sin, S, Hq, Hkv, d, b, q_out, k_out, qbar, kbar, stream=None):
    """Rotary embedding of bf16 q_in/k_in into q_out/k_out (may alias) plus block means."""
    _check(_lib.fp_rope_pool(_ptr(q_in), _ptr(k_in), _ptr(rope_cos), _ptr(rope_sin), S, Hq, Hkv, d, b, _ptr(q_out),
                             _ptr(k_out), _ptr(qbar), _ptr(kbar), _stream(stream)), "fp_rope_pool")


def fp_build_index_pooled(q, k, qbar, kbar, S, Hq, Hkv, d, b, gamma, tau, idx: Index, stream=None):
    _check(_lib.fp_build_index_pooled(_ptr(q), _ptr(k), _ptr(qbar), _ptr(kbar), S, Hq, Hkv, d, b, float(gamma),
                                      float(tau), idx.handle, _stream(stream)), "fp_build_index_pooled")


def fp_index_info(idx: Index):
    vals = [ctypes.c_int() for _ in range(6)]
    _check(_lib.fp_index_info(idx.handle, *[ctypes.byref(v) for v in vals]), "fp_index_info")
    return dict(zip(("S", "Hq", "Hkv", "d", "b", "qk_dtype"), [v.value for v in vals]))


def fp_index_nnz(idx: Index, stream=None) -> int:
    v = ctypes.c_int64()
    _check(_lib.fp_index_nnz(idx.handle, ctypes.byref(v), _stream(stream)), "fp_index_nnz")
    return v.value


def fp_index_export(idx: Index, stream=None):
    """Host copies: CSR (row_ptr, col) over rows h*n + r, pattern, jsd, vhat, shat, pest."""
    import numpy as np
    nnz = fp_index_nnz(idx, stream)
    Hn = idx.Hq * idx.n
    row_ptr = np.zeros(Hn + 1, dtype=np.int32)
    col = np.zeros(max(nnz, 1), dtype=np.int32)
    pattern = np.zeros(idx.Hq, dtype=np.uint8)
    jsd = np.zeros(idx.Hq, dtype=np.float32)
    vhat = np.zeros(Hn, dtype=np.float32)
    shat = np.zeros(Hn, dtype=np.float32)
    pest = np.zeros(Hn, dtype=np.float32)
    _check(_lib.fp_index_export(idx.handle, row_ptr.ctypes.data, col.ctypes.data, pattern.ctypes.data,
                                jsd.ctypes.data, vhat.ctypes.data, shat.ctypes.data, pest.ctypes.data,
                                _stream(stream)), "fp_index_export")
    return {"row_ptr": row_ptr, "col": col[:nnz], "pattern": pattern, "jsd": jsd,
            "vhat": vhat.reshape(idx.Hq, idx.n), "shat": shat.reshape(idx.Hq, idx.n),
            "pest": pest.reshape(idx.Hq, idx.n), "nnz": nnz}


def fp_get_device_error(stream=None) -> int:
    return int(_lib.fp_get_device_error(_stream(stream)))


def fp_debug_wait_timeout(timeout_us: int, stream=None):
    _check(_lib.fp_debug_wait_timeout(int(timeout_us), _stream(stream)), "fp_debug_wait_timeout")


def fp_debug_qk_tile_i8(q8, k8, S, Hq, Hkv, d, h, p0, j0, out, stream=None):
    _check(_lib.fp_debug_qk_tile_i8(_ptr(q8), _ptr(k8), S, Hq, Hkv, d, h, p0, j0, _ptr(out), _stream(stream)),
           "fp_debug_qk_tile_i8")


def fp_index_share(idx, eps, stream=None):
    """Head-pattern sharing on a built index: classes by JSD of vhat < eps
    within each GQA group, every member's lists replaced by the class union."""
    _check(_lib.fp_index_share(idx.handle, float(eps), _stream(stream)), "fp_index_share")


def fp_index_csr(idx, row_ptr, col=None, stream=None):
    """Device CSR of the index into caller-owned device int32 tensors
    (row_ptr [Hq*n + 1], col [nnz] or None for the offsets only)."""
    _check(_lib.fp_index_csr(idx.handle, _ptr(row_ptr), _ptr(col), _stream(stream)), "fp_index_csr")


def fp_index_group_lists(idx, grp_ptr, grp_col=None, grp_mask=None, stream=None):
    """Per-(KV head, query block) union lists with head masks into caller-owned
    device tensors (grp_ptr int32 [Hkv*n + 1]; grp_col int32, grp_mask int32
    bit patterns [total], or both None for the offsets only)."""
    _check(_lib.fp_index_group_lists(idx.handle, _ptr(grp_ptr), _ptr(grp_col), _ptr(grp_mask), _stream(stream)),
           "fp_index_group_lists")


def fp_index_classes(idx, stream=None):
    import numpy as np
    cls = np.zeros(idx.Hq, dtype=np.int32)
    _check(_lib.fp_index_classes(idx.handle, cls.ctypes.data, _stream(stream)), "fp_index_classes")
    return cls


def fp_choose_block_size(idx, gamma, stream=None):
    """Block size chosen by the content rule from an index built at b = 128: (b, rho)."""
    b, rho = ctypes.c_int(0), ctypes.c_float(0.0)
    _check(_lib.fp_choose_block_size(idx.handle, float(gamma), ctypes.byref(b), ctypes.byref(rho), _stream(stream)),
           "fp_choose_block_size")
    return b.value, rho.value


def fp_debug_capture_i8(which, h, tile, chunk, out):
    """Arms (out a device int32 [128][128] tensor) or disarms (out None) the
    capture of one raw int8 score tile: which 0 = index pass, 1 = attention."""
    _check(_lib.fp_debug_capture_i8(int(which), int(h), int(tile), int(chunk), _ptr(out)), "fp_debug_capture_i8")


def fp_pattern_stats_noalloc(q, k, S, Hq, Hkv, d, b, tau, qk_dtype, q_scale, k_scale, vhat, shat, pest, jsd,
                             pattern, stream=None):
    """Per-head vhat/shat/pest/jsd/pattern into caller-owned device buffers,
    using the library's fixed scratch array instead of any allocation."""
    _check(_lib.fp_pattern_stats_noalloc(_ptr(q), _ptr(k), S, Hq, Hkv, d, b, float(tau), int(qk_dtype),
                                         _ptr(q_scale), _ptr(k_scale), _ptr(vhat), _ptr(shat), _ptr(pest),
                                         _ptr(jsd), _ptr(pattern), _stream(stream)), "fp_pattern_stats_noalloc")


class Prefill:
    """Owns one fp_prefill pipeline (include/fp_prefill.h): device copies of a
    layer and one index per KV-head group, for host-to-host runs."""

    def __init__(self, S, Hq, Hkv, d, b, qk_dtype=FP_QK_BF16, groups=0):
        h = ctypes.c_void_p()
        _check(_lib.fp_prefill_create(S, Hq, Hkv, d, b, int(qk_dtype), int(groups), ctypes.byref(h)),
               "fp_prefill_create")
        self.handle = h.value
        self.S, self.Hq, self.Hkv, self.d, self.b, self.qk_dtype = S, Hq, Hkv, d, b, qk_dtype
        self.groups = groups if groups else Hkv

    def run(self, h_q, h_k, h_v, h_q_scale, h_k_scale, gamma, tau, h_out, stream=None):
        """Host tensors in, host tensor out (pinned for overlap); asynchronous on `stream`."""
        _check(_lib.fp_prefill_run(self.handle, _ptr(h_q), _ptr(h_k), _ptr(h_v), _ptr(h_q_scale),
                                   _ptr(h_k_scale), float(gamma), float(tau), _ptr(h_out), _stream(stream)),
               "fp_prefill_run")

    def enqueue(self, h_q, h_k, h_v, h_q_scale, h_k_scale, gamma, tau, h_out, stream=None):
        """Queues a run; consecutive runs overlap.  h_out is ready after wait()."""
        _check(_lib.fp_prefill_enqueue(self.handle, _ptr(h_q), _ptr(h_k), _ptr(h_v), _ptr(h_q_scale),
                                       _ptr(h_k_scale), float(gamma), float(tau), _ptr(h_out), _stream(stream)),
               "fp_prefill_enqueue")

    def wait(self, stream=None):
        """Makes `stream` wait for the outputs of every queued run."""
        _check(_lib.fp_prefill_wait(self.handle, _stream(stream)), "fp_prefill_wait")

    def group_index(self, group):
        """The fp_index of KV-head group `group` of the last run (owned by the pipeline)."""
        h = ctypes.c_void_p()
        _check(_lib.fp_prefill_group_index(self.handle, int(group), ctypes.byref(h)), "fp_prefill_group_index")
        hkv = self.Hkv // self.groups if self.groups <= self.Hkv else 1
        idx = Index(h.value, self.S, self.Hq // self.groups, hkv, self.d, self.b)
        idx.free = lambda: None  # owned by the pipeline
        return idx

    def free(self):
        if self.handle:
            _lib.fp_prefill_free(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass


class Varlen:
    """Owns one fp_varlen set (include/fp_sparse.h): one index per packed
    sequence; cu_seqlens is a host sequence of nseq + 1 offsets."""

    def __init__(self, cu_seqlens, Hq, Hkv, d, b):
        import numpy as np
        cu = np.ascontiguousarray(np.asarray(cu_seqlens, dtype=np.int32))
        h = ctypes.c_void_p()
        _check(_lib.fp_varlen_create(cu.ctypes.data, len(cu) - 1, Hq, Hkv, d, b, ctypes.byref(h)),
               "fp_varlen_create")
        self.handle = h.value
        self.cu, self.Hq, self.Hkv, self.d, self.b = [int(c) for c in cu], Hq, Hkv, d, b

    def build_index(self, q, k, gamma, tau, qk_dtype, q_scale=None, k_scale=None, stream=None):
        _check(_lib.fp_varlen_build_index(self.handle, _ptr(q), _ptr(k), float(gamma), float(tau), int(qk_dtype),
                                          _ptr(q_scale), _ptr(k_scale), _stream(stream)), "fp_varlen_build_index")

    def sparse_attn(self, q, k, v, out, q_scale=None, k_scale=None, stream=None):
        _check(_lib.fp_varlen_sparse_attn(self.handle, _ptr(q), _ptr(k), _ptr(v), _ptr(q_scale), _ptr(k_scale),
                                          _ptr(out), _stream(stream)), "fp_varlen_sparse_attn")

    def index(self, seq):
        """The Index of sequence `seq` (owned by the set), or None when it is empty."""
        h = ctypes.c_void_p()
        _check(_lib.fp_varlen_index(self.handle, int(seq), ctypes.byref(h)), "fp_varlen_index")
        if not h.value:
            return None
        idx = Index(h.value, self.cu[seq + 1] - self.cu[seq], self.Hq, self.Hkv, self.d, self.b)
        idx.free = lambda: None  # owned by the set
        return idx

    def free(self):
        if self.handle:
            _lib.fp_varlen_free(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass


# ---------------------------------------------------------------- fp_decode.h
# Tensors of tokens are torch tensors [heads, tokens, d] with any strides whose
# last one is 1 (head-major tensors, or transposed views of token-major rows).

_DTYPES = {torch.bfloat16: FP_DT_BF16, torch.float16: FP_DT_F16, torch.float32: FP_DT_F32, torch.int8: FP_DT_INT8,
           torch.float8_e4m3fn: FP_DT_E4M3}


def _refuse(where, why):
    raise FpError(FP_ERR_ARG, f"{where}: {why}")


# The checks below run before every call of a few microseconds, so they are few
# and read each property of a tensor once.

def _here(where, t):
    """The device of t, which must be the current one: its stream is the one used."""
    dev = t.get_device()
    if dev < 0:
        _refuse(where, "tensors must be on a CUDA device")
    if dev != torch.cuda.current_device():
        _refuse(where, f"tensors on cuda:{dev}, which is not the current device")
    return dev


def _raw_stream(stream, dev):
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _table(where, name, t, dtype, shape, dev):
    """Address of a contiguous tensor of this type and shape."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        _refuse(where, f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on cuda:{dev}")
    return t.data_ptr()


def _tokens(where, name, t, dtype, shape, dev):
    """Address, token stride and head stride of a [heads, tokens, d] tensor."""
    st = t.stride()
    if t.dtype is not dtype or t.shape != shape or st[2] != 1 or t.get_device() != dev:
        _refuse(where, f"{name} must be a {dtype} tensor of shape {tuple(shape)} with contiguous elements on cuda:{dev}")
    return t.data_ptr(), st[1], st[0]


_NONE = (None, 0, 0)


class Rope:
    """The rotary frequencies of one model (fp_rope; host memory only).  The
    first rot_dim (default: all) of d elements of a head are rotated; scaling
    is one of FP_ROPE_*, with its parameters as include/fp_decode.h says."""

    def __init__(self, d, rot_dim=None, layout=FP_ROPE_HALF, theta=10000.0, scaling=FP_ROPE_NONE, factor=1.0,
                 orig_len=0.0, low=0.0, high=0.0, amplitude=1.0):
        self.handle = None
        self.d, self.rot_dim, self.layout = d, d if rot_dim is None else rot_dim, layout
        h = ctypes.c_void_p()
        _check(_lib.fp_rope_create(d, self.rot_dim, layout, theta, scaling, factor, orig_len, low, high, amplitude,
                                   ctypes.byref(h)), "fp_rope_create")
        self.handle = h.value

    def freqs(self):
        """Radians per position of the rot_dim/2 pairs, fp64."""
        import numpy as np
        f = np.zeros(self.rot_dim // 2)
        _check(_lib.fp_rope_freqs(self.handle, f.ctypes.data), "fp_rope_freqs")
        return f

    def apply(self, q_in, k_in, q_out, k_out, pos, inverse=False, stream=None):
        """Rotates q_in [Hq, T, d] and k_in [Hkv, T, d] (either may be None, with its
        output) by the positions pos (int32 [T]) into q_out, k_out (which may be the
        inputs); inverse: the transpose, the gradient of the inputs."""
        where, x = "fp_rope_apply", q_in if q_in is not None else k_in
        if x is None or x.dim() != 3:
            _refuse(where, "q or k must be given, as [heads, tokens, d]")
        if (q_in is None) != (q_out is None) or (k_in is None) != (k_out is None):
            _refuse(where, "an input and its output go together")
        dev, T, dt = _here(where, x), x.shape[1], x.dtype
        hq = hkv = 0
        qi = qo = ki = ko = _NONE
        if q_in is not None:
            hq = q_in.shape[0]
            shape = (hq, T, self.d)
            qi, qo = _tokens(where, "q_in", q_in, dt, shape, dev), _tokens(where, "q_out", q_out, dt, shape, dev)
        if k_in is not None:
            hkv = k_in.shape[0]
            shape = (hkv, T, self.d)
            ki, ko = _tokens(where, "k_in", k_in, dt, shape, dev), _tokens(where, "k_out", k_out, dt, shape, dev)
        _check(_lib.fp_rope_apply(self.handle, *qi, *ki, *qo, *ko, _DTYPES.get(dt, -1), T, hq, hkv,
                                  _table(where, "pos", pos, torch.int32, (T,), dev), inverse, _raw_stream(stream, dev)), where)

    def free(self):
        if self.handle:
            _lib.fp_rope_free(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass


class KvCache:
    """A paged key/value cache over caller-owned pools (fp_kv): k_pool, v_pool
    [pages, Hkv, page, d] bf16, fp16, int8 or float8_e4m3fn, and for the latter two
    k_scale, v_scale fp32 [pages, Hkv, page].  The pools are kept alive."""

    def __init__(self, k_pool, v_pool, k_scale=None, v_scale=None):
        self.handle = None
        where = "fp_kv_create"
        if k_pool.dim() != 4:
            _refuse(where, "pools are [pages, Hkv, page, d]")
        pages, self.Hkv, self.page, self.d = k_pool.shape
        dev = _here(where, k_pool)
        ptr = [_table(where, n, t, k_pool.dtype, k_pool.shape, dev) for n, t in (("k_pool", k_pool), ("v_pool", v_pool))]
        ptr += [t if t is None else _table(where, n, t, torch.float32, k_pool.shape[:3], dev)
                for n, t in (("k_scale", k_scale), ("v_scale", v_scale))]
        self.pools, self.pages, self.device = (k_pool, v_pool, k_scale, v_scale), pages, dev
        h = ctypes.c_void_p()
        _check(_lib.fp_kv_create(*ptr, _DTYPES.get(k_pool.dtype, -1), pages, self.page, self.Hkv, self.d, ctypes.byref(h)),
               where)
        self.handle = h.value

    def write(self, k, v, slots, stream=None):
        """Writes the tokens k, v [Hkv, T, d] (either may be None) to slots (int64 [T],
        page * page_size + offset; negative: skipped), quantising each row."""
        where, x = "fp_kv_write", k if k is not None else v
        if x is None or x.dim() != 3:
            _refuse(where, "k or v must be given, as [heads, tokens, d]")
        dev, T, dt = self.device, x.shape[1], x.dtype
        shape = (self.Hkv, T, self.d)
        kk = _NONE if k is None else _tokens(where, "k", k, dt, shape, dev)
        vv = _NONE if v is None else _tokens(where, "v", v, dt, shape, dev)
        _check(_lib.fp_kv_write(self.handle, *kk, *vv, _DTYPES.get(dt, -1), T,
                                _table(where, "slots", slots, torch.int64, (T,), dev), _raw_stream(stream, dev)), where)

    def read(self, block_table, cu_seqlens, k, v, first=None, stream=None):
        """Reads cached tokens into k, v [Hkv, T, d] (either may be None): rows
        cu_seqlens[s] .. cu_seqlens[s+1]-1 receive the tokens first[s] (default 0), ..
        of sequence s.  block_table int32 [nseq, max_pages], cu_seqlens int32
        [nseq + 1], first int32 [nseq], on the device."""
        where, x = "fp_kv_read", k if k is not None else v
        if x is None or x.dim() != 3 or block_table.dim() != 2:
            _refuse(where, "k or v must be given, as [heads, tokens, d], and block_table is [nseq, max_pages]")
        dev, T, dt = self.device, x.shape[1], x.dtype
        shape = (self.Hkv, T, self.d)
        kk = _NONE if k is None else _tokens(where, "k", k, dt, shape, dev)
        vv = _NONE if v is None else _tokens(where, "v", v, dt, shape, dev)
        nseq, width = block_table.shape
        _check(_lib.fp_kv_read(self.handle, _table(where, "block_table", block_table, torch.int32, (nseq, width), dev), width,
                               _table(where, "cu_seqlens", cu_seqlens, torch.int32, (nseq + 1,), dev),
                               first if first is None else _table(where, "first", first, torch.int32, (nseq,), dev),
                               nseq, T, *kk, *vv, _DTYPES.get(dt, -1), _raw_stream(stream, dev)), where)

    def free(self):
        if self.handle:
            _lib.fp_kv_free(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass


def fp_tree_attn_workspace(nseq, max_q, Hq, Hkv, d) -> int:
    """Bytes of workspace of fp_tree_attn on the current device, for at most max_q new tokens a sequence."""
    n = _lib.fp_tree_attn_workspace(nseq, max_q, Hq, Hkv, d)
    if n == 0:
        _refuse("fp_tree_attn_workspace", "sizes out of range, or no usable device")
    return n


def fp_tree_attn(q, kv: KvCache, block_table, kv_len, cu_q, max_q, mask, scale, out, work, lse=None, stream=None):
    """Attention of the new tokens q [Hq, T, d] (rows cu_q[s] .. of sequence s, at
    most max_q each) over the kv_len[s] cached tokens of their sequences, the last
    of which are the new ones; mask int64 [T, ceil(max_q/64)] (bit j of row i: token
    i sees new token j of its sequence) or None for j <= i.  Into out [Hq, T, d] and
    lse fp32 [Hq, T]; work: a uint8 tensor of fp_tree_attn_workspace bytes."""
    where = "fp_tree_attn"
    if q.dim() != 3 or block_table.dim() != 2:
        _refuse(where, "q is [Hq, T, d], block_table [nseq, max_pages]")
    dev, dt = kv.device, q.dtype
    Hq, T, _ = q.shape
    nseq, width = block_table.shape
    shape = (Hq, T, kv.d)
    if not work.is_contiguous() or work.get_device() != dev:
        _refuse(where, f"work must be contiguous, on cuda:{dev}")
    _check(_lib.fp_tree_attn(kv.handle, *_tokens(where, "q", q, dt, shape, dev), _DTYPES.get(dt, -1), T, Hq,
                             _table(where, "block_table", block_table, torch.int32, (nseq, width), dev), width,
                             _table(where, "kv_len", kv_len, torch.int32, (nseq,), dev),
                             _table(where, "cu_q", cu_q, torch.int32, (nseq + 1,), dev), nseq, max_q,
                             mask if mask is None else _table(where, "mask", mask, torch.int64, (T, (max_q + 63) // 64), dev),
                             scale, *_tokens(where, "out", out, dt, shape, dev),
                             lse if lse is None else _table(where, "lse", lse, torch.float32, (Hq, T), dev),
                             work.data_ptr(), work.nbytes, _raw_stream(stream, dev)), where)
