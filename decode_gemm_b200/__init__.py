"""Python binding of libunweight (lossless BF16 weight compression fused with the matmul).

Argument marshalling only: every step of the computation runs in the CUDA
library ``libunweight.so`` built in this directory (``python
decode_gemm_b200/build.py``).  Importing this package fails loudly when the
library is missing; there is no Python or CPU fallback.

The functions carry the names of the C ABI in ``include/unweight.h``.  Tensors
are ``torch`` tensors on the GPU (device memory and streams come from torch);
host arrays are ``numpy`` arrays.  A device tensor goes to the library as its
data pointer, as in the C ABI: it must be contiguous, on the handle's device
and at least as large as the header states for that argument (nothing here
checks its size).  Every call raises :class:`UwError` when the library returns
a status other than ``UW_OK``.
"""
from __future__ import annotations

import ctypes as C
import os
import struct

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libunweight.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with `python decode_gemm_b200/build.py` "
        "(nvcc, sm_100a). There is no fallback implementation.")

lib = C.CDLL(LIB_PATH)

# ----------------------------------------------------------------- constants --
UW_OK, UW_ERR_ARG, UW_ERR_SHAPE, UW_ERR_FORMAT, UW_ERR_UNSUPPORTED = 0, 1, 2, 3, 4
UW_ERR_OOM, UW_ERR_CUDA, UW_ERR_DEVICE, UW_ERR_TIMEOUT, UW_ERR_WORKSPACE = 5, 6, 7, 8, 9
UW_ERR_IO = 10
UW_PIPE_AUTO, UW_PIPE_FULL, UW_PIPE_EXP, UW_PIPE_PALETTE_RT, UW_PIPE_PALETTE_DIRECT = 0, 1, 2, 3, 4
UW_FLAG_BAD_INPUT, UW_FLAG_TIMEOUT = 1, 2   # bits of the serving calls' flags word
UW_PIPE_HUFFMAN_DIRECT = 5   # the Huffman-direct product (M <= DOT_MAX_M)
DOT_MAX_M = 8     # tokens the Huffman-direct product serves per call
PIPELINES = {"full": UW_PIPE_FULL, "exp": UW_PIPE_EXP, "palette_rt": UW_PIPE_PALETTE_RT,
             "palette_direct": UW_PIPE_PALETTE_DIRECT}


class uw_encode_opts(C.Structure):
    _fields_ = [("max_code_len", C.c_int32), ("chunk_syms", C.c_int32),
                ("prepare_direct", C.c_int32), ("reserved", C.c_int32)]


class uw_format(C.Structure):
    _fields_ = [
        ("N", C.c_int64), ("K", C.c_int64),
        ("max_code_len", C.c_int32), ("chunk_syms", C.c_int32),
        ("code_len", C.c_uint8 * 256), ("palette", C.c_uint8 * 16),
        ("n_words", C.c_int64), ("words", C.POINTER(C.c_uint32)),
        ("n_chunks", C.c_int64), ("chunk_off", C.POINTER(C.c_uint32)),
        ("sm", C.POINTER(C.c_uint8)),
        ("n_esc_words", C.c_int64), ("esc_bits", C.POINTER(C.c_uint32)),
        ("n_esc_groups", C.c_int64), ("esc_off", C.POINTER(C.c_uint32)),
        ("n_esc_rows", C.c_int64), ("esc_exp", C.POINTER(C.c_uint8)),
    ]


class uw_stats_t(C.Structure):
    _fields_ = [
        ("N", C.c_int64), ("K", C.c_int64),
        ("bits_per_exponent", C.c_double), ("entropy_bits", C.c_double),
        ("top16_coverage", C.c_double),
        ("n_rows", C.c_int64), ("n_escape_rows", C.c_int64),
        ("max_len_used", C.c_int32), ("n_symbols", C.c_int32),
        ("bytes_stream", C.c_int64), ("bytes_offsets", C.c_int64), ("bytes_sm", C.c_int64),
        ("bytes_escape", C.c_int64), ("bytes_palette_idx", C.c_int64),
        ("bytes_huffman_bundle", C.c_int64), ("bytes_palette_bundle", C.c_int64),
    ]

    def as_dict(self):
        return {name: getattr(self, name) for name, _ in self._fields_}


class uw_gemm_config(C.Structure):
    _fields_ = [("pipeline", C.c_int32), ("tile_n", C.c_int32), ("stages", C.c_int32),
                ("gemm_ctas", C.c_int32), ("decode_ctas", C.c_int32), ("halves", C.c_int32),
                ("pair", C.c_int32), ("gemv", C.c_int32)]

    def as_dict(self):
        return {k: getattr(self, k) for k in ("pipeline", "tile_n", "stages", "gemm_ctas",
                                               "decode_ctas", "halves", "pair", "gemv")}


class uw_mlp_layer(C.Structure):
    _fields_ = [("gate", C.c_void_p), ("up", C.c_void_p), ("down", C.c_void_p)]


class uw_mlp_opts(C.Structure):
    _fields_ = [("overlap", C.c_int32), ("decode_ctas", C.c_int32), ("gemm_ctas", C.c_int32),
                ("reserved", C.c_int32)]

    def as_dict(self):
        return {k: getattr(self, k) for k in ("overlap", "decode_ctas", "gemm_ctas")}


_vp, _i32, _i64, _sz = C.c_void_p, C.c_int32, C.c_int64, C.c_size_t


class uw_paged_cache(C.Structure):
    _fields_ = [("k_dev", _vp), ("v_dev", _vp), ("n_pages", _i64), ("page_stride", _i64),
                ("slot_stride", _i64), ("head_stride", _i64), ("page_size", _i32),
                ("n_kv_heads", _i32), ("head_dim", _i32), ("reserved", _i32)]


class uw_paged_plan_args(C.Structure):
    _fields_ = [(n, _vp) for n in ("ctx_len_dev", "new_len_dev", "free_pages_dev", "head_in_dev",
                                   "head_out_dev", "table_dev", "cu_q_dev", "kv_len_dev",
                                   "positions_dev", "slots_dev", "flags_dev")] + [
        ("table_stride", _i64), ("n_rows", _i64), ("n_requests", _i32), ("table_width", _i32),
        ("n_free", _i32), ("page_size", _i32)]


class uw_qk_norm_rope_args(C.Structure):
    _fields_ = [(n, _vp) for n in ("q_dev", "k_dev", "v_dev", "q_weight_dev", "k_weight_dev",
                                   "positions_dev", "inv_freq_dev", "slots_dev", "q_out_dev",
                                   "flags_dev")] + [
        ("cache", uw_paged_cache), ("n_rows", _i64), ("q_stride", _i64), ("k_stride", _i64),
        ("v_stride", _i64), ("q_out_stride", _i64), ("n_heads", _i32), ("rot_dim", _i32),
        ("interleaved", _i32), ("eps", C.c_float)]


class uw_paged_attention_args(C.Structure):
    _fields_ = [(n, _vp) for n in ("q_dev", "table_dev", "cu_q_dev", "kv_len_dev", "out_dev",
                                   "lse_dev", "flags_dev", "ws_dev")] + [
        ("cache", uw_paged_cache), ("ws_bytes", _sz), ("n_rows", _i64), ("q_stride", _i64),
        ("out_stride", _i64), ("table_stride", _i64), ("n_requests", _i32), ("table_width", _i32),
        ("n_heads", _i32), ("window", _i32), ("out_f32", _i32), ("scale", C.c_float)]


class uw_sample_args(C.Structure):
    _fields_ = [(n, _vp) for n in ("logits_dev", "u_dev", "temperature_dev", "top_k_dev",
                                   "top_p_dev", "min_p_dev", "ids_dev", "prob_dev")] + [
        ("n_rows", _i64), ("row_stride", _i64), ("vocab", _i32), ("logits_bf16", _i32)]


_SIGS = {
    "uw_status_str": ([C.c_int], C.c_char_p),
    "uw_abi_version": ([], C.c_int),
    "uw_default_encode_opts": ([C.POINTER(uw_encode_opts)], None),
    "uw_encode_host": ([_vp, _i64, _i64, C.POINTER(uw_encode_opts), C.POINTER(_vp)], C.c_int),
    "uw_host_view": ([_vp, C.POINTER(uw_format)], C.c_int),
    "uw_host_free": ([_vp], None),
    "uw_validate_format": ([C.POINTER(uw_format)], C.c_int),
    "uw_host_stats": ([_vp, C.POINTER(uw_stats_t)], C.c_int),
    "uw_host_save": ([_vp, C.c_char_p], C.c_int),
    "uw_host_load": ([C.c_char_p, C.POINTER(_vp)], C.c_int),
    "uw_load": ([C.c_char_p, C.POINTER(uw_encode_opts), _vp, C.POINTER(_vp)], C.c_int),
    "uw_upload": ([C.POINTER(uw_format), C.POINTER(uw_encode_opts), _vp, C.POINTER(_vp)], C.c_int),
    "uw_encode": ([_vp, _i64, _i64, C.POINTER(uw_encode_opts), _vp, C.POINTER(_vp)], C.c_int),
    "uw_free": ([_vp], C.c_int),
    "uw_set_stream": ([_vp, _vp], C.c_int),
    "uw_stats": ([_vp, C.POINTER(uw_stats_t)], C.c_int),
    "uw_workspace_bytes": ([_vp, _i32, _i64, C.POINTER(_sz)], C.c_int),
    "uw_set_workspace": ([_vp, _vp, _sz], C.c_int),
    "uw_alloc_workspace": ([_vp, _sz], C.c_int),
    "uw_decode_full": ([_vp, _vp], C.c_int),
    "uw_decode_exp": ([_vp, _vp], C.c_int),
    "uw_decode_rows": ([_vp, _vp, _i64, _vp], C.c_int),
    "uw_transcode_palette": ([_vp, _vp], C.c_int),
    "uw_gemm": ([_vp, _vp, _vp, _i64, C.c_int], C.c_int),
    "uw_gemm_f32": ([_vp, _vp, _vp, _i64, C.c_int], C.c_int),
    "uw_gemm_ex": ([_vp, _vp, _vp, _i64, C.POINTER(uw_gemm_config), _i32], C.c_int),
    "uw_autotune": ([C.POINTER(_vp), _i32, C.POINTER(_i64), _i32, C.c_char_p], C.c_int),
    "uw_load_profile": ([C.POINTER(_vp), _i32, C.c_char_p], C.c_int),
    "uw_get_choice": ([_vp, _i64, C.POINTER(uw_gemm_config)], C.c_int),
    "uw_last_device_status": ([_vp], C.c_int),
    "uw_trace_enable": ([_vp, _i32], C.c_int),
    "uw_gemm_palette_noalloc": ([_vp, _vp, _vp, _i64, _i32], C.c_int),
    "uw_swiglu": ([_vp, _vp, _vp, _i64, _vp], C.c_int),
    "uw_mlp_workspace_bytes": ([C.POINTER(uw_mlp_layer), _i32, _i64, C.POINTER(uw_mlp_opts),
                                C.POINTER(_sz)], C.c_int),
    "uw_mlp_forward": ([C.POINTER(uw_mlp_layer), _i32, _vp, _vp, _i64, _vp, _sz, _vp, _vp,
                        C.POINTER(uw_mlp_opts)], C.c_int),
    "uw_mlp_forward_record": ([C.POINTER(uw_mlp_layer), _i32, _vp, _vp, _i64, _vp, _sz, _vp,
                               _vp, C.POINTER(uw_mlp_opts), _vp], C.c_int),
    "uw_mlp_tune_split": ([C.POINTER(uw_mlp_layer), _i32, _vp, _vp, _i64, _vp, _sz, _vp, _vp,
                           C.POINTER(uw_mlp_opts)], C.c_int),
    "uw_paged_plan": ([C.POINTER(uw_paged_plan_args), _vp], C.c_int),
    "uw_qk_norm_rope": ([C.POINTER(uw_qk_norm_rope_args), _vp], C.c_int),
    "uw_paged_attention_workspace_bytes": ([_i32, _i32, _i32, C.POINTER(_sz)], C.c_int),
    "uw_paged_attention": ([C.POINTER(uw_paged_attention_args), _vp], C.c_int),
    "uw_sample": ([C.POINTER(uw_sample_args), _vp], C.c_int),
    "uw_trace_read": ([_vp, C.POINTER(_i32), C.POINTER(C.c_float), _i32, C.POINTER(_i32)], C.c_int),
}
for _name, (_args, _res) in _SIGS.items():
    _f = getattr(lib, _name)
    _f.argtypes = _args
    _f.restype = _res

EXPORTED = tuple(_SIGS)


class UwError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = int(status)
        super().__init__(f"{what}: {uw_status_str(status)} ({status})")


def uw_status_str(status: int) -> str:
    return lib.uw_status_str(int(status)).decode()


def _check(status: int, what: str) -> None:
    if status != UW_OK:
        raise UwError(status, what)


def default_opts(**kw) -> uw_encode_opts:
    o = uw_encode_opts()
    lib.uw_default_encode_opts(C.byref(o))
    for k, v in kw.items():
        setattr(o, k, int(v))
    return o


def _stream_ptr(stream) -> int | None:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    return getattr(stream, "cuda_stream", stream)


def _dptr(t) -> int:
    return int(t.data_ptr())


# ------------------------------------------------------------------ host side --

class HostEncoded:
    """Host-side encoding (``uw_encode_host``); numpy views via :meth:`arrays`."""

    def __init__(self, ptr):
        self._ptr = _vp(ptr)
        # (module globals may be gone when __del__ runs at interpreter exit)
        self._free, self._null = lib.uw_host_free, _vp(0)

    @property
    def ptr(self):
        return self._ptr

    def view(self) -> uw_format:
        f = uw_format()
        _check(lib.uw_host_view(self._ptr, C.byref(f)), "uw_host_view")
        return f

    def arrays(self) -> dict:
        return format_arrays(self.view())

    def stats(self) -> dict:
        s = uw_stats_t()
        _check(lib.uw_host_stats(self._ptr, C.byref(s)), "uw_host_stats")
        return s.as_dict()

    def __del__(self):
        ptr, free = getattr(self, "_ptr", None), getattr(self, "_free", None)
        if ptr is not None and ptr.value and free is not None:
            free(ptr)
            self._ptr = self._null


def uw_encode_host(w: np.ndarray, opts: uw_encode_opts | None = None) -> HostEncoded:
    w = np.ascontiguousarray(w, dtype=np.uint16)
    n, k = w.shape
    out = _vp()
    _check(lib.uw_encode_host(w.ctypes.data, n, k, C.byref(opts) if opts else None,
                              C.byref(out)), "uw_encode_host")
    return HostEncoded(out.value)


def format_arrays(f: uw_format) -> dict:
    """Copy every array of a format view into numpy."""
    def arr(ptr, n, dt):
        n = int(n)
        if n == 0:
            return np.zeros(0, dt)
        return np.ctypeslib.as_array(ptr, shape=(n,)).copy().astype(dt)
    return dict(
        N=f.N, K=f.K, max_code_len=f.max_code_len, chunk_syms=f.chunk_syms,
        code_len=np.array(f.code_len[:], np.uint8), palette=np.array(f.palette[:], np.uint8),
        words=arr(f.words, f.n_words, np.uint32),
        chunk_off=arr(f.chunk_off, f.n_chunks + 1, np.uint32),
        sm=arr(f.sm, f.N * f.K, np.uint8),
        esc_bits=arr(f.esc_bits, f.n_esc_words, np.uint32),
        esc_off=arr(f.esc_off, f.n_esc_groups + 1, np.uint32),
        esc_exp=arr(f.esc_exp, f.n_esc_rows * 64, np.uint8),
    )


class FormatBuffers:
    """A ``uw_format`` that points into numpy arrays it keeps alive."""

    def __init__(self, N, K, max_code_len, chunk_syms, code_len, palette, words, chunk_off, sm,
                 esc_bits, esc_off, esc_exp):
        self._keep = []

        def ptr(a, ct):
            a = np.ascontiguousarray(a)
            self._keep.append(a)
            return a.ctypes.data_as(C.POINTER(ct))

        f = uw_format()
        f.N, f.K = int(N), int(K)
        f.max_code_len, f.chunk_syms = int(max_code_len), int(chunk_syms)
        f.code_len[:] = [int(x) for x in np.asarray(code_len, np.uint8)]
        f.palette[:] = [int(x) for x in np.asarray(palette, np.uint8)]
        words = np.asarray(words, np.uint32)
        f.n_words, f.words = words.size, ptr(words, C.c_uint32)
        chunk_off = np.asarray(chunk_off, np.uint32)
        f.n_chunks, f.chunk_off = chunk_off.size - 1, ptr(chunk_off, C.c_uint32)
        f.sm = ptr(np.asarray(sm, np.uint8).reshape(-1), C.c_uint8)
        esc_bits = np.asarray(esc_bits, np.uint32).reshape(-1)
        f.n_esc_words, f.esc_bits = esc_bits.size, ptr(esc_bits, C.c_uint32)
        esc_off = np.asarray(esc_off, np.uint32)
        f.n_esc_groups, f.esc_off = esc_off.size - 1, ptr(esc_off, C.c_uint32)
        esc_exp = np.asarray(esc_exp, np.uint8).reshape(-1)
        f.n_esc_rows = esc_exp.size // 64
        f.esc_exp = ptr(esc_exp if esc_exp.size else np.zeros(64, np.uint8), C.c_uint8)
        self.fmt = f


def uw_validate_format(fmt: uw_format) -> int:
    """Returns the status code (does not raise): UW_OK or an error."""
    return int(lib.uw_validate_format(C.byref(fmt)))


# ---------------------------------------------------------------- device side --

class Handle:
    """A device-resident encoded matrix (``uw_handle_t``)."""

    def __init__(self, ptr, N, K):
        self._ptr = _vp(ptr)
        self.N, self.K = int(N), int(K)
        self._ws = None  # torch tensor kept alive while registered
        # (module globals may be gone when __del__ runs at interpreter exit)
        self._free, self._null = lib.uw_free, _vp(0)

    @property
    def ptr(self):
        return self._ptr

    def stats(self) -> dict:
        s = uw_stats_t()
        _check(lib.uw_stats(self._ptr, C.byref(s)), "uw_stats")
        return s.as_dict()

    def free(self):
        ptr = getattr(self, "_ptr", None)
        if ptr is not None and ptr.value:
            self._free(ptr)
            self._ptr = self._null

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass


def uw_host_save(h: HostEncoded, path: str) -> None:
    """Write a host encoding to a bundle file (see include/unweight.h)."""
    _check(lib.uw_host_save(h.ptr, os.fsencode(path)), "uw_host_save")


def uw_host_load(path: str) -> HostEncoded:
    """Read a bundle file into a host encoding (checksummed and validated)."""
    out = _vp()
    _check(lib.uw_host_load(os.fsencode(path), C.byref(out)), "uw_host_load")
    return HostEncoded(out.value)


def uw_load(path: str, opts: uw_encode_opts | None = None, stream=None) -> Handle:
    """A bundle file straight to the device (uw_host_load + uw_upload)."""
    out = _vp()
    _check(lib.uw_load(os.fsencode(path), C.byref(opts) if opts else None,
                       _vp(_stream_ptr(stream)), C.byref(out)), "uw_load")
    h = Handle(out.value, 0, 0)
    st = h.stats()
    h.N, h.K = int(st["N"]), int(st["K"])
    return h


def uw_upload(fmt: uw_format, opts: uw_encode_opts | None = None, stream=None) -> Handle:
    out = _vp()
    _check(lib.uw_upload(C.byref(fmt), C.byref(opts) if opts else None,
                         _vp(_stream_ptr(stream)), C.byref(out)), "uw_upload")
    return Handle(out.value, fmt.N, fmt.K)


def uw_encode(w: np.ndarray, opts: uw_encode_opts | None = None, stream=None) -> Handle:
    w = np.ascontiguousarray(w, dtype=np.uint16)
    n, k = w.shape
    out = _vp()
    _check(lib.uw_encode(w.ctypes.data, n, k, C.byref(opts) if opts else None,
                         _vp(_stream_ptr(stream)), C.byref(out)), "uw_encode")
    return Handle(out.value, n, k)


def uw_free(h: Handle) -> None:
    h.free()


def uw_set_stream(h: Handle, stream=None) -> None:
    _check(lib.uw_set_stream(h.ptr, _vp(_stream_ptr(stream))), "uw_set_stream")


def uw_stats(h: Handle) -> dict:
    return h.stats()


def uw_workspace_bytes(h: Handle, pipeline: int, M: int) -> int:
    out = _sz()
    _check(lib.uw_workspace_bytes(h.ptr, int(pipeline), int(M), C.byref(out)),
           "uw_workspace_bytes")
    return int(out.value)


def uw_set_workspace(h: Handle, ws) -> None:
    """Register a caller-owned device buffer (a torch tensor; kept alive here)."""
    if ws is None:
        _check(lib.uw_set_workspace(h.ptr, None, 0), "uw_set_workspace")
        h._ws = None
        return
    nbytes = ws.numel() * ws.element_size()
    _check(lib.uw_set_workspace(h.ptr, _vp(_dptr(ws)), nbytes), "uw_set_workspace")
    h._ws = ws


def uw_alloc_workspace(h: Handle, nbytes: int) -> None:
    _check(lib.uw_alloc_workspace(h.ptr, int(nbytes)), "uw_alloc_workspace")


def uw_decode_full(h: Handle, w_out) -> None:
    _check(lib.uw_decode_full(h.ptr, _vp(_dptr(w_out))), "uw_decode_full")


def uw_decode_exp(h: Handle, e_out) -> None:
    _check(lib.uw_decode_exp(h.ptr, _vp(_dptr(e_out))), "uw_decode_exp")


def uw_transcode_palette(h: Handle, idx_out) -> None:
    _check(lib.uw_transcode_palette(h.ptr, _vp(_dptr(idx_out))), "uw_transcode_palette")


def uw_decode_rows(h: Handle, rows, out) -> None:
    """BF16 rows `rows` (device int64 tensor) of the encoded matrix into `out`
    ([len(rows), K] on the device): an embedding lookup on compressed weights."""
    _check(lib.uw_decode_rows(h.ptr, _vp(_dptr(rows)), int(rows.numel()), _vp(_dptr(out))),
           "uw_decode_rows")


def uw_gemm(h: Handle, X, Y, M: int, pipeline: int = UW_PIPE_AUTO) -> None:
    _check(lib.uw_gemm(h.ptr, _vp(_dptr(X)), _vp(_dptr(Y)), int(M), int(pipeline)), "uw_gemm")


def uw_gemm_f32(h: Handle, X, Y, M: int, pipeline: int = UW_PIPE_AUTO) -> None:
    _check(lib.uw_gemm_f32(h.ptr, _vp(_dptr(X)), _vp(_dptr(Y)), int(M), int(pipeline)),
           "uw_gemm_f32")


def gemm_config(pipeline: int, tile_n: int = 0, stages: int = 0, gemm_ctas: int = 0,
                decode_ctas: int = 0, halves: int = 0, pair: int = 0,
                gemv: int = 0) -> uw_gemm_config:
    """A variant: gemv = 1 selects the CUDA-core matrix-vector kernel (M <= 2),
    0 the tensor-core GEMM."""
    c = uw_gemm_config()
    c.pipeline, c.tile_n, c.stages = int(pipeline), int(tile_n), int(stages)
    c.gemm_ctas, c.decode_ctas, c.halves = int(gemm_ctas), int(decode_ctas), int(halves)
    c.pair, c.gemv = int(pair), int(gemv)
    return c


def uw_gemm_ex(h: Handle, X, Y, M: int, cfg: uw_gemm_config, out_f32: bool) -> None:
    _check(lib.uw_gemm_ex(h.ptr, _vp(_dptr(X)), _vp(_dptr(Y)), int(M), C.byref(cfg),
                          1 if out_f32 else 0), "uw_gemm_ex")


def uw_gemm_palette_noalloc(h: Handle, X, Y, M: int, out_f32: bool = False) -> None:
    """Pipeline-4 matmul that allocates nothing (split-K scratch is a fixed
    array inside the library); M <= 64.  See include/unweight.h."""
    _check(lib.uw_gemm_palette_noalloc(h.ptr, _vp(_dptr(X)), _vp(_dptr(Y)), int(M),
                                       1 if out_f32 else 0), "uw_gemm_palette_noalloc")


def uw_swiglu(g, u, h, n: int | None = None, stream=None) -> None:
    n = g.numel() if n is None else int(n)
    _check(lib.uw_swiglu(_vp(_dptr(g)), _vp(_dptr(u)), _vp(_dptr(h)), n,
                         _vp(_stream_ptr(stream))), "uw_swiglu")


def mlp_layers(layers):
    """[(gate, up, down) Handles] -> ctypes array of uw_mlp_layer."""
    arr = (uw_mlp_layer * len(layers))()
    for i, (g, u, d) in enumerate(layers):
        arr[i].gate, arr[i].up, arr[i].down = g.ptr.value, u.ptr.value, d.ptr.value
    return arr


def mlp_opts(overlap=False, decode_ctas=0, gemm_ctas=0) -> uw_mlp_opts:
    o = uw_mlp_opts()
    o.overlap, o.decode_ctas, o.gemm_ctas = int(bool(overlap)), int(decode_ctas), int(gemm_ctas)
    return o


def uw_mlp_workspace_bytes(layers, M: int, opts: uw_mlp_opts | None = None) -> int:
    arr = mlp_layers(layers)
    out = _sz()
    _check(lib.uw_mlp_workspace_bytes(arr, len(layers), int(M), C.byref(opts) if opts else None,
                                      C.byref(out)), "uw_mlp_workspace_bytes")
    return int(out.value)


def uw_mlp_forward(layers, X, Y, M: int, ws, opts: uw_mlp_opts | None = None, stream=None,
                   side_stream=None) -> None:
    arr = mlp_layers(layers)
    nbytes = ws.numel() * ws.element_size()
    side = _vp(_stream_ptr(side_stream)) if side_stream is not None else None
    _check(lib.uw_mlp_forward(arr, len(layers), _vp(_dptr(X)), _vp(_dptr(Y)), int(M),
                              _vp(_dptr(ws)), nbytes, _vp(_stream_ptr(stream)), side,
                              C.byref(opts) if opts else None), "uw_mlp_forward")


def uw_mlp_forward_record(layers, X, Y, M: int, ws, act, opts: uw_mlp_opts | None = None,
                          stream=None, side_stream=None) -> None:
    """uw_mlp_forward, also writing each layer's g, u, h and output into act
    (device, per layer M*(3F + D) BF16 values in that order)."""
    arr = mlp_layers(layers)
    nbytes = ws.numel() * ws.element_size()
    side = _vp(_stream_ptr(side_stream)) if side_stream is not None else None
    _check(lib.uw_mlp_forward_record(arr, len(layers), _vp(_dptr(X)), _vp(_dptr(Y)), int(M),
                                     _vp(_dptr(ws)), nbytes, _vp(_stream_ptr(stream)), side,
                                     C.byref(opts) if opts else None, _vp(_dptr(act))),
           "uw_mlp_forward_record")


def uw_mlp_tune_split(layers, X, Y, M: int, ws, stream=None, side_stream=None) -> uw_mlp_opts:
    arr = mlp_layers(layers)
    best = uw_mlp_opts()
    nbytes = ws.numel() * ws.element_size()
    _check(lib.uw_mlp_tune_split(arr, len(layers), _vp(_dptr(X)), _vp(_dptr(Y)), int(M),
                                 _vp(_dptr(ws)), nbytes, _vp(_stream_ptr(stream)),
                                 _vp(_stream_ptr(side_stream)), C.byref(best)),
           "uw_mlp_tune_split")
    return best


# --------------------------------------------------------------- a serving step --
#
# These calls take their sizes from the tensors, so the tensors are checked:
# their type, their size, and that all lie on one device.  `stream` defaults to
# the current stream of that device.  A decoding step makes such calls between
# kernels of a few microseconds, so the checks are few and the arguments are
# packed in one go (a ctypes structure of 25 fields costs three times as much).

_TYPES: dict = {}   # dtype sets, filled at the first call (torch is imported by its users)
_raw_stream = None  # device number -> its current stream


def _types():
    global _raw_stream
    if not _TYPES:
        import torch
        _raw_stream = torch._C._cuda_getCurrentRawStream
        bf16 = (torch.bfloat16, torch.int16, torch.uint16)
        _TYPES.update(bf16=bf16, f32=(torch.float32,), i32=(torch.int32,), i64=(torch.int64,),
                      u32=(torch.int32, torch.uint32), u8=(torch.uint8,), real=(torch.float32,) + bf16)
    return _TYPES


def _struct_of(cls):
    codes = {_vp: "P", _i64: "q", _sz: "N", _i32: "i", C.c_float: "f"}
    return "".join(_struct_of(t) if t is uw_paged_cache else codes[t] for _, t in cls._fields_)


_PACK_PLAN, _PACK_ROPE, _PACK_ATTENTION, _PACK_SAMPLE = (
    struct.Struct("@" + _struct_of(c)).pack
    for c in (uw_paged_plan_args, uw_qk_norm_rope_args, uw_paged_attention_args, uw_sample_args))


def _refuse(call, dev, t, what, kinds, size):
    if t.dtype not in kinds:
        raise UwError(UW_ERR_ARG, f"{call}: {what} is {t.dtype}, not one of {kinds}")
    if t.get_device() != dev:
        raise UwError(UW_ERR_ARG, f"{call}: {what} is on {t.device}, not on the first tensor's device")
    if (t.numel() if type(size) is int else t.shape) != size:
        raise UwError(UW_ERR_SHAPE, f"{call}: {what} is {tuple(t.shape)}, not {size}")
    raise UwError(UW_ERR_ARG, f"{call}: {what} is not packed: strides {t.stride()}")


def _vectors(call, dev, specs):
    """Pointers of packed tensors (tensor or None, name, dtypes, number of elements)."""
    out = []
    for t, what, kinds, n in specs:
        if t is None:
            out.append(0)
        elif t.dtype in kinds and t.numel() == n and t.get_device() == dev and t.is_contiguous():
            out.append(t.data_ptr())
        else:
            _refuse(call, dev, t, what, kinds, n)
    return out


def _rows(call, dev, t, what, kinds, shape):
    """(pointer, elements from row to row) of a tensor whose rows are packed."""
    strides = t.stride()
    if t.dtype not in kinds or t.get_device() != dev or t.shape != shape:
        _refuse(call, dev, t, what, kinds, shape)
    if len(shape) == 3:
        _, n, m = shape
        if (strides[2] != 1 and m > 1) or (strides[1] != m and n > 1):
            _refuse(call, dev, t, what, kinds, shape)
        width = n * m
    else:
        width = shape[1]
        if strides[1] != 1 and width > 1:
            _refuse(call, dev, t, what, kinds, shape)
    return t.data_ptr(), strides[0] if shape[0] > 1 else width


def _cache_fields(call, dev, k, v, dim):
    """uw_paged_cache of keys and values [page, slot, head, dim], in any order in memory."""
    kinds, shape = _TYPES["bf16"], k.shape
    if len(shape) != 4 or shape[3] != dim:
        raise UwError(UW_ERR_SHAPE, f"{call}: k_cache is {tuple(shape)}, not (pages, page_size, heads, {dim})")
    strides, of_v = k.stride(), v.stride()
    if 1 in shape and v.shape == shape:  # (no stride of an axis of one entry means anything: the same for both)
        strides, of_v = ([dim if n == 1 else s for n, s in zip(shape[:3], t)] + [t[3]] for t in (strides, of_v))
    if k.dtype not in kinds or k.get_device() != dev or (strides[3] != 1 and dim > 1):
        _refuse(call, dev, k, "k_cache", kinds, shape)
    if v.dtype not in kinds or v.get_device() != dev or v.shape != shape or of_v != strides:
        _refuse(call, dev, v, "v_cache", kinds, shape)
    return k.data_ptr(), v.data_ptr(), shape[0], strides[0], strides[1], strides[2], shape[1], shape[2], dim, 0


def _serve(fn, name, dev, pack, fields, stream):
    try:
        args = pack(*fields)
    except struct.error as e:  # (a number that its field cannot hold)
        raise UwError(UW_ERR_ARG, f"{name}: {e}") from None
    if stream is None:
        stream = _raw_stream(dev) if dev >= 0 else 0
    else:
        stream = getattr(stream, "cuda_stream", stream)
    status = fn(args, stream)
    if status:
        raise UwError(status, name)


def uw_paged_plan(ctx_len, new_len, page_size: int, free_pages, table, cu_q, kv_len, positions,
                  slots, head_out, head_in=None, flags=None, stream=None) -> None:
    """Block tables and slot maps of one step from the requests' lengths (int32 tensors; slots
    int64): see include/unweight.h.  table [B, width] is updated in place."""
    f, dev, i32 = "uw_paged_plan", ctx_len.get_device(), (_TYPES or _types())["i32"]
    n, rows, spare, width = ctx_len.numel(), positions.numel(), free_pages.numel(), table.shape[-1]
    at, apart = _rows(f, dev, table, "table", i32, (n, width))
    ptr = _vectors(f, dev, (
        (ctx_len, "ctx_len", i32, n), (new_len, "new_len", i32, n), (free_pages, "free_pages", i32, spare),
        (head_in, "head_in", i32, 1), (head_out, "head_out", i32, 1), (cu_q, "cu_q", i32, n + 1),
        (kv_len, "kv_len", i32, n), (positions, "positions", i32, rows),
        (slots, "slots", _TYPES["i64"], rows), (flags, "flags", _TYPES["u32"], 1)))
    _serve(_plan_fn, f, dev, _PACK_PLAN, (*ptr[:5], at, *ptr[5:], apart, rows, n, width, spare, page_size), stream)


def uw_qk_norm_rope(q, k, v, positions, inv_freq, slots, k_cache, v_cache, q_out, q_weight=None,
                    k_weight=None, eps: float = 1e-6, interleaved: bool = False, flags=None,
                    stream=None) -> None:
    """Norms of q [T, H, D] and k [T, Hkv, D] per head (where there is a weight), rotation of the
    first 2 * len(inv_freq) values, queries to q_out, keys and v to the cache
    [pages, page_size, Hkv, D] at `slots`: see include/unweight.h."""
    f, dev, bf16 = "uw_qk_norm_rope", q.get_device(), (_TYPES or _types())["bf16"]
    shape = q.shape
    if len(shape) != 3:
        raise UwError(UW_ERR_SHAPE, f"{f}: q is {tuple(shape)}, not (rows, heads, dim)")
    rows, heads, dim = shape
    cache = _cache_fields(f, dev, k_cache, v_cache, dim)
    kv, half = (rows, cache[7], dim), inv_freq.numel()
    qp, qs = _rows(f, dev, q, "q", bf16, shape)
    kp, ks = _rows(f, dev, k, "k", bf16, kv)
    vp, vs = _rows(f, dev, v, "v", bf16, kv)
    op, os_ = _rows(f, dev, q_out, "q_out", bf16, shape)
    wq, wk, pos, inv, at, flag = _vectors(f, dev, (
        (q_weight, "q_weight", bf16, dim), (k_weight, "k_weight", bf16, dim),
        (positions, "positions", _TYPES["i32"], rows), (inv_freq, "inv_freq", _TYPES["f32"], half),
        (slots, "slots", _TYPES["i64"], rows), (flags, "flags", _TYPES["u32"], 1)))
    _serve(_rope_fn, f, dev, _PACK_ROPE, (qp, kp, vp, wq, wk, pos, inv, at, op, flag, *cache, rows, qs, ks, vs, os_,
                                          heads, 2 * half, 1 if interleaved else 0, eps), stream)


def uw_paged_attention_workspace_bytes(n_heads: int, n_kv_heads: int, head_dim: int) -> int:
    out = _sz()
    _check(lib.uw_paged_attention_workspace_bytes(int(n_heads), int(n_kv_heads), int(head_dim),
                                                  C.byref(out)),
           "uw_paged_attention_workspace_bytes")
    return int(out.value)


def uw_paged_attention(q, k_cache, v_cache, table, cu_q, kv_len, out, scale: float | None = None,
                       window: int = 0, lse=None, ws=None, flags=None, stream=None) -> None:
    """Attention of the requests' new tokens q [T, H, D] over their pages; out [T, H, D] BF16 or
    FP32, lse [T, H] FP32; scale None: 1 / sqrt(D): see include/unweight.h."""
    f, dev, bf16 = "uw_paged_attention", q.get_device(), (_TYPES or _types())["bf16"]
    shape = q.shape
    if len(shape) != 3:
        raise UwError(UW_ERR_SHAPE, f"{f}: q is {tuple(shape)}, not (rows, heads, dim)")
    rows, heads, dim = shape
    i32, n, width, ws_bytes = _TYPES["i32"], kv_len.numel(), table.shape[-1], 0 if ws is None else ws.numel()
    qp, qs = _rows(f, dev, q, "q", bf16, shape)
    op, os_ = _rows(f, dev, out, "out", _TYPES["real"], shape)
    tp, ts = _rows(f, dev, table, "table", i32, (n, width))
    cu, kv, lp, flag, wp = _vectors(f, dev, (
        (cu_q, "cu_q", i32, n + 1), (kv_len, "kv_len", i32, n), (lse, "lse", _TYPES["f32"], rows * heads),
        (flags, "flags", _TYPES["u32"], 1), (ws, "ws", _TYPES["u8"], ws_bytes)))
    _serve(_attention_fn, f, dev, _PACK_ATTENTION, (
        qp, tp, cu, kv, op, lp, flag, wp, *_cache_fields(f, dev, k_cache, v_cache, dim), ws_bytes, rows, qs, os_, ts,
        n, width, heads, window, 0 if out.dtype in bf16 else 1, dim ** -0.5 if scale is None else scale), stream)


def uw_sample(logits, u, ids, temperature=None, top_k=None, top_p=None, min_p=None, prob=None,
              stream=None) -> None:
    """One id per row of logits [M, vocab] (FP32 or BF16) from the uniform numbers u [M], after
    temperature, top-k, top-p and min-p ([M] each): see include/unweight.h."""
    f, dev, f32 = "uw_sample", logits.get_device(), (_TYPES or _types())["f32"]
    shape = logits.shape
    if len(shape) != 2:
        raise UwError(UW_ERR_SHAPE, f"{f}: logits is {tuple(shape)}, not (rows, vocab)")
    n, vocab = shape
    at, apart = _rows(f, dev, logits, "logits", _TYPES["real"], shape)
    ptr = _vectors(f, dev, (
        (u, "u", f32, n), (temperature, "temperature", f32, n), (top_k, "top_k", _TYPES["i32"], n),
        (top_p, "top_p", f32, n), (min_p, "min_p", f32, n), (ids, "ids", _TYPES["i64"], n), (prob, "prob", f32, n)))
    _serve(_sample_fn, f, dev, _PACK_SAMPLE, (at, *ptr, n, apart, vocab, 0 if logits.dtype in f32 else 1), stream)


# the same entry points, taking the packed bytes of their argument structure
_plan_fn, _rope_fn, _attention_fn, _sample_fn = (
    C.CFUNCTYPE(C.c_int, C.c_char_p, _vp)((n, lib))
    for n in ("uw_paged_plan", "uw_qk_norm_rope", "uw_paged_attention", "uw_sample"))


def uw_autotune(handles, Ms, profile_out_json: str | None = None) -> None:
    arr = (_vp * len(handles))(*[h.ptr for h in handles])
    ms = (_i64 * len(Ms))(*[int(m) for m in Ms])
    _check(lib.uw_autotune(arr, len(handles), ms, len(Ms),
                           profile_out_json.encode() if profile_out_json else None), "uw_autotune")


def uw_load_profile(handles, profile_json: str) -> None:
    arr = (_vp * len(handles))(*[h.ptr for h in handles])
    _check(lib.uw_load_profile(arr, len(handles), profile_json.encode()), "uw_load_profile")


def uw_get_choice(h: Handle, M: int) -> dict:
    c = uw_gemm_config()
    _check(lib.uw_get_choice(h.ptr, int(M), C.byref(c)), "uw_get_choice")
    return c.as_dict()


KERNEL_KINDS = ("decode_full", "decode_exp", "transcode", "gemm_bf16", "gemm_exp",
                "gemm_palette", "splitk_fixup", "gemv_bf16", "gemv_exp", "gemv_palette",
                "decode_dot")


def uw_trace_enable(h: Handle, enable: bool = True) -> None:
    _check(lib.uw_trace_enable(h.ptr, 1 if enable else 0), "uw_trace_enable")


def uw_trace_read(h: Handle, capacity: int = 16384):
    """[(kernel kind name, milliseconds)] of the launches traced since the last read."""
    kinds = (_i32 * capacity)()
    ms = (C.c_float * capacity)()
    n = _i32()
    _check(lib.uw_trace_read(h.ptr, kinds, ms, capacity, C.byref(n)), "uw_trace_read")
    return [(KERNEL_KINDS[kinds[i]], float(ms[i])) for i in range(min(n.value, capacity))]


def uw_last_device_status(h: Handle) -> int:
    """Synchronises the handle's stream; returns (does not raise) the device status."""
    return int(lib.uw_last_device_status(h.ptr))
