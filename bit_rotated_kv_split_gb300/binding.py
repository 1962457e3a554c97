"""ctypes binding of liboscar.so (include/oscar.h): argument marshalling only.

Every function keeps the C name and forwards torch tensors as raw device or
host pointers; all computation happens inside the library.  Importing this
module loads the library and raises if it is missing - there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
from ctypes import c_double, c_float, c_int32, c_int64, c_size_t, c_void_p

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
# the in-tree library; OSCAR_LIBRARY names another build of it (a
# verification build, for instance)
LIB_PATH = os.environ.get("OSCAR_LIBRARY") or os.path.join(_PKG, "liboscar.so")

OSCAR_OK = 0
STATUS_NAMES = {0: "OK", 1: "INVALID_ARG", 2: "ALIGNMENT", 3: "WORKSPACE", 4: "CUDA",
                5: "NO_CONVERGENCE", 6: "UNSUPPORTED", 7: "FILE"}
DEV_PAGE_BOUNDS, DEV_LENGTH, DEV_TIMEOUT = 0x1, 0x2, 0x4
OSCAR_STEP_OVERLAP_PREVIOUS = 0x1     # oscar_decode_step flag


class OscarError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        super().__init__("%s failed: %s (%d)" % (fn, STATUS_NAMES.get(status, "?"), status))


class LayerDesc(ctypes.Structure):
    """Mirror of `oscar_layer_desc`."""
    _fields_ = [
        ("batch", c_int32), ("n_q_heads", c_int32), ("n_kv_heads", c_int32), ("head_dim", c_int32),
        ("sink_cap", c_int32), ("recent_cap", c_int32), ("max_pages_per_seq", c_int32),
        ("max_hist", c_int32), ("n_pages", c_int64), ("tau_k", c_float), ("tau_v", c_float),
        ("pages", c_void_p), ("page_table", c_void_p), ("hist_len", c_void_p),
        ("sink_k", c_void_p), ("sink_v", c_void_p), ("sink_len", c_void_p),
        ("recent_k", c_void_p), ("recent_v", c_void_p), ("recent_len", c_void_p),
        ("recent_start", c_void_p), ("r_k", c_void_p), ("r_v", c_void_p), ("dev_status", c_void_p),
        ("quant_group_k", c_int32), ("quant_group_v", c_int32),
        ("codebook", c_int32), ("levels_k", c_float * 4), ("levels_v", c_float * 4),
    ]


class Int4Desc(ctypes.Structure):
    """Mirror of `oscar_int4_desc`."""
    keep = None   # a tensor whose memory it points to
    keep_others = ()   # the others
    _fields_ = [
        ("batch", c_int32), ("n_q_heads", c_int32), ("n_kv_heads", c_int32), ("head_dim", c_int32),
        ("max_pages_per_seq", c_int32), ("max_len", c_int32), ("n_pages", c_int64),
        ("tau_k", c_float), ("tau_v", c_float), ("pages", c_void_p), ("page_table", c_void_p),
        ("seq_len", c_void_p), ("dev_status", c_void_p), ("quant_group_k", c_int32), ("quant_group_v", c_int32),
    ]


class RopeDesc(ctypes.Structure):
    """Mirror of `oscar_rope_desc`."""
    keep = None   # a tensor whose memory it points to
    _fields_ = [("cos_sin", c_void_p), ("n_positions", c_int64), ("rot_dim", c_int32), ("interleaved", c_int32)]


class ScoreDesc(ctypes.Structure):
    """Mirror of `oscar_score_desc`."""
    keep = None   # a tensor whose memory it points to
    _fields_ = [("scale", c_float), ("softcap", c_float), ("window", c_int32), ("reserved", c_int32),
                ("slopes", c_void_p)]


class PromptDesc(ctypes.Structure):
    """Mirror of `oscar_prompt_desc`."""
    keep = None   # a tensor whose memory it points to
    _fields_ = [
        ("batch", c_int32), ("n_q_heads", c_int32), ("n_kv_heads", c_int32), ("head_dim", c_int32),
        ("max_q", c_int32), ("max_k", c_int32), ("causal", c_int32), ("reserved", c_int32),
        ("total_q", c_int64), ("total_k", c_int64), ("dev_status", c_void_p),
    ]


def _load():
    if not os.path.exists(LIB_PATH):
        raise RuntimeError("liboscar.so is not built (%s); run bit_rotated_kv_split_gb300.build" % LIB_PATH)
    lib = ctypes.CDLL(LIB_PATH)
    P = c_void_p
    sig = {
        "oscar_status_string": (ctypes.c_char_p, [c_int32]),
        "oscar_abi_version": (c_int32, []),
        "oscar_set_page_wait_limit": (c_int64, [c_int64]),
        "oscar_block_bytes": (c_int64, [c_int32, c_int32]),
        "oscar_build_rotation": (c_int32, [P, c_int64, c_int32, P, P]),
        "oscar_build_canalized_rotation": (c_int32, [c_int32, c_int32, P]),
        "oscar_build_rotation_from_covariance": (c_int32, [P, c_int32, P, P]),
        "oscar_covariance": (c_int32, [P, c_int64, c_int32, c_int64, P, P, ctypes.POINTER(c_size_t), P]),
        "oscar_value_covariance": (c_int32, [P, c_int64, P, P, c_int64, c_int32, c_int64, P, P,
                                             ctypes.POINTER(c_size_t), P]),
        "oscar_score_weighted_rows": (c_int32, [P, c_int64, P, P, c_int64, c_int32, c_double, P]),
        "oscar_clip_threshold": (c_int32, [P, c_int64, c_int32, c_int32, P, c_double, P]),
        "oscar_fit_codebook": (c_int32, [P, c_int64, c_int32, P, c_double, c_int32, P]),
        "oscar_rotation_file_write": (c_int32, [ctypes.c_char_p, c_int32, c_int32, c_int32, P, P, P, P]),
        "oscar_rotation_file_info": (c_int32, [ctypes.c_char_p, P, P, P]),
        "oscar_rotation_file_read": (c_int32, [ctypes.c_char_p, c_int32, c_int32, c_int32, P, P, P, P]),
        "oscar_quantize_append": (c_int32, [ctypes.POINTER(LayerDesc), P, P, c_int64, c_int64, P,
                                            P, P, c_int32, P, P, P]),
        "oscar_quantize_append_overlapped": (c_int32, [ctypes.POINTER(LayerDesc), P, P, c_int64, c_int64, P,
                                                       P, P, c_int32, P, P, P]),
        "oscar_decode_attention": (c_int32, [ctypes.POINTER(LayerDesc), P, P, P,
                                             ctypes.POINTER(c_size_t), P]),
        "oscar_decode_attention_static": (c_int32, [ctypes.POINTER(LayerDesc), P, P, P]),
        "oscar_decode_step": (c_int32, [ctypes.POINTER(LayerDesc), P, P, c_size_t, P, P, c_int64, c_int64, P, P,
                                        P, c_int32, P, P, P, P, P, c_size_t, P, ctypes.c_uint32, P]),
        "oscar_int4_block_bytes": (c_int64, [c_int32, c_int32, c_int32]),
        "oscar_rope_append_int4": (c_int32, [P, P, P, c_int64, P, c_int64, P, c_int64, P, P, P, c_int32, P, P, P]),
        "oscar_gather_int4": (c_int32, [P, P, P, c_int32, P, c_int64, P, c_int64, P]),
        "oscar_decode_attention_int4": (c_int32, [P, P, P, c_int64, P, P, P, P]),
        "oscar_prompt_attention": (c_int32, [P, P, P, c_int64, P, c_int64, P, c_int64, P, P, P, P, P, P, P, P]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


lib = _load()


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _check(fn, status):
    if status != OSCAR_OK:
        raise OscarError(fn, status)


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    return stream if isinstance(stream, int) else stream.cuda_stream


def oscar_status_string(status: int) -> str:
    return lib.oscar_status_string(status).decode()


def oscar_abi_version() -> int:
    return lib.oscar_abi_version()


def oscar_set_page_wait_limit(limit_ns: int) -> int:
    """Limit of the decode kernel's waits for page copies (<= 0: the default, 1 s); returns the previous one."""
    return int(lib.oscar_set_page_wait_limit(int(limit_ns)))


def oscar_block_bytes(quant_group_k: int = 128, quant_group_v: int = 128) -> int:
    """Bytes of one (page, KV head) block of the pool; 0 for an invalid group size."""
    return lib.oscar_block_bytes(int(quant_group_k), int(quant_group_v))


def _f64(a):
    return np.ascontiguousarray(a, dtype=np.float64)


def oscar_build_rotation(x: np.ndarray):
    """(R [d][d], eigenvalues [d]) from calibration rows x [n][d] (host float64)."""
    x = _f64(x)
    n, d = x.shape
    r = np.empty((d, d), dtype=np.float64)
    w = np.empty(d, dtype=np.float64)
    _check("oscar_build_rotation", lib.oscar_build_rotation(x.ctypes.data, n, d, r.ctypes.data, w.ctypes.data))
    return r, w


def oscar_build_canalized_rotation(d: int, block: int):
    """Block-diagonal OScaR rotation R [d][d] (host float64)."""
    r = np.empty((d, d), dtype=np.float64)
    _check("oscar_build_canalized_rotation", lib.oscar_build_canalized_rotation(d, block, r.ctypes.data))
    return r


def oscar_build_rotation_from_covariance(c: np.ndarray):
    """(R [d][d], eigenvalues [d]) from a covariance c [d][d] (host float64)."""
    c = _f64(c)
    d = c.shape[0]
    r = np.empty((d, d), dtype=np.float64)
    w = np.empty(d, dtype=np.float64)
    _check("oscar_build_rotation_from_covariance",
           lib.oscar_build_rotation_from_covariance(c.ctypes.data, d, r.ctypes.data, w.ctypes.data))
    return r, w


def oscar_covariance_workspace_bytes(n: int) -> int:
    size = c_size_t(0)
    _check("oscar_covariance", lib.oscar_covariance(None, int(n), 128, 128, None, None, ctypes.byref(size), None))
    return size.value


def oscar_covariance(x, c_out, workspace, stream=None) -> None:
    """c_out [128][128] fp32 (device) = x^T x / n over the bf16 rows x [n][ld] (device)."""
    n, ld = int(x.shape[0]), int(x.stride(0))
    size = c_size_t(workspace.numel() * workspace.element_size())
    _check("oscar_covariance", lib.oscar_covariance(_ptr(x), n, 128, ld, _ptr(c_out), _ptr(workspace),
                                                    ctypes.byref(size), _stream(stream)))


def oscar_value_covariance_workspace_bytes(n_q: int) -> int:
    size = c_size_t(0)
    _check("oscar_value_covariance", lib.oscar_value_covariance(None, int(n_q), None, None, 1, 128, 128, None, None,
                                                                ctypes.byref(size), None))
    return size.value


def oscar_value_covariance(q, k, v, c_out, workspace, stream=None) -> None:
    """c_out [128][128] fp32 (device) = (S V)^T (S V) / n_q, S = softmax(q k^T / sqrt(128)),
    over bf16 rows q [n_q][ld], k, v [n_k][ld] (device, one row stride)."""
    n_q, n_k, ld = int(q.shape[0]), int(k.shape[0]), int(q.stride(0))
    if int(k.stride(0)) != ld or int(v.stride(0)) != ld or int(v.shape[0]) != n_k:
        raise ValueError("q, k and v must share one row stride; k and v one row count")
    size = c_size_t(workspace.numel() * workspace.element_size())
    _check("oscar_value_covariance", lib.oscar_value_covariance(
        _ptr(q), n_q, _ptr(k), _ptr(v), n_k, 128, ld, _ptr(c_out), _ptr(workspace), ctypes.byref(size),
        _stream(stream)))


def oscar_score_weighted_rows(q: np.ndarray, k: np.ndarray, v: np.ndarray, scale: float = None):
    q, k, v = _f64(q), _f64(k), _f64(v)
    d = q.shape[1]
    out = np.empty((q.shape[0], d), dtype=np.float64)
    scale = 1.0 / np.sqrt(d) if scale is None else scale
    _check("oscar_score_weighted_rows", lib.oscar_score_weighted_rows(
        q.ctypes.data, q.shape[0], k.ctypes.data, v.ctypes.data, k.shape[0], d, scale, out.ctypes.data))
    return out


def oscar_clip_threshold(acts: np.ndarray, r: np.ndarray, quantile: float = 0.999) -> float:
    """acts [n_heads][rows][d], r [n_heads][d][d] (host float64)."""
    acts, r = _f64(acts), _f64(r)
    h, rows, d = acts.shape
    tau = c_double(0.0)
    _check("oscar_clip_threshold", lib.oscar_clip_threshold(
        acts.ctypes.data, rows, h, d, r.ctypes.data, quantile, ctypes.byref(tau)))
    return tau.value


def oscar_rotation_file_write(path: str, r_k: np.ndarray, r_v: np.ndarray, tau_k, tau_v) -> None:
    """r_k, r_v [n_layers][n_kv][d][d], tau_k, tau_v [n_layers] (stored as float32)."""
    r_k = np.ascontiguousarray(r_k, dtype=np.float32)
    r_v = np.ascontiguousarray(r_v, dtype=np.float32)
    tk = np.ascontiguousarray(np.atleast_1d(tau_k), dtype=np.float32)
    tv = np.ascontiguousarray(np.atleast_1d(tau_v), dtype=np.float32)
    n_layers, n_kv, d = r_k.shape[0], r_k.shape[1], r_k.shape[2]
    _check("oscar_rotation_file_write", lib.oscar_rotation_file_write(
        os.fsencode(path), n_layers, n_kv, d, r_k.ctypes.data, r_v.ctypes.data, tk.ctypes.data, tv.ctypes.data))


def oscar_rotation_file_read(path: str):
    """(r_k, r_v [n_layers][n_kv][d][d] float32, tau_k, tau_v [n_layers] float32)."""
    dims = [c_int32(0), c_int32(0), c_int32(0)]
    _check("oscar_rotation_file_info", lib.oscar_rotation_file_info(os.fsencode(path), *[ctypes.byref(x) for x in dims]))
    n_layers, n_kv, d = (x.value for x in dims)
    r_k = np.empty((n_layers, n_kv, d, d), np.float32)
    r_v = np.empty_like(r_k)
    tk = np.empty(n_layers, np.float32)
    tv = np.empty(n_layers, np.float32)
    _check("oscar_rotation_file_read", lib.oscar_rotation_file_read(
        os.fsencode(path), n_layers, n_kv, d, r_k.ctypes.data, r_v.ctypes.data, tk.ctypes.data, tv.ctypes.data))
    return r_k, r_v, tk, tv


def oscar_fit_codebook(x: np.ndarray, r: np.ndarray, tau: float, iters: int = 100) -> np.ndarray:
    """Four Lloyd-Max levels (float32 holding fp16 values) from calibration rows
    x [n][d] rotated by r [d][d] and clipped at tau (host float64)."""
    x, r = _f64(x), _f64(r)
    out = np.empty(4, dtype=np.float32)
    _check("oscar_fit_codebook", lib.oscar_fit_codebook(x.ctypes.data, x.shape[0], x.shape[1], r.ctypes.data,
                                                        float(tau), int(iters), out.ctypes.data))
    return out


def oscar_quantize_append(desc: LayerDesc, k_src, v_src, src_rows: int, row_stride: int, src_index,
                          dst_req, dst_pos, n: int, new_k=None, new_v=None, stream=None) -> None:
    _check("oscar_quantize_append", lib.oscar_quantize_append(
        ctypes.byref(desc), _ptr(k_src), _ptr(v_src), int(src_rows), int(row_stride), _ptr(src_index),
        _ptr(dst_req), _ptr(dst_pos), int(n), _ptr(new_k), _ptr(new_v), _stream(stream)))


def oscar_quantize_append_overlapped(desc: LayerDesc, k_src, v_src, src_rows: int, row_stride: int, src_index,
                                     dst_req, dst_pos, n: int, new_k=None, new_v=None, stream=None) -> None:
    _check("oscar_quantize_append_overlapped", lib.oscar_quantize_append_overlapped(
        ctypes.byref(desc), _ptr(k_src), _ptr(v_src), int(src_rows), int(row_stride), _ptr(src_index),
        _ptr(dst_req), _ptr(dst_pos), int(n), _ptr(new_k), _ptr(new_v), _stream(stream)))


def oscar_decode_workspace_bytes(desc: LayerDesc) -> int:
    size = c_size_t(0)
    _check("oscar_decode_attention", lib.oscar_decode_attention(
        ctypes.byref(desc), None, None, None, ctypes.byref(size), None))
    return size.value


def oscar_decode_attention(desc: LayerDesc, q, out, workspace, workspace_bytes: int = None,
                           stream=None) -> None:
    size = c_size_t(workspace.numel() * workspace.element_size() if workspace_bytes is None
                    else workspace_bytes)
    _check("oscar_decode_attention", lib.oscar_decode_attention(
        ctypes.byref(desc), _ptr(q), _ptr(out), _ptr(workspace), ctypes.byref(size), _stream(stream)))


def oscar_decode_step(desc: LayerDesc, host_in, dev_in, in_bytes: int, k_src, v_src, src_rows: int,
                      row_stride: int, src_index, dst_req, dst_pos, n: int, new_k, new_v, q, out, workspace,
                      workspace_bytes: int, host_out=None, stream=None, flags: int = 0) -> None:
    """One decode step: H2D copy of the staged inputs, demotion, decode, D2H copy of the output.
    flags: 0 or OSCAR_STEP_OVERLAP_PREVIOUS (the demotion overlaps the kernel before it)."""
    _check("oscar_decode_step", lib.oscar_decode_step(
        ctypes.byref(desc), _ptr(host_in), _ptr(dev_in), int(in_bytes), _ptr(k_src), _ptr(v_src), int(src_rows),
        int(row_stride), _ptr(src_index), _ptr(dst_req), _ptr(dst_pos), int(n), _ptr(new_k), _ptr(new_v),
        _ptr(q), _ptr(out), _ptr(workspace), int(workspace_bytes), _ptr(host_out), int(flags), _stream(stream)))


def oscar_decode_attention_static(desc: LayerDesc, q, out, stream=None) -> None:
    """Decode attention with the library's fixed workspace (no allocation by anyone)."""
    _check("oscar_decode_attention_static", lib.oscar_decode_attention_static(
        ctypes.byref(desc), _ptr(q), _ptr(out), _stream(stream)))


# ---------------------------------------------------------------- 4-bit layers

def oscar_int4_block_bytes(head_dim: int, quant_group_k: int = 0, quant_group_v: int = 0) -> int:
    """Bytes of one (page, KV head) block of a 4-bit layer; 0 for an invalid head size or group."""
    return lib.oscar_int4_block_bytes(int(head_dim), int(quant_group_k), int(quant_group_v))


def _int32(name, n) -> int:
    n = int(n)
    if not -2 ** 31 <= n < 2 ** 31:
        raise ValueError("%s: %d is no 32-bit integer" % (name, n))
    return n


def rope_desc(cos_sin, rot_dim: int, interleaved: bool = False) -> RopeDesc:
    """Position rotation by cos_sin [n_positions][rot_dim] fp32 (device): rot_dim / 2 cosines, then the sines.

    The descriptor keeps the tensor alive.
    """
    d = RopeDesc()
    if rot_dim:
        if cos_sin.dim() != 2 or cos_sin.shape[1] != rot_dim or str(cos_sin.dtype) != "torch.float32" \
                or not cos_sin.is_contiguous():
            raise ValueError("cos_sin must be contiguous float32 [n_positions][rot_dim]")
        d.cos_sin, d.n_positions = cos_sin.data_ptr(), cos_sin.shape[0]
        d.keep = cos_sin
    d.rot_dim, d.interleaved = _int32("rot_dim", rot_dim), int(bool(interleaved))
    return d


def score_desc(scale: float = 0.0, softcap: float = 0.0, window: int = 0, slopes=None) -> ScoreDesc:
    """Form of the scores: scale (0 = 1 / sqrt(head_dim)), tanh cap, window, slopes [H_q] fp32 (device).

    The descriptor keeps the slopes alive.
    """
    d = ScoreDesc()
    d.scale, d.softcap, d.window = float(scale), float(softcap), _int32("window", window)
    if slopes is not None:
        if str(slopes.dtype) != "torch.float32" or slopes.dim() != 1 or not slopes.is_contiguous():
            raise ValueError("slopes must be contiguous float32 [n_q_heads]")
        d.slopes = slopes.data_ptr()
        d.n_slopes, d.keep = slopes.shape[0], slopes
    return d


def prompt_desc(batch: int, n_q_heads: int, n_kv_heads: int, head_dim: int, max_q: int, max_k: int, total_q: int,
                total_k: int, causal: bool = True, dev_status=None) -> PromptDesc:
    """A batch of packed prompts: bounds on one request's queries and keys, rows in all."""
    d = PromptDesc()
    for name, n in (("batch", batch), ("n_q_heads", n_q_heads), ("n_kv_heads", n_kv_heads), ("head_dim", head_dim),
                    ("max_q", max_q), ("max_k", max_k)):
        setattr(d, name, _int32(name, n))
    d.total_q, d.total_k = int(total_q), int(total_k)
    d.causal = int(bool(causal))
    if dev_status is not None:
        if dev_status.numel() < 1 or dev_status.element_size() != 4:
            raise ValueError("dev_status must be an int32 word")
        d.dev_status = dev_status.data_ptr()
        d.keep = dev_status
    return d


_torch = None


def _half(t):
    """bfloat16 or raw 16-bit integers: fp16 rows have the size of bf16's and would be read as such."""
    global _torch
    if _torch is None:
        import torch
        _torch = torch
    return t.dtype is _torch.bfloat16 or (t.element_size() == 2 and not t.is_floating_point())


def _heads(name, t, heads, d):
    """Row stride of bf16 rows t [n][heads][d] (bfloat16, or its bits as uint16) whose heads lie side by side."""
    shape = t.shape
    if len(shape) != 3 or shape[1] != heads or shape[2] != d or not _half(t):
        raise ValueError("%s must be bfloat16 [n][%d][%d]" % (name, heads, d))
    if shape[0] == 0:
        return heads * d
    row, head, one = t.stride()
    if one != 1 or (heads > 1 and head != d):
        raise ValueError("%s: the heads of a row must lie side by side" % name)
    return heads * d if shape[0] == 1 else row


def _index(name, t, n):
    if t is not None and (t.dim() != 1 or t.numel() < n or t.element_size() != 4 or t.is_floating_point()
                          or not t.is_contiguous()):
        raise ValueError("%s must be contiguous int32 with at least %d entries" % (name, n))


def _contiguous(name, t, shape, itemsize):
    if t is not None and (t.shape != shape or not t.is_contiguous() or not (
            _half(t) if itemsize == 2 else t.element_size() == 4 and t.is_floating_point())):
        raise ValueError("%s must be contiguous %s %s" % (name, "bfloat16" if itemsize == 2 else "float32", list(shape)))


def _workspace_size(t):
    if not t.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return c_size_t(t.numel() * t.element_size())


_raw_stream = None


def _on_device(name, stream, tensors, fn, args):
    """Calls the library with the tensors' device current and, without a stream, on that device's current stream."""
    global _torch, _raw_stream
    if _raw_stream is None:
        import torch
        _torch = torch
        # the current stream's handle without a Stream object around it (3 us a call less)
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda index: torch.cuda.current_stream(index).cuda_stream)
    cuda = _torch.cuda
    index = tensors[0].get_device()
    for t in tensors:
        if t is not None and (t.get_device() != index or index < 0):
            raise ValueError("%s: every tensor must be on one CUDA device" % name)
    handle = _raw_stream(index) if stream is None else _stream(stream)
    if index != cuda.current_device():
        with cuda.device(index):
            status = fn(*args, handle)
    else:
        status = fn(*args, handle)
    if status != OSCAR_OK:
        raise OscarError(name, status)


def _ref(d):
    return None if d is None else ctypes.byref(d)


def _slopes_ok(score, heads):
    if score is not None and score.slopes and getattr(score, "n_slopes", heads) != heads:
        raise ValueError("score: %d slopes for %d query heads" % (score.n_slopes, heads))


def oscar_rope_append_int4(desc: Int4Desc, rope, q, k, v, dst_req, dst_pos, q_out, k_out=None, rope_pos=None,
                           stream=None) -> None:
    """Rotates q [n][H_q][d] and k [n][H_kv][d] (bf16) by position into q_out, k_out and appends k, v to the pages.

    q and q_out may both be None; k_out may be None.  Rows may be strided (slices of one projection's output).
    """
    hq, hk, d, n = desc.n_q_heads, desc.n_kv_heads, desc.head_dim, int(k.shape[0])
    qs = _heads("q", q, hq, d) if q is not None else 0
    ks, vs = _heads("k", k, hk, d), _heads("v", v, hk, d)
    if v.shape[0] != n or (q is not None and q.shape[0] != n):
        raise ValueError("q, k and v must have one row count")
    _index("dst_req", dst_req, n), _index("dst_pos", dst_pos, n), _index("rope_pos", rope_pos, n)
    _contiguous("q_out", q_out, (n, hq, d), 2)
    _contiguous("k_out", k_out, (n, hk, d), 2)
    _on_device("oscar_rope_append_int4", stream, (k, v, dst_req, dst_pos, q, q_out, k_out, rope_pos, desc.keep, rope and rope.keep,
                                                  *desc.keep_others),
               lib.oscar_rope_append_int4, (
                   ctypes.byref(desc), _ref(rope), _ptr(q), qs, k.data_ptr(), ks, v.data_ptr(), vs, dst_req.data_ptr(),
                   dst_pos.data_ptr(), _ptr(rope_pos), n, _ptr(q_out), _ptr(k_out)))


def oscar_gather_int4(desc: Int4Desc, src_req, src_pos, k_out, v_out, stream=None) -> None:
    """Cached rows (src_req[i], src_pos[i]) as bf16 into k_out, v_out [n][H_kv][d] (rows may be strided)."""
    hk, d, n = desc.n_kv_heads, desc.head_dim, int(k_out.shape[0])
    ks, vs = _heads("k_out", k_out, hk, d), _heads("v_out", v_out, hk, d)
    if v_out.shape[0] != n:
        raise ValueError("k_out and v_out must have one row count")
    _index("src_req", src_req, n), _index("src_pos", src_pos, n)
    _on_device("oscar_gather_int4", stream, (k_out, v_out, src_req, src_pos, desc.keep, *desc.keep_others), lib.oscar_gather_int4, (
        ctypes.byref(desc), src_req.data_ptr(), src_pos.data_ptr(), n, k_out.data_ptr(), ks, v_out.data_ptr(), vs))


def oscar_decode_int4_workspace_bytes(desc: Int4Desc) -> int:
    size = c_size_t(0)
    _check("oscar_decode_attention_int4", lib.oscar_decode_attention_int4(
        ctypes.byref(desc), None, None, 0, None, None, ctypes.byref(size), None))
    return size.value


def oscar_decode_attention_int4(desc: Int4Desc, q, out, workspace, score=None, stream=None) -> None:
    """out [B][H_q][d] bf16 = attention of one query per request q [B][H_q][d] over the 4-bit cache."""
    hq, d, b = desc.n_q_heads, desc.head_dim, desc.batch
    qs = _heads("q", q, hq, d)
    if q.shape[0] != b:
        raise ValueError("q must have one row per request")
    _contiguous("out", out, (b, hq, d), 2)
    _slopes_ok(score, hq)
    size = _workspace_size(workspace)
    _on_device("oscar_decode_attention_int4", stream, (q, out, workspace, desc.keep, score and score.keep, *desc.keep_others),
               lib.oscar_decode_attention_int4, (
                   ctypes.byref(desc), _ref(score), q.data_ptr(), qs, out.data_ptr(), workspace.data_ptr(),
                   ctypes.byref(size)))


def oscar_prompt_workspace_bytes(desc: PromptDesc) -> int:
    size = c_size_t(0)
    _check("oscar_prompt_attention", lib.oscar_prompt_attention(
        ctypes.byref(desc), None, None, 0, None, 0, None, 0, None, None, None, None, None, None,
        ctypes.byref(size), None))
    return size.value


def oscar_prompt_attention(desc: PromptDesc, q, k, v, cu_q, cu_k, out, workspace, score=None, prefix_len=None,
                           lse=None, stream=None) -> None:
    """out [total_q][H_q][d] bf16 (and lse [total_q][H_q] fp32) of packed prompts; rows cu_q / cu_k [B + 1] int32."""
    hq, hk, d = desc.n_q_heads, desc.n_kv_heads, desc.head_dim
    qs, ks, vs = _heads("q", q, hq, d), _heads("k", k, hk, d), _heads("v", v, hk, d)
    if q.shape[0] != desc.total_q or k.shape[0] != desc.total_k or v.shape[0] != desc.total_k:
        raise ValueError("q must have total_q rows, k and v total_k")
    _index("cu_q", cu_q, desc.batch + 1), _index("cu_k", cu_k, desc.batch + 1)
    _index("prefix_len", prefix_len, desc.batch)
    _contiguous("out", out, (desc.total_q, hq, d), 2)
    _contiguous("lse", lse, (desc.total_q, hq), 4)
    _slopes_ok(score, hq)
    size = _workspace_size(workspace)
    _on_device("oscar_prompt_attention", stream, (
        q, k, v, cu_q, cu_k, out, workspace, prefix_len, lse, desc.keep, score and score.keep),
               lib.oscar_prompt_attention, (
                   ctypes.byref(desc), _ref(score), q.data_ptr(), qs, _ptr(k), ks, _ptr(v), vs, cu_q.data_ptr(),
                   cu_k.data_ptr(), _ptr(prefix_len), out.data_ptr(), _ptr(lse), workspace.data_ptr(),
                   ctypes.byref(size)))
