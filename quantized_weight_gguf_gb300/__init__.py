"""Python binding of libqmm (include/qmm.h): fused dequantize-and-multiply
``y = x @ W`` over GGUF/ggml-packed weights on one GB300 GPU.

Argument marshalling only: every step of the product runs in the CUDA
kernels of ``libqmm.so``. PyTorch supplies device memory and streams. The
functions carry the C names (``qmm_matmul``, ``qmm_matmul_ex``,
``qmm_dequant`` ...) and take plain integers / device pointers or torch
tensors; ``matmul``, ``dequant``, ``matmul_backward_input``,
``matmul_experts``, ``matmul_affine``, ``dequant_affine`` and ``matmul_glu``
are tensor-level conveniences over them, and so are ``KvCache``,
``kv_append``, ``kv_read`` and ``attend`` over the paged key-value cache.
If ``libqmm.so`` has not been built, every call raises: there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
import threading

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libqmm.so")

FORMATS = {"bf16": 0, "f16": 1, "q4_0": 2, "q4_k": 3, "q6_k": 4, "q8_0": 5, "q5_0": 6,
           "affine4": 7, "affine8": 8}
PATH_AUTO, PATH_GEMV, PATH_MMA = 0, 1, 2
FLAG_OVERLAP_PREV = 1
FLAG_X_READY = 2
FLAG_SPLIT_W = 4
STATUS = {0: "QMM_OK", 1: "QMM_ERR_FORMAT", 2: "QMM_ERR_SHAPE", 3: "QMM_ERR_SIZE",
          4: "QMM_ERR_RANGE", 5: "QMM_ERR_NULL", 6: "QMM_ERR_ALIGN", 7: "QMM_ERR_CUDA",
          8: "QMM_ERR_DEVICE_TIMEOUT", 9: "QMM_ERR_WORKSPACE", 10: "QMM_ERR_UNSUPPORTED",
          11: "QMM_ERR_BAD_ID", 12: "QMM_ERR_BAD_PAGE"}
EXPORTS = ("qmm_weight_bytes", "qmm_matmul", "qmm_set_stream", "qmm_matmul_ex",
           "qmm_workspace_bytes", "qmm_select_path", "qmm_matmul_host", "qmm_dequant",
           "qmm_device_status", "qmm_last_error", "qmm_version", "qmm_matmul_noalloc",
           "qmm_matmul_backward_input", "qmm_backward_input_workspace_bytes",
           "qmm_matmul_experts", "qmm_matmul_affine", "qmm_dequant_affine", "qmm_matmul_glu",
           "qmm_glu_workspace_bytes", "qmm_check_bounded_wait", "qmm_matmul_experts_affine",
           "qmm_experts_workspace_bytes", "qmm_kv_page_bytes", "qmm_kv_append", "qmm_kv_read",
           "qmm_attend", "qmm_attend_workspace_bytes")


class QmmError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS.get(status, status)}: {message}")
        self.status = status


class qmm_args(ctypes.Structure):
    _fields_ = [("fmt", ctypes.c_int), ("w", ctypes.c_void_p), ("w_len", ctypes.c_size_t),
                ("x", ctypes.c_void_p), ("y", ctypes.c_void_p), ("k", ctypes.c_int64),
                ("n", ctypes.c_int64), ("n_tokens", ctypes.c_int64), ("j_start", ctypes.c_int64),
                ("j_end", ctypes.c_int64), ("accumulate", ctypes.c_int), ("path", ctypes.c_int),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
                ("stream", ctypes.c_void_p), ("flags", ctypes.c_int)]


class qmm_kv_cache(ctypes.Structure):
    _fields_ = [("fmt_k", ctypes.c_int), ("fmt_v", ctypes.c_int), ("pages", ctypes.c_void_p),
                ("pages_len", ctypes.c_size_t), ("n_pages", ctypes.c_int64),
                ("page_size", ctypes.c_int64), ("n_kv_heads", ctypes.c_int64),
                ("head_dim", ctypes.c_int64), ("page_table", ctypes.c_void_p),
                ("table_stride", ctypes.c_int64), ("max_pages", ctypes.c_int64),
                ("lens", ctypes.c_void_p), ("n_seqs", ctypes.c_int64)]


class qmm_kv_append_args(ctypes.Structure):
    _fields_ = [("cache", qmm_kv_cache), ("n_new", ctypes.c_int64), ("k", ctypes.c_void_p),
                ("v", ctypes.c_void_p), ("k_stride", ctypes.c_int64), ("v_stride", ctypes.c_int64),
                ("q", ctypes.c_void_p), ("q_out", ctypes.c_void_p), ("q_stride", ctypes.c_int64),
                ("q_out_stride", ctypes.c_int64), ("n_heads", ctypes.c_int64),
                ("rope", ctypes.c_void_p), ("rope_len", ctypes.c_int64), ("n_rot", ctypes.c_int64),
                ("rope_style", ctypes.c_int), ("stream", ctypes.c_void_p), ("flags", ctypes.c_int)]


class qmm_kv_read_args(ctypes.Structure):
    _fields_ = [("cache", qmm_kv_cache), ("first", ctypes.c_int64), ("count", ctypes.c_int64),
                ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("stream", ctypes.c_void_p),
                ("flags", ctypes.c_int)]


class qmm_attend_args(ctypes.Structure):
    _fields_ = [("cache", qmm_kv_cache), ("n_new", ctypes.c_int64), ("n_heads", ctypes.c_int64),
                ("q", ctypes.c_void_p), ("out", ctypes.c_void_p), ("q_stride", ctypes.c_int64),
                ("out_stride", ctypes.c_int64), ("scale", ctypes.c_float),
                ("window", ctypes.c_int64), ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_size_t), ("stream", ctypes.c_void_p),
                ("flags", ctypes.c_int)]


_lib = None


def load(path: str = LIB_PATH):
    """Load libqmm.so (raises if it is missing) and declare its signatures."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"libqmm.so is not built ({path}); run __graft_entry__.build() "
                           "or python -m quantized_weight_gguf_gb300.build_lib")
    lib = ctypes.CDLL(path)
    i64, vp, sz, i = ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
    pa = ctypes.POINTER(qmm_args)
    sig = {
        "qmm_weight_bytes": (sz, [i, i64, i64]),
        "qmm_matmul": (i, [i, vp, vp, i64, i64, i64, vp]),
        "qmm_set_stream": (None, [vp]),
        "qmm_matmul_ex": (i, [pa]),
        "qmm_workspace_bytes": (sz, [pa]),
        "qmm_select_path": (i, [pa]),
        "qmm_matmul_host": (i, [pa, vp, vp, vp]),
        "qmm_dequant": (i, [i, vp, i64, i64, vp, vp]),
        "qmm_device_status": (i, [vp]),
        "qmm_last_error": (ctypes.c_char_p, []),
        "qmm_version": (i, []),
        "qmm_matmul_noalloc": (i, [pa]),
        "qmm_matmul_backward_input": (i, [pa]),
        "qmm_backward_input_workspace_bytes": (sz, [pa]),
        "qmm_matmul_experts": (i, [pa, vp, i64, i64]),
        "qmm_experts_workspace_bytes": (sz, [pa, i64, i64]),
        "qmm_matmul_affine": (i, [pa, vp, vp]),
        "qmm_matmul_glu": (i, [pa, vp, i]),
        "qmm_glu_workspace_bytes": (sz, [pa]),
        "qmm_check_bounded_wait": (i, [vp]),
        "qmm_matmul_experts_affine": (i, [pa, vp, i64, i64, vp, vp]),
        "qmm_dequant_affine": (i, [i, vp, vp, vp, i64, i64, vp, vp]),
        "qmm_kv_page_bytes": (sz, [i, i, i64, i64, i64]),
        "qmm_kv_append": (i, [ctypes.POINTER(qmm_kv_append_args)]),
        "qmm_kv_read": (i, [ctypes.POINTER(qmm_kv_read_args)]),
        "qmm_attend": (i, [ctypes.POINTER(qmm_attend_args)]),
        "qmm_attend_workspace_bytes": (sz, [ctypes.POINTER(qmm_attend_args)]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def _ptr(v):
    if v is None:
        return None
    if isinstance(v, int):
        return v
    if hasattr(v, "data_ptr"):
        return v.data_ptr()
    if hasattr(v, "ctypes"):
        return v.ctypes.data
    raise TypeError(f"cannot take a pointer of {type(v)}")


def _fmt(f):
    return FORMATS[f] if isinstance(f, str) else int(f)


def _check(status: int):
    if status != 0:
        raise QmmError(status, load().qmm_last_error().decode())
    return status


def _keep_until_done(buf, stream):
    """A per-call scratch tensor allocated on torch's current stream but used
    by kernels on another stream: tell the caching allocator, so the memory
    is not handed out again before that stream's work is done."""
    if buf is None or stream is None or stream == 0:
        return
    import torch
    s = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(
        int(getattr(stream, "cuda_stream", stream)), device=buf.device)
    if s.cuda_stream != torch.cuda.current_stream(buf.device).cuda_stream:
        buf.record_stream(s)


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    return int(getattr(stream, "cuda_stream", stream))


# --------------------------------------------------------- C-named calls ----

def qmm_weight_bytes(fmt, k: int, n: int) -> int:
    return load().qmm_weight_bytes(_fmt(fmt), k, n)


def qmm_set_stream(stream) -> None:
    load().qmm_set_stream(_stream(stream))


def qmm_matmul(fmt, w, x, k: int, n: int, n_tokens: int, y) -> int:
    return _check(load().qmm_matmul(_fmt(fmt), _ptr(w), _ptr(x), k, n, n_tokens, _ptr(y)))


def make_args(fmt, w, x, y, k, n, n_tokens, *, w_len=0, j_start=0, j_end=0, accumulate=False,
              path=PATH_AUTO, workspace=None, workspace_bytes=0, stream=None, flags=0) -> qmm_args:
    return qmm_args(_fmt(fmt), _ptr(w), w_len, _ptr(x), _ptr(y), k, n, n_tokens, j_start, j_end,
                    int(bool(accumulate)), int(path), _ptr(workspace), workspace_bytes,
                    _stream(stream) if stream != 0 else 0, int(flags))


def qmm_matmul_ex(args: qmm_args) -> int:
    return _check(load().qmm_matmul_ex(ctypes.byref(args)))


def qmm_matmul_noalloc(args: qmm_args) -> int:
    return _check(load().qmm_matmul_noalloc(ctypes.byref(args)))


def qmm_matmul_backward_input(args: qmm_args) -> int:
    return _check(load().qmm_matmul_backward_input(ctypes.byref(args)))


ACT_SWIGLU, ACT_GEGLU = 1, 2
ACTS = {"swiglu": ACT_SWIGLU, "geglu": ACT_GEGLU}


def qmm_matmul_glu(args: qmm_args, w_up, act) -> int:
    act = ACTS[act] if isinstance(act, str) else int(act)
    return _check(load().qmm_matmul_glu(ctypes.byref(args), _ptr(w_up), act))


def qmm_glu_workspace_bytes(args: qmm_args) -> int:
    return load().qmm_glu_workspace_bytes(ctypes.byref(args))


def qmm_matmul_affine(args: qmm_args, scales, biases) -> int:
    return _check(load().qmm_matmul_affine(ctypes.byref(args), _ptr(scales), _ptr(biases)))


def qmm_dequant_affine(fmt, w, scales, biases, k: int, n: int, out, stream=None) -> int:
    return _check(load().qmm_dequant_affine(_fmt(fmt), _ptr(w), _ptr(scales), _ptr(biases), k, n,
                                            _ptr(out), _stream(stream)))


def qmm_matmul_experts_affine(args: qmm_args, ids, n_experts: int, top_k: int, scales,
                              biases) -> int:
    return _check(load().qmm_matmul_experts_affine(ctypes.byref(args), _ptr(ids), n_experts, top_k,
                                                   _ptr(scales), _ptr(biases)))


def qmm_matmul_experts(args: qmm_args, ids, n_experts: int, top_k: int) -> int:
    return _check(load().qmm_matmul_experts(ctypes.byref(args), _ptr(ids), n_experts, top_k))


def qmm_experts_workspace_bytes(args: qmm_args, n_experts: int, top_k: int) -> int:
    return load().qmm_experts_workspace_bytes(ctypes.byref(args), n_experts, top_k)


def qmm_backward_input_workspace_bytes(args: qmm_args) -> int:
    return load().qmm_backward_input_workspace_bytes(ctypes.byref(args))


def qmm_workspace_bytes(args: qmm_args) -> int:
    return load().qmm_workspace_bytes(ctypes.byref(args))


def qmm_select_path(args: qmm_args) -> int:
    return load().qmm_select_path(ctypes.byref(args))


def qmm_matmul_host(args: qmm_args, dev_w, dev_x, dev_y) -> int:
    return _check(load().qmm_matmul_host(ctypes.byref(args), _ptr(dev_w), _ptr(dev_x), _ptr(dev_y)))


def qmm_dequant(fmt, w, k: int, n: int, out, stream=None) -> int:
    return _check(load().qmm_dequant(_fmt(fmt), _ptr(w), k, n, _ptr(out), _stream(stream)))


def qmm_check_bounded_wait(stream=None) -> int:
    return _check(load().qmm_check_bounded_wait(_stream(stream)))


def qmm_device_status(stream=None) -> int:
    return _check(load().qmm_device_status(_stream(stream)))


def qmm_last_error() -> str:
    return load().qmm_last_error().decode()


def qmm_version() -> int:
    return load().qmm_version()


# ------------------------------------------------------ tensor helpers ----

def matmul(fmt, w, x, k: int, n: int, *, y=None, j_start=0, j_end=0, accumulate=False,
           path=PATH_AUTO, stream=None, flags=0):
    """y = x @ W for torch CUDA tensors: w uint8 packed bytes, x float32 [N, k].
    Returns y float32 [N, n] (the given y when passed). Scratch for the
    tensor-core path is a torch allocation on x's device."""
    import torch
    if x.dim() == 1:
        x = x.unsqueeze(0)
    nt = x.shape[0]
    if y is None:
        y = torch.empty((nt, n), dtype=torch.float32, device=x.device)
    a = make_args(fmt, w, x, y, k, n, nt, w_len=w.numel() * w.element_size(), j_start=j_start,
                  j_end=j_end, accumulate=accumulate, path=path, stream=stream, flags=flags)
    need = qmm_workspace_bytes(a)
    ws = None
    if need:
        ws = torch.empty(need, dtype=torch.uint8, device=x.device)
        a.workspace = ws.data_ptr()
        a.workspace_bytes = need
    qmm_matmul_ex(a)
    _keep_until_done(ws, stream)
    return y


def matmul_backward_input(fmt, w, dy, k: int, n: int, *, dx=None, j_start=0, j_end=0,
                          accumulate=False, stream=None, flags=0):
    """dx = W^T dy over the rows [j_start, j_end) for torch CUDA tensors: w
    uint8 packed bytes, dy float32 [n]. Returns dx float32 [k] (the given dx
    when passed). Scratch is the library's own buffer."""
    import torch
    if dx is None:
        dx = torch.empty(k, dtype=torch.float32, device=dy.device)
    a = make_args(fmt, w, dy, dx, k, n, 1, w_len=w.numel() * w.element_size(), j_start=j_start,
                  j_end=j_end, accumulate=accumulate, stream=stream, flags=flags)
    qmm_matmul_backward_input(a)
    return dx


def matmul_experts(fmt, w, x, ids, k: int, n: int, n_experts: int, *, y=None, j_start=0,
                   j_end=0, accumulate=False, path=PATH_AUTO, stream=None, flags=0, scales=None,
                   biases=None):
    """Expert-indexed product for torch CUDA tensors: w uint8 (n_experts
    stacked slices of n rows), x float32 [n_pos, k], ids int32 [n_pos, top_k]
    on the device. Returns y float32 [n_pos * top_k, n] (the given y when
    passed). Scratch of the grouped form is a torch allocation on x's device."""
    import torch
    if x.dim() == 1:
        x = x.unsqueeze(0)
    if ids.dim() == 1:
        ids = ids.unsqueeze(0)
    n_pos, top_k = ids.shape
    if y is None:
        y = torch.empty((n_pos * top_k, n), dtype=torch.float32, device=x.device)
    a = make_args(fmt, w, x, y, k, n, n_pos, w_len=w.numel() * w.element_size(), j_start=j_start,
                  j_end=j_end, accumulate=accumulate, path=path, stream=stream, flags=flags)
    if scales is not None or biases is not None:
        qmm_matmul_experts_affine(a, ids, n_experts, top_k, scales, biases)
        return y
    need = qmm_experts_workspace_bytes(a, n_experts, top_k)
    ws = None
    if need:
        ws = torch.empty(need, dtype=torch.uint8, device=x.device)
        a.workspace, a.workspace_bytes = ws.data_ptr(), need
    qmm_matmul_experts(a, ids, n_experts, top_k)
    _keep_until_done(ws, stream)
    return y


def dequant(fmt, w, k: int, n: int, stream=None):
    """fp32 [n, k] weights from packed bytes (torch CUDA uint8 tensor)."""
    import torch
    out = torch.empty((n, k), dtype=torch.float32, device=w.device)
    qmm_dequant(fmt, w, k, n, out, stream)
    return out


def matmul_affine(fmt, w, scales, biases, x, k: int, n: int, *, y=None, j_start=0, j_end=0,
                  accumulate=False, path=PATH_AUTO, workspace=None, workspace_bytes=0,
                  stream=None, flags=0):
    """y = x @ W for an affine matrix ("affine4" / "affine8") on torch CUDA
    tensors: w uint8 code words, scales / biases bf16 or int16 [n, k/64],
    x float32 [N, k]. Returns y float32 [N, n] (the given y when passed)."""
    import torch
    if x.dim() == 1:
        x = x.unsqueeze(0)
    nt = x.shape[0]
    if y is None:
        y = torch.empty((nt, n), dtype=torch.float32, device=x.device)
    a = make_args(fmt, w, x, y, k, n, nt, w_len=w.numel() * w.element_size(), j_start=j_start,
                  j_end=j_end, accumulate=accumulate, path=path, stream=stream, flags=flags)
    own = None
    if workspace is None:
        need = qmm_workspace_bytes(a)
        if need:
            own = workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
            workspace_bytes = need
    if workspace is not None:
        a.workspace, a.workspace_bytes = _ptr(workspace), workspace_bytes
    qmm_matmul_affine(a, scales, biases)
    _keep_until_done(own, stream)
    return y


def dequant_affine(fmt, w, scales, biases, k: int, n: int, stream=None):
    """fp32 [n, k] weights of an affine matrix (torch CUDA tensors)."""
    import torch
    out = torch.empty((n, k), dtype=torch.float32, device=w.device)
    qmm_dequant_affine(fmt, w, scales, biases, k, n, out, stream)
    return out


def matmul_glu(act, fmt, w_gate, w_up, x, k: int, n: int, *, y=None, j_start=0, j_end=0,
               accumulate=False, path=PATH_AUTO, stream=None, flags=0):
    """y = act(x Wg) * (x Wu) ("swiglu" / "geglu") for torch CUDA tensors; the
    scratch of the several-token form is a torch allocation on x's device."""
    import torch
    if x.dim() == 1:
        x = x.unsqueeze(0)
    nt = x.shape[0]
    if y is None:
        y = torch.empty((nt, n), dtype=torch.float32, device=x.device)
    a = make_args(fmt, w_gate, x, y, k, n, nt, w_len=w_gate.numel() * w_gate.element_size(),
                  j_start=j_start, j_end=j_end, accumulate=accumulate, path=path, stream=stream,
                  flags=flags)
    need = qmm_glu_workspace_bytes(a)
    ws = None
    if need:
        ws = torch.empty(need, dtype=torch.uint8, device=x.device)
        a.workspace, a.workspace_bytes = ws.data_ptr(), need
    qmm_matmul_glu(a, w_up, act)
    _keep_until_done(ws, stream)
    return y


# -------------------------------------------------- paged key-value cache ----

ROPE_HALF, ROPE_PAIRS = 0, 1
ROPE_STYLES = {"half": ROPE_HALF, "pairs": ROPE_PAIRS}


def qmm_kv_page_bytes(fmt_k, fmt_v, page_size: int, n_kv_heads: int, head_dim: int) -> int:
    return load().qmm_kv_page_bytes(_fmt(fmt_k), _fmt(fmt_v), page_size, n_kv_heads, head_dim)


def qmm_kv_append(args: qmm_kv_append_args) -> int:
    return _check(load().qmm_kv_append(ctypes.byref(args)))


def qmm_kv_read(args: qmm_kv_read_args) -> int:
    return _check(load().qmm_kv_read(ctypes.byref(args)))


def qmm_attend(args: qmm_attend_args) -> int:
    return _check(load().qmm_attend(ctypes.byref(args)))


def qmm_attend_workspace_bytes(args: qmm_attend_args) -> int:
    return load().qmm_attend_workspace_bytes(ctypes.byref(args))


_torch_mod = None


def _torch():
    """torch, imported on first use (the C-named calls above work without it)."""
    global _torch_mod
    if _torch_mod is None:
        import torch
        _torch_mod = torch
    return _torch_mod


def _stream_of(stream, tensor):
    """The raw handle of `stream`, or of torch's current stream on the tensor's device."""
    if stream is not None:
        return _stream(stream)
    torch = _torch()
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)   # a tenth of current_stream's time
    index = tensor.device.index
    if raw is not None and index is not None:
        return raw(index)
    return torch.cuda.current_stream(tensor.device).cuda_stream


# Scratch of attend calls on torch's current stream, kept per host thread, device
# and stream and grown as needed; an allocation per call took 6 of a small call's
# 15 us. The kernels of a stream run one after the other, so the calls that one
# thread makes on it can share scratch. Calls of two threads cannot: a call is two
# launches, which another thread's may come between on a stream that both use.
_attend_scratch = threading.local()


def _scratch_of_stream(need: int, device, handle: int):
    held = _attend_scratch.__dict__          # of this thread
    key = (device.index, handle)
    ws = held.get(key)
    if ws is None or ws.numel() < need:
        ws = held[key] = _torch().empty(max(need, 1 << 20), dtype=_torch().uint8, device=device)
    return ws


class KvCache:
    """A pool of cache pages: `pages` is a uint8 CUDA tensor [n_pages, page bytes]
    (one page holds page_size positions of every kv head), the formats are
    "f16", "bf16", "q8_0" or "q4_0" (the same for K and V, or K "q8_0" and V
    "q4_0"). head_dim is a multiple of 32 up to 512; attend takes 64, 96, 128, 192
    and 256 of them. Page tables and lengths belong to the calls. Every tensor of a call
    is on the pool's device: the kernels follow the addresses that they are given."""

    def __init__(self, fmt_k, fmt_v, pages, page_size: int, n_kv_heads: int, head_dim: int):
        self.fmt_k, self.fmt_v, self.pages = _fmt(fmt_k), _fmt(fmt_v), pages
        self.page_size, self.n_kv_heads, self.head_dim = page_size, n_kv_heads, head_dim
        self.page_bytes = qmm_kv_page_bytes(fmt_k, fmt_v, page_size, n_kv_heads, head_dim)
        if self.page_bytes == 0:
            raise QmmError(2, qmm_last_error())
        if pages.dim() != 2 or pages.shape[1] != self.page_bytes or not pages.is_contiguous() \
                or pages.element_size() != 1:
            raise ValueError(f"pages must be contiguous bytes [n_pages, {self.page_bytes}], "
                             f"got {tuple(pages.shape)}")
        self._device = pages.get_device()    # -1: host memory
        # each call starts from a copy of its arguments with the pool filled in
        pool = qmm_kv_cache(self.fmt_k, self.fmt_v, pages.data_ptr(), pages.numel(), pages.shape[0],
                            page_size, n_kv_heads, head_dim)
        self._append = qmm_kv_append_args(cache=pool)
        self._read = qmm_kv_read_args(cache=pool)
        self._attend = qmm_attend_args(cache=pool)

    def __setattr__(self, name, value):
        # the filled-in arguments hold the pool's address and shape
        if name in self.__dict__:
            raise AttributeError(f"a cache's {name} does not change")
        super().__setattr__(name, value)

    @classmethod
    def empty(cls, fmt_k, fmt_v, n_pages: int, page_size: int, n_kv_heads: int, head_dim: int,
              device="cuda"):
        """A cache over `n_pages` pages of new memory (not cleared)."""
        import torch
        size = qmm_kv_page_bytes(fmt_k, fmt_v, page_size, n_kv_heads, head_dim)
        if size == 0:
            raise QmmError(2, qmm_last_error())
        pages = torch.empty((n_pages, size), dtype=torch.uint8, device=device)
        return cls(fmt_k, fmt_v, pages, page_size, n_kv_heads, head_dim)

    def _args(self, template, page_table, lens):
        """A call's arguments with its int32 page_table [n_seqs, max_pages] (rows may be strided)
        and lens [n_seqs], and n_seqs."""
        here = self._device
        if here < 0 or page_table.get_device() != here or lens.get_device() != here:
            lens_only = page_table.get_device() == here >= 0
            self._other_device(*(("lens", lens) if lens_only else ("page_table", page_table)))
        int32 = _torch().int32
        shape, count = page_table.shape, lens.shape
        if len(shape) != 2 or len(count) != 1 or shape[0] != count[0] \
                or page_table.dtype is not int32 or lens.dtype is not int32:
            raise ValueError("page_table and lens must be int32 [n_seqs, max_pages] and [n_seqs]")
        n_seqs, max_pages = shape
        stride = page_table.stride()
        if (max_pages > 1 and stride[1] != 1) or (n_seqs > 1 and lens.stride()[0] != 1):
            raise ValueError("entries of page_table's rows and of lens must be adjacent")
        a = type(template).from_buffer_copy(template)
        c = a.cache
        c.page_table = page_table.data_ptr()
        c.table_stride = stride[0] if n_seqs > 1 else max_pages
        c.max_pages = max_pages
        c.lens = lens.data_ptr()
        c.n_seqs = n_seqs
        return a, n_seqs

    def _other_device(self, name, t):
        raise ValueError(f"{name} ({t.device}) and the cache's pages ({self.pages.device}) must be on one CUDA device")

    def view(self, page_table, lens) -> qmm_kv_cache:
        """The C description of this pool with a call's page_table and lens."""
        return self._args(self._read, page_table, lens)[0].cache

    def rows(self, name, t, n_seqs: int):
        """Row stride of fp32 rows [n_seqs, n_new, heads, head_dim] and their n_new and heads."""
        shape, dim = t.shape, self.head_dim
        if len(shape) != 4 or shape[0] != n_seqs or shape[3] != dim or t.dtype is not _torch().float32:
            raise ValueError(f"{name} must be float32 [{n_seqs}, n_new, heads, {dim}], "
                             f"got {tuple(shape)}")
        if t.get_device() != self._device:
            self._other_device(name, t)
        s0, s1, s2, s3 = t.stride()
        n_new, heads = shape[1], shape[2]
        row = s1 if n_new > 1 else s0 if n_seqs > 1 else heads * dim
        if s3 != 1 or (heads > 1 and s2 != dim) or (n_new > 1 and n_seqs > 1 and s0 != n_new * s1):
            raise ValueError(f"{name}: the heads of a row must be adjacent and rows equally spaced")
        return row, n_new, heads


def rope_table(n_pos: int, n_rot: int, base: float = 10000.0, scale: float = 1.0, device="cuda"):
    """Rotary table [n_pos, n_rot / 2, 2] float32 for kv_append: cos and sin of
    position * scale * base^(-2 a / n_rot), from float64."""
    import torch
    turns = base ** (-2.0 * torch.arange(n_rot // 2, dtype=torch.float64) / n_rot)
    angle = torch.arange(n_pos, dtype=torch.float64).unsqueeze(1) * (scale * turns)
    return torch.stack((angle.cos(), angle.sin()), -1).float().to(device)


def kv_append(cache: KvCache, k, v, page_table, lens, *, q=None, q_out=None, rope=None,
              rope_style="half", stream=None):
    """Append the rows k, v [n_seqs, n_new, n_kv_heads, head_dim] at the last
    n_new of each sequence's lens positions; with `rope` (see rope_table) k is
    rotated, and q [n_seqs, n_new, n_heads, head_dim] into q_out (returned; a
    new tensor when not given)."""
    a, n_seqs = cache._args(cache._append, page_table, lens)
    a.k_stride, n_new, heads = cache.rows("k", k, n_seqs)
    a.v_stride, v_new, v_heads = cache.rows("v", v, n_seqs)
    if heads != cache.n_kv_heads or v_new != n_new or v_heads != heads:
        raise ValueError(f"k and v must have {cache.n_kv_heads} heads and the same rows")
    a.n_new, a.k, a.v = n_new, k.data_ptr(), v.data_ptr()
    if q is not None:
        a.q_stride, q_new, a.n_heads = cache.rows("q", q, n_seqs)
        if q_out is None:
            q_out = _torch().empty(q.shape, dtype=q.dtype, device=q.device)
        a.q_out_stride, o_new, o_heads = cache.rows("q_out", q_out, n_seqs)
        if q_new != n_new or o_new != n_new or o_heads != a.n_heads:
            raise ValueError("q and q_out must have k's rows and the same heads")
        a.q, a.q_out = q.data_ptr(), q_out.data_ptr()
    if rope is not None:
        shape = rope.shape
        if len(shape) != 3 or shape[2] != 2 or not rope.is_contiguous() \
                or rope.dtype is not _torch().float32:
            raise ValueError("rope must be contiguous float32 [positions, n_rot / 2, 2]")
        if rope.get_device() != cache._device:
            cache._other_device("rope", rope)
        a.rope, a.rope_len, a.n_rot = rope.data_ptr(), shape[0], 2 * shape[1]
    a.rope_style = ROPE_STYLES[rope_style] if isinstance(rope_style, str) else int(rope_style)
    a.stream = _stream_of(stream, cache.pages)
    qmm_kv_append(a)
    return q_out


def kv_read(cache: KvCache, page_table, lens, count: int, *, first=None, k=None, v=None,
            stream=None):
    """fp32 k and v [n_seqs, count, n_kv_heads, head_dim] of the positions
    first .. first + count - 1 of every sequence (first None or -1: its last
    `count` positions); zeros where a sequence has no such position."""
    a, n_seqs = cache._args(cache._read, page_table, lens)
    shape = (n_seqs, count, cache.n_kv_heads, cache.head_dim)
    a.first, a.count = -1 if first is None else first, count
    given, torch = (("k", k), ("v", v)), _torch()
    for name, t in given:
        if t is None:
            continue
        if t.shape != shape or not t.is_contiguous() or t.dtype is not torch.float32:
            raise ValueError(f"{name} must be contiguous float32 {shape}")
        if t.get_device() != cache._device:
            cache._other_device(name, t)
    if k is None:
        k = torch.empty(shape, dtype=torch.float32, device=cache.pages.device)
    if v is None:
        v = torch.empty(shape, dtype=torch.float32, device=cache.pages.device)
    a.k, a.v = k.data_ptr(), v.data_ptr()
    a.stream = _stream_of(stream, cache.pages)
    qmm_kv_read(a)
    return k, v


def attend(cache: KvCache, q, page_table, lens, *, scale=None, window=0, out=None, workspace=None,
           stream=None):
    """Attention of the last n_new positions of every sequence over the cache:
    q [n_seqs, n_new, n_heads, head_dim] (n_heads a multiple of the cache's kv
    heads), scale 1 / sqrt(head_dim) unless given, window 0 (all positions) or
    the number of last positions that a row sees. Returns out, shaped like q
    (the given one when passed). Scratch is `workspace` (uint8) when given;
    else one that the host thread keeps for torch's current stream, or (on another `stream`,
    or under graph capture) a torch allocation of the call."""
    a, n_seqs = cache._args(cache._attend, page_table, lens)
    a.q_stride, n_new, n_heads = cache.rows("q", q, n_seqs)
    if out is None:
        out = _torch().empty(q.shape, dtype=q.dtype, device=q.device)
    a.out_stride, o_new, o_heads = cache.rows("out", out, n_seqs)
    if o_new != n_new or o_heads != n_heads:
        raise ValueError("out must have q's shape")
    a.n_new, a.n_heads, a.q, a.out = n_new, n_heads, q.data_ptr(), out.data_ptr()
    a.scale = cache.head_dim ** -0.5 if scale is None else scale
    a.window = window
    a.stream = _stream_of(stream, cache.pages)
    ws = None
    if workspace is None:
        need, torch = qmm_attend_workspace_bytes(a), _torch()
        if need and stream is None and not torch.cuda.is_current_stream_capturing():
            workspace = _scratch_of_stream(need, cache.pages.device, a.stream)
        elif need:
            ws = workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    if workspace is not None:
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
        if workspace.get_device() != cache._device:
            cache._other_device("workspace", workspace)
        a.workspace, a.workspace_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    qmm_attend(a)
    if stream is not None:
        _keep_until_done(ws, stream)
    return out
