"""ctypes binding of libllmint8.so (the C ABI in include/llmint8.h).

Argument marshalling only: every step of the layer runs in the library's
CUDA kernels. PyTorch provides device memory and streams. The functions keep
the C names; tensors are passed as device pointers, the stream as the current
torch stream. If the library is missing, loading fails loudly: there is no
CPU fallback.
"""
from __future__ import annotations

import bisect
import ctypes
import math
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libllmint8.so")

OK = 0
STATUS_NAMES = {0: "OK", -1: "ERR_NULL", -2: "ERR_SHAPE", -3: "ERR_ALIGN",
                -4: "ERR_WORKSPACE", -5: "ERR_CUDA", -6: "ERR_DEVICE_STATUS",
                -7: "ERR_ARG", -8: "ERR_UNSUPPORTED", -9: "ERR_TOO_LARGE"}
NOALLOC_MAX_SCRATCH_BYTES = 64 << 20  # LLMINT8_NOALLOC_MAX_SCRATCH_BYTES
# device status bits (LLMINT8_DEV_*)
DEV_TIMEOUT_SELFTEST = 0x20
DEV_OUTLIER_CAP = 0x40
SCALE_VECTORWISE = 0  # LLMINT8_SCALE_VECTORWISE: per row of X / column of W
# where the prefill path builds the fp16 outlier rows of W (LLMINT8_WO_*)
WO_SHARED, WO_BEFORE_GEMM, WO_EACH_CTA = 0, 1, 2
SCALE_TENSORWISE = 1  # LLMINT8_SCALE_TENSORWISE: one constant per tensor
# llmint8_matmul_opts.path (LLMINT8_PATH_*)
PATH_AUTO, PATH_PREFILL, PATH_DECODE, PATH_PREFILL_SINGLE, PATH_PREFILL_PAIR = 0, 1, 2, 3, 4

_c_i64, _c_i32, _c_f32 = ctypes.c_int64, ctypes.c_int32, ctypes.c_float
_vp, _sz = ctypes.c_void_p, ctypes.c_size_t


class llmint8_weight(ctypes.Structure):
    _fields_ = [("h", _c_i64), ("o", _c_i64), ("wq_dev", _vp), ("aw_dev", _vp),
                ("w16_dev", _vp)]


class llmint8_matmul_opts(ctypes.Structure):
    _fields_ = [("gemm_event_start", _vp), ("gemm_event_stop", _vp),
                ("ci_dev", _vp), ("path", _c_i32), ("launches", _c_i32),
                ("x_scale", _c_i32), ("max_outliers", _c_i32),
                ("status_host", _vp), ("wo_build", _c_i32)]


class llmint8_adapters(ctypes.Structure):
    _fields_ = [("h", _c_i64), ("o", _c_i64), ("n", _c_i32), ("r", _c_i32),
                ("a_dev", _vp), ("b_dev", _vp), ("scale_dev", _vp), ("rank_dev", _vp)]


class llmint8_grad(ctypes.Structure):
    _fields_ = [("grad_dev", _vp), ("out_dev", _vp), ("n", _c_i64), ("type", _c_i32)]


class llmint8_grad_list(ctypes.Structure):
    _fields_ = [("table_dev", _vp), ("table_bytes", _sz), ("n", _c_i64), ("chunks", _c_i64)]


class Llmint8Error(RuntimeError):
    def __init__(self, fn: str, code: int):
        self.code = code
        super().__init__(f"{fn} failed: {STATUS_NAMES.get(code, code)}"
                         f" ({status_string(code) if _lib is not None else ''})")


_lib = None


def load_library():
    """Load libllmint8.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} not found: build it with `python -m "
            "mixed_precision_int8_b200.build` (or __graft_entry__.build())")
    lib = ctypes.CDLL(LIB_PATH)
    sig = {
        "llmint8_status_string": ([_c_i32], ctypes.c_char_p),
        "llmint8_workspace_size": ([_c_i64, _c_i64, _c_i64], _sz),
        "llmint8_workspace_size_ex": ([_c_i64, _c_i64, _c_i64, _c_i64], _sz),
        "llmint8_workspace_size_host": ([_c_i64, _c_i64, _c_i64], _sz),
        "llmint8_workspace_size_host_ex": ([_c_i64, _c_i64, _c_i64, _c_i64], _sz),
        "llmint8_workspace_init": ([_vp, _sz, _vp], _c_i32),
        "llmint8_prepare_weight": ([_vp, _c_i64, _c_i64,
                                    ctypes.POINTER(llmint8_weight), _vp], _c_i32),
        "llmint8_prepare_weight_ex": ([_vp, _c_i64, _c_i64, _c_i32,
                                       ctypes.POINTER(llmint8_weight), _vp], _c_i32),
        "llmint8_prepare_weight_cols": ([_vp, _c_i64, _c_i64, _c_i64, _c_i64, _c_i32,
                                         ctypes.POINTER(llmint8_weight), _vp], _c_i32),
        "llmint8_quantize_rows_scratch_size": ([_c_i64], _sz),
        "llmint8_quantize_rows_ex": ([_vp, _c_i64, _c_i64, _c_f32, _c_i32, _vp,
                                      _vp, _vp, _vp, _vp, _vp, _sz, _vp], _c_i32),
        "llmint8_quantize_rows": ([_vp, _c_i64, _c_i64, _c_f32, _vp, _vp, _vp,
                                   _vp, _vp, _vp, _sz, _vp], _c_i32),
        "llmint8_matmul": ([_vp, _c_i64, ctypes.POINTER(llmint8_weight), _c_f32,
                            _vp, _vp, _sz, _vp], _c_i32),
        "llmint8_matmul_ex": ([_vp, _c_i64, ctypes.POINTER(llmint8_weight),
                               _c_f32, _vp, _vp, _sz,
                               ctypes.POINTER(llmint8_matmul_opts), _vp], _c_i32),
        "llmint8_matmul_host": ([_vp, _c_i64, ctypes.POINTER(llmint8_weight),
                                 _c_f32, _vp, _vp, _sz, _vp], _c_i32),
        "llmint8_matmul_host_ex": ([_vp, _c_i64, ctypes.POINTER(llmint8_weight),
                                    _c_f32, _vp, _vp, _sz,
                                    ctypes.POINTER(llmint8_matmul_opts), _vp], _c_i32),
        "llmint8_read_outlier_tiles": ([_vp, _sz, _c_i64, _c_i64, _c_i64, _vp,
                                        _vp, _vp, _vp], _c_i32),
        "llmint8_read_outlier_tiles_ex": ([_vp, _sz, _c_i64, _c_i64, _c_i64,
                                           _c_i64, _vp, _vp, _vp, _vp], _c_i32),
        "llmint8_read_device_status": ([_vp, _sz, _vp, _vp], _c_i32),
        "llmint8_decode_max_rows": ([], _c_i64),
        "llmint8_prefill_kernel": ([_c_i64, _c_i64, _c_i64], _c_i32),
        "llmint8_matmul_noalloc": ([_vp, _c_i64, ctypes.POINTER(llmint8_weight),
                                    _c_f32, _vp, _vp], _c_i32),
        "llmint8_wait_selftest": ([_vp, _sz, ctypes.c_uint64, _vp], _c_i32),
        "llmint8_noalloc_read_device_status": ([_vp, _vp], _c_i32),
        "llmint8_adapters_workspace_size": ([_c_i64, _c_i64, _c_i64, _c_i32, _c_i32], _sz),
        "llmint8_adapters_forward": ([_vp, _c_i64, ctypes.POINTER(llmint8_adapters), _vp, _vp,
                                      _vp, _vp, _vp, _sz, _vp], _c_i32),
        "llmint8_adapters_backward": ([_vp, _vp, _c_i64, ctypes.POINTER(llmint8_adapters),
                                       _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp], _c_i32),
        "llmint8_matmul_backward_workspace_size": ([_c_i64, _c_i64, _c_i64], _sz),
        "llmint8_matmul_backward": ([_vp, _c_i64, ctypes.POINTER(llmint8_weight), _vp, _vp,
                                     _vp, _sz, _vp], _c_i32),
        "llmint8_layernorm_forward": ([_vp, _c_i32, _c_i64, _c_i64, _vp, _vp, _c_i32, _c_f32,
                                       _vp, _vp, _vp, _vp], _c_i32),
        "llmint8_layernorm_workspace_size": ([_c_i64, _c_i64], _sz),
        "llmint8_layernorm_backward": ([_vp, _vp, _c_i32, _c_i64, _c_i64, _vp, _c_i32, _vp,
                                        _vp, _vp, _vp, _vp, _vp, _sz, _vp], _c_i32),
        "llmint8_grad_list_size": ([_c_i64], _sz),
        "llmint8_grad_list_init": ([ctypes.POINTER(llmint8_grad), _c_i64,
                                    ctypes.POINTER(llmint8_grad_list), _vp], _c_i32),
        "llmint8_clip_grads": ([ctypes.POINTER(llmint8_grad_list), _c_f32, _vp, _vp], _c_i32),
    }
    for name, (args, res) in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    _lib = lib
    return lib


EXPORTED = ("llmint8_status_string", "llmint8_workspace_size",
            "llmint8_workspace_size_host", "llmint8_workspace_init",
            "llmint8_prepare_weight", "llmint8_quantize_rows_scratch_size",
            "llmint8_quantize_rows", "llmint8_matmul", "llmint8_matmul_ex",
            "llmint8_matmul_host", "llmint8_read_outlier_tiles",
            "llmint8_read_device_status", "llmint8_decode_max_rows",
            "llmint8_matmul_noalloc", "llmint8_wait_selftest",
            "llmint8_prepare_weight_ex", "llmint8_quantize_rows_ex",
            "llmint8_matmul_host_ex", "llmint8_workspace_size_ex",
            "llmint8_workspace_size_host_ex", "llmint8_read_outlier_tiles_ex",
            "llmint8_noalloc_read_device_status", "llmint8_prepare_weight_cols",
            "llmint8_prefill_kernel",
            "llmint8_adapters_workspace_size", "llmint8_adapters_forward",
            "llmint8_adapters_backward", "llmint8_matmul_backward_workspace_size",
            "llmint8_matmul_backward", "llmint8_layernorm_forward",
            "llmint8_layernorm_workspace_size", "llmint8_layernorm_backward",
            "llmint8_grad_list_size", "llmint8_grad_list_init", "llmint8_clip_grads")


def status_string(code: int) -> str:
    return load_library().llmint8_status_string(code).decode()


def _check(fn: str, code: int):
    if code != OK:
        raise Llmint8Error(fn, code)


def _stream(stream: Optional[torch.cuda.Stream] = None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    return ctypes.c_void_p(t.data_ptr())


def _f16_dev(t: torch.Tensor, name: str):
    if t.dtype != torch.float16 or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA float16 tensor")


class PreparedWeight:
    """Device buffers of a prepared weight: wq int8 [o,h], aw float32 [o],
    and optionally the fp16 weight itself (w16 [h,o], kept referenced here)
    whose outlier rows then serve as the fp16 outlier rows of W."""

    def __init__(self, wq: torch.Tensor, aw: torch.Tensor,
                 w16: Optional[torch.Tensor] = None):
        self.wq = wq
        self.aw = aw
        self.w16 = w16
        self.o, self.h = wq.shape
        self.c = llmint8_weight(self.h, self.o, wq.data_ptr(), aw.data_ptr(),
                                w16.data_ptr() if w16 is not None else None)


class Workspace:
    """A caller-owned device workspace (torch uint8 buffer) for one stream.

    max_outliers (0: h, any alpha) sizes its outlier tiles; calls on it pass
    the same capacity to the library."""

    def __init__(self, s: int, h: int, o: int, device=None, host: bool = False,
                 max_outliers: int = 0):
        lib = load_library()
        size_fn = (lib.llmint8_workspace_size_host_ex if host
                   else lib.llmint8_workspace_size_ex)
        self.nbytes = int(size_fn(s, h, o, int(max_outliers)))
        if self.nbytes == 0:
            raise ValueError(f"invalid workspace size arguments {(s, h, o, max_outliers)}")
        self.buf = torch.empty(self.nbytes, dtype=torch.uint8,
                               device=device or "cuda")
        self.s, self.h, self.o = s, h, o
        self.max_outliers = int(max_outliers)
        _check("llmint8_workspace_init",
               lib.llmint8_workspace_init(_ptr(self.buf), self.nbytes, _stream()))


def llmint8_workspace_size(s: int, h: int, o: int, max_outliers: int = 0) -> int:
    return int(load_library().llmint8_workspace_size_ex(s, h, o, int(max_outliers)))


class HostStatusWord:
    """A pinned host int32 that the device writes: passed as status_host, it
    receives the status bits of each call's kernels, and the next call on it
    raises ERR_DEVICE_STATUS (code -6) before enqueuing anything."""

    def __init__(self):
        self.t = torch.zeros((1,), dtype=torch.int32).pin_memory()

    @property
    def value(self) -> int:
        return int(self.t[0].item())

    def clear(self):
        self.t[0] = 0


def llmint8_decode_max_rows() -> int:
    return int(load_library().llmint8_decode_max_rows())


def llmint8_prefill_kernel(s: int, h: int, o: int) -> int:
    """PATH_* value of the kernel the automatic choice runs for [s,h] x [h,o]
    on the current device (PATH_DECODE, PATH_PREFILL_SINGLE or
    PATH_PREFILL_PAIR)."""
    r = int(load_library().llmint8_prefill_kernel(int(s), int(h), int(o)))
    _check("llmint8_prefill_kernel", r if r < 0 else 0)
    return r


def llmint8_prepare_weight(W: torch.Tensor, stream=None,
                           keep_fp16: bool = False,
                           w_scale: int = SCALE_VECTORWISE) -> PreparedWeight:
    """W fp16 [h,o] on the GPU -> PreparedWeight (int8 [o,h] codes + scales).

    With keep_fp16 the weight keeps W (a reference, not a copy) and the
    layer's fp16 outlier rows of W are W's own values. w_scale =
    SCALE_TENSORWISE gives every column the one absmax of all of W."""
    _f16_dev(W, "W")
    h, o = W.shape
    wq = torch.empty((o, h), dtype=torch.int8, device=W.device)
    aw = torch.empty((o,), dtype=torch.float32, device=W.device)
    pw = PreparedWeight(wq, aw, W if keep_fp16 else None)
    _check("llmint8_prepare_weight_ex", load_library().llmint8_prepare_weight_ex(
        _ptr(W), h, o, int(w_scale), ctypes.byref(pw.c), _stream(stream)))
    return pw


def llmint8_prepare_weight_cols(W: torch.Tensor, col0: int, o: int, stream=None,
                                w_scale: int = SCALE_VECTORWISE) -> PreparedWeight:
    """Columns [col0, col0 + o) of W fp16 [h, o_total] (on the GPU) prepared
    as a weight of their own: one column-parallel shard."""
    _f16_dev(W, "W")
    h, ldw = W.shape
    wq = torch.empty((o, h), dtype=torch.int8, device=W.device)
    aw = torch.empty((o,), dtype=torch.float32, device=W.device)
    pw = PreparedWeight(wq, aw, None)
    _check("llmint8_prepare_weight_cols", load_library().llmint8_prepare_weight_cols(
        _ptr(W), h, ldw, int(col0), int(o), int(w_scale), ctypes.byref(pw.c),
        _stream(stream)))
    return pw


def llmint8_quantize_rows(X: torch.Tensor, alpha: float = 6.0, stream=None,
                          x_scale: int = SCALE_VECTORWISE):
    """Steps 1 and 4 (activation side) -> (Xq, ax, flags, idx, n_outliers).

    x_scale = SCALE_TENSORWISE quantises all rows against one constant.

    n_outliers is a 1-element device tensor (it is never read back here);
    idx holds valid entries in its first n_outliers slots.
    """
    _f16_dev(X, "X")
    s, h = X.shape
    dev = X.device
    lib = load_library()
    Xq = torch.empty((s, h), dtype=torch.int8, device=dev)
    ax = torch.empty((s,), dtype=torch.float32, device=dev)
    flags = torch.empty((h,), dtype=torch.uint8, device=dev)
    idx = torch.empty((h,), dtype=torch.int32, device=dev)
    n = torch.empty((1,), dtype=torch.int32, device=dev)
    nb = int(lib.llmint8_quantize_rows_scratch_size(h))
    scratch = torch.empty(max(nb, 256), dtype=torch.uint8, device=dev)
    _check("llmint8_quantize_rows_ex", lib.llmint8_quantize_rows_ex(
        _ptr(X), s, h, float(alpha), int(x_scale), _ptr(Xq), _ptr(ax),
        _ptr(flags), _ptr(idx), _ptr(n), _ptr(scratch), nb, _stream(stream)))
    return Xq, ax, flags, idx, n


def llmint8_matmul(X: torch.Tensor, w: PreparedWeight, alpha: float = 6.0,
                   out: Optional[torch.Tensor] = None,
                   workspace: Optional[Workspace] = None,
                   ci: Optional[torch.Tensor] = None, path: int = 0,
                   events=None, stream=None,
                   x_scale: int = SCALE_VECTORWISE,
                   status_host: Optional[HostStatusWord] = None,
                   wo_build: int = WO_SHARED) -> torch.Tensor:
    """C = LLM.int8()(X, W): X fp16 [s,h] on the GPU -> fp16 [s,o].

    ci (optional, int32 [s,o]) receives the exact int32 accumulators; path
    forces a kernel (PATH_*: prefill 1, decode 2, prefill with one CTA per
    tile 3, prefill with CTA pairs 4); events = (start, stop)
    torch.cuda.Event pair recorded around the GEMM kernel; x_scale =
    SCALE_TENSORWISE quantises X with one constant for the whole tensor;
    status_host (a HostStatusWord) reports device anomalies on the next call;
    wo_build picks where the fp16 outlier rows of W are built (WO_*).
    The workspace's max_outliers is passed along.
    """
    _f16_dev(X, "X")
    s, h = X.shape
    if h != w.h:
        raise ValueError(f"X has h={h}, weight has h={w.h}")
    if out is None:
        out = torch.empty((s, w.o), dtype=torch.float16, device=X.device)
    if workspace is None:
        workspace = Workspace(s, h, w.o, device=X.device)
    opts = llmint8_matmul_opts()
    opts.path = int(path)
    opts.x_scale = int(x_scale)
    opts.max_outliers = workspace.max_outliers
    opts.wo_build = int(wo_build)
    if status_host is not None:
        opts.status_host = status_host.t.data_ptr()
    if ci is not None:
        if ci.dtype != torch.int32 or ci.shape != (s, w.o):
            raise ValueError("ci must be int32 [s,o]")
        opts.ci_dev = ci.data_ptr()
    if events is not None:
        for e in events:  # torch creates its events lazily, on first record
            if not e.cuda_event:
                e.record(stream if stream is not None
                         else torch.cuda.current_stream())
        opts.gemm_event_start = events[0].cuda_event
        opts.gemm_event_stop = events[1].cuda_event
    _check("llmint8_matmul_ex", load_library().llmint8_matmul_ex(
        _ptr(X), s, ctypes.byref(w.c), float(alpha), _ptr(out),
        _ptr(workspace.buf), workspace.nbytes, ctypes.byref(opts),
        _stream(stream)))
    llmint8_matmul.last_launches = int(opts.launches)
    return out


def llmint8_matmul_noalloc(X: torch.Tensor, w: PreparedWeight,
                           alpha: float = 6.0,
                           out: Optional[torch.Tensor] = None,
                           stream=None) -> torch.Tensor:
    """llmint8_matmul without a caller workspace: the library's own static
    device scratch is used instead (see include/llmint8.h for who needs this
    and its limits). Only `out` may be allocated here, by torch, when it is
    not given."""
    _f16_dev(X, "X")
    s, h = X.shape
    if h != w.h:
        raise ValueError(f"X has h={h}, weight has h={w.h}")
    if out is None:
        out = torch.empty((s, w.o), dtype=torch.float16, device=X.device)
    _check("llmint8_matmul_noalloc", load_library().llmint8_matmul_noalloc(
        _ptr(X), s, ctypes.byref(w.c), float(alpha), _ptr(out), _stream(stream)))
    return out


def llmint8_matmul_host(X_host: torch.Tensor, w: PreparedWeight,
                        alpha: float, out_host: torch.Tensor,
                        workspace: Workspace, stream=None,
                        x_scale: int = SCALE_VECTORWISE) -> torch.Tensor:
    """End-to-end form: host fp16 X in, host fp16 C out (synchronises)."""
    if X_host.is_cuda or out_host.is_cuda:
        raise ValueError("X_host and out_host must be host tensors")
    s, h = X_host.shape
    opts = llmint8_matmul_opts()
    opts.x_scale = int(x_scale)
    opts.max_outliers = workspace.max_outliers
    _check("llmint8_matmul_host_ex", load_library().llmint8_matmul_host_ex(
        _ptr(X_host), s, ctypes.byref(w.c), float(alpha), _ptr(out_host),
        _ptr(workspace.buf), workspace.nbytes, ctypes.byref(opts), _stream(stream)))
    return out_host


def llmint8_read_outlier_tiles(workspace: Workspace, s: Optional[int] = None,
                               stream=None, tiles: bool = True):
    """(n, XO [s,n] fp16, WO [n,o] fp16) of the last matmul on `workspace`,
    which had `s` rows (default: the row count the workspace was sized for;
    the workspace layout depends on it). tiles=False reads |O| alone."""
    h, o = workspace.h, workspace.o
    s = workspace.s if s is None else int(s)
    cap = workspace.max_outliers or h
    n = ctypes.c_int32(0)
    if not tiles:
        _check("llmint8_read_outlier_tiles_ex", load_library().llmint8_read_outlier_tiles_ex(
            _ptr(workspace.buf), workspace.nbytes, s, h, o, workspace.max_outliers,
            ctypes.byref(n), None, None, _stream(stream)))
        return n.value, None, None
    XO = torch.empty((s * cap,), dtype=torch.float16)
    WO = torch.empty((cap * o,), dtype=torch.float16)
    _check("llmint8_read_outlier_tiles_ex", load_library().llmint8_read_outlier_tiles_ex(
        _ptr(workspace.buf), workspace.nbytes, s, h, o, workspace.max_outliers,
        ctypes.byref(n), _ptr(XO), _ptr(WO), _stream(stream)))
    k = n.value
    if k > cap:  # the call kept no outlier tiles
        return k, None, None
    return k, XO[: s * k].view(s, k), WO[: k * o].view(k, o)


def llmint8_wait_selftest(workspace: Workspace, limit_ns: int = 2_000_000,
                          stream=None) -> None:
    """Enqueue the bounded-wait self-test (its waits run out by design)."""
    _check("llmint8_wait_selftest", load_library().llmint8_wait_selftest(
        _ptr(workspace.buf), workspace.nbytes, int(limit_ns), _stream(stream)))


def llmint8_noalloc_read_device_status(stream=None) -> int:
    """Status bits of the allocation-free entry point on the current device
    (read and cleared; its state block is cleared too)."""
    bits = ctypes.c_int32(0)
    rc = load_library().llmint8_noalloc_read_device_status(ctypes.byref(bits),
                                                           _stream(stream))
    if rc not in (OK, -6):
        _check("llmint8_noalloc_read_device_status", rc)
    return bits.value


def llmint8_read_device_status(workspace: Workspace, stream=None) -> int:
    bits = ctypes.c_int32(0)
    rc = load_library().llmint8_read_device_status(
        _ptr(workspace.buf), workspace.nbytes, ctypes.byref(bits), _stream(stream))
    if rc not in (OK, -6):
        _check("llmint8_read_device_status", rc)
    return bits.value


# ------------------------------------------------ operators next to the layer

_TYPES = {torch.float16: 0, torch.float32: 1, torch.bfloat16: 2}  # LLMINT8_F16 / F32 / BF16


class _Launch:
    """The device and stream a call runs on: the tensors' own device, made
    current for the call, and `stream` (which must be that device's) or its
    current stream. What the call allocates belongs to that stream."""

    __slots__ = ("device", "stream", "_prev", "_ctx")

    def __init__(self, device: torch.device, stream=None):
        self.device = device
        self.stream = stream

    def __enter__(self):
        index, stream = self.device.index, self.stream
        self._prev = self._ctx = None
        if stream is not None and stream.device != self.device:
            raise ValueError(f"stream is on {stream.device}, the tensors are on {self.device}")
        prev = torch.cuda.current_device()
        if prev != index:
            torch.cuda.set_device(index)
            self._prev = prev
        if stream is None:
            return torch._C._cuda_getCurrentRawStream(index)
        self._ctx = torch.cuda.stream(stream)
        self._ctx.__enter__()
        return stream.cuda_stream

    def __exit__(self, *exc):
        if self._ctx is not None:
            self._ctx.__exit__(*exc)
        if self._prev is not None:
            torch.cuda.set_device(self._prev)
        return False


def _tensor(t: torch.Tensor, name: str, dtype, shape, device=None):
    """t must be a contiguous CUDA tensor of this dtype and shape (a tuple),
    on `device` when given. Returns its address."""
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or not (
            t.is_cuda if device is None else t.device == device):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {shape} on "
                         f"{device or 'a CUDA device'}, not {t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _optional(t, name: str, dtype, shape, device):
    return None if t is None else _tensor(t, name, dtype, shape, device)


def _matrix(t: torch.Tensor, name: str):
    if t.dim() != 2:
        raise ValueError(f"{name} must have two dimensions")
    return t.shape


class _OpWorkspace:
    """A caller-owned device workspace (torch uint8 buffer) for one stream."""

    def __init__(self, nbytes: int, args, device=None):
        self.nbytes = int(nbytes)
        if self.nbytes == 0:
            raise ValueError(f"invalid workspace size arguments {args}")
        device = torch.empty(0, device=device or "cuda").device
        with _Launch(device) as st:
            self.buf = torch.empty(self.nbytes, dtype=torch.uint8, device=device)
            _check("llmint8_workspace_init",
                   load_library().llmint8_workspace_init(_ptr(self.buf), self.nbytes, st))


class AdapterWorkspace(_OpWorkspace):
    """Workspace of llmint8_adapters_forward and _backward for up to s rows."""

    def __init__(self, s: int, h: int, o: int, n: int, r: int, device=None):
        super().__init__(load_library().llmint8_adapters_workspace_size(s, h, o, n, r),
                         (s, h, o, n, r), device)


class BackwardWorkspace(_OpWorkspace):
    """Workspace of llmint8_matmul_backward for [s, o] gradients of an [h, o] weight."""

    def __init__(self, s: int, h: int, o: int, device=None):
        super().__init__(load_library().llmint8_matmul_backward_workspace_size(s, h, o),
                         (s, h, o), device)


class LayerNormWorkspace(_OpWorkspace):
    """Workspace of llmint8_layernorm_backward for [s, h] rows."""

    def __init__(self, s: int, h: int, device=None):
        super().__init__(load_library().llmint8_layernorm_workspace_size(s, h), (s, h), device)


def _ws(workspace, device):
    """(address, bytes) of a workspace on this device."""
    buf = workspace.buf
    if buf.device != device:
        raise ValueError(f"workspace is on {buf.device}, not on {device}")
    return buf.data_ptr(), workspace.nbytes


class Adapters:
    """n low-rank adapters beside one projection: A fp16 [n, r, h], B fp16
    [n, r, o] (row t of each: one rank-one term), scale float32 [n], and
    optionally the rank each adapter uses (int32 [n], default all r). The
    tensors are kept, not copied: their values may change between calls."""

    def __init__(self, A: torch.Tensor, B: torch.Tensor, scale: torch.Tensor,
                 ranks: Optional[torch.Tensor] = None):
        if A.dim() != 3 or B.dim() != 3:
            raise ValueError("A must be [n, r, h] and B [n, r, o]")
        n, r, h = A.shape
        o = B.shape[2]
        dev = A.device
        _tensor(A, "A", torch.float16, (n, r, h))
        _tensor(B, "B", torch.float16, (n, r, o), dev)
        _tensor(scale, "scale", torch.float32, (n,), dev)
        if ranks is not None:
            _tensor(ranks, "ranks", torch.int32, (n,), dev)
        self.A, self.B, self.scale, self.ranks = A, B, scale, ranks
        self.n, self.r, self.h, self.o, self.device = n, r, h, o, dev
        self.c = llmint8_adapters(h, o, n, r, A.data_ptr(), B.data_ptr(), scale.data_ptr(),
                                  ranks.data_ptr() if ranks is not None else None)
        self.ref = ctypes.byref(self.c)


def llmint8_adapters_forward(X: torch.Tensor, adapters: Adapters, ids: torch.Tensor,
                             base: Optional[torch.Tensor] = None,
                             out: Optional[torch.Tensor] = None,
                             v: Optional[torch.Tensor] = None,
                             workspace: Optional[AdapterWorkspace] = None,
                             stream=None) -> torch.Tensor:
    """out = base + every row's adapter: X fp16 [s,h], ids int32 [s] (a row
    whose id is outside [0, n) uses none) -> fp16 [s,o].

    base (fp16 [s,o], default zeros) is the projection's output; out may be
    base itself. v (float32 [s,r]) receives X . A for the backward pass.

    Without a workspace the call makes one of its own, whose status (a wait
    that ran out: llmint8_read_device_status) nobody can read afterwards."""
    ad, dev = adapters, adapters.device
    s = _matrix(X, "X")[0]
    f16 = torch.float16
    args = (_tensor(X, "X", f16, (s, ad.h), dev), s, ad.ref,
            _tensor(ids, "ids", torch.int32, (s,), dev),
            _optional(base, "base", f16, (s, ad.o), dev))
    pv = _optional(v, "v", torch.float32, (s, ad.r), dev)
    with _Launch(dev, stream) as st:
        if out is None:
            out = torch.empty((s, ad.o), dtype=f16, device=dev)
        if workspace is None:
            workspace = AdapterWorkspace(s, ad.h, ad.o, ad.n, ad.r, dev)
        _check("llmint8_adapters_forward", load_library().llmint8_adapters_forward(
            *args, _tensor(out, "out", f16, (s, ad.o), dev), pv, *_ws(workspace, dev), st))
    return out


def llmint8_adapters_backward(X: Optional[torch.Tensor], dY: torch.Tensor, adapters: Adapters,
                              ids: torch.Tensor, v: Optional[torch.Tensor] = None,
                              base: Optional[torch.Tensor] = None,
                              dX: Optional[torch.Tensor] = None,
                              dA: Optional[torch.Tensor] = None,
                              dB: Optional[torch.Tensor] = None,
                              workspace: Optional[AdapterWorkspace] = None, stream=None,
                              want=(True, True, True)):
    """(dX fp16 [s,h], dA float32 [n,r,h], dB float32 [n,r,o]) for dY fp16
    [s,o], the gradient of llmint8_adapters_forward's out.

    v is what the forward call left there (default: computed again); base
    (fp16 [s,h], default zeros) is the gradient that reaches X through the
    projection and is added into dX, which may be base itself. want = (dX, dA,
    dB) leaves out what is not wanted (None is returned in its place).

    Without a workspace the call makes one of its own, whose status (a wait
    that ran out: llmint8_read_device_status) nobody can read afterwards."""
    ad, dev = adapters, adapters.device
    s = _matrix(dY, "dY")[0]
    f16, f32 = torch.float16, torch.float32
    want_x, want_a, want_b = (w or t is not None for w, t in zip(want, (dX, dA, dB)))
    if X is None and (want_a or (want_b and v is None)):
        raise ValueError("X is needed for dA, and for dB without v")
    args = (_optional(X, "X", f16, (s, ad.h), dev), _tensor(dY, "dY", f16, (s, ad.o), dev), s,
            ad.ref, _tensor(ids, "ids", torch.int32, (s,), dev),
            _optional(v, "v", f32, (s, ad.r), dev), _optional(base, "base", f16, (s, ad.h), dev))
    with _Launch(dev, stream) as st:
        if dX is None and want_x:
            dX = torch.empty((s, ad.h), dtype=f16, device=dev)
        if dA is None and want_a:
            dA = torch.empty((ad.n, ad.r, ad.h), dtype=f32, device=dev)
        if dB is None and want_b:
            dB = torch.empty((ad.n, ad.r, ad.o), dtype=f32, device=dev)
        if workspace is None:
            workspace = AdapterWorkspace(s, ad.h, ad.o, ad.n, ad.r, dev)
        _check("llmint8_adapters_backward", load_library().llmint8_adapters_backward(
            *args, _optional(dX, "dX", f16, (s, ad.h), dev),
            _optional(dA, "dA", f32, (ad.n, ad.r, ad.h), dev),
            _optional(dB, "dB", f32, (ad.n, ad.r, ad.o), dev), *_ws(workspace, dev), st))
    return dX, dA, dB


def llmint8_matmul_backward(dY: torch.Tensor, w: PreparedWeight,
                            base: Optional[torch.Tensor] = None,
                            out: Optional[torch.Tensor] = None,
                            workspace: Optional[BackwardWorkspace] = None,
                            stream=None) -> torch.Tensor:
    """dX = dY . W^T through the frozen int8 weight (+ base): dY fp16 [s,o]
    -> fp16 [s,h]. out may be base itself.

    Without a workspace the call makes one of its own, whose status (a wait
    that ran out: llmint8_read_device_status) nobody can read afterwards."""
    s = _matrix(dY, "dY")[0]
    dev, f16 = w.wq.device, torch.float16
    py, pb = _tensor(dY, "dY", f16, (s, w.o), dev), _optional(base, "base", f16, (s, w.h), dev)
    with _Launch(dev, stream) as st:
        if out is None:
            out = torch.empty((s, w.h), dtype=f16, device=dev)
        if workspace is None:
            workspace = BackwardWorkspace(s, w.h, w.o, dev)
        _check("llmint8_matmul_backward", load_library().llmint8_matmul_backward(
            py, s, ctypes.byref(w.c), pb, _tensor(out, "out", f16, (s, w.h), dev),
            *_ws(workspace, dev), st))
    return out


def _ln_type(t: torch.Tensor, name: str) -> int:
    code = _TYPES.get(t.dtype, 2)
    if code == 2:
        raise ValueError(f"{name} must be float16 or float32, not {t.dtype}")
    return code


def llmint8_layernorm_forward(X: torch.Tensor, gamma: torch.Tensor,
                              beta: Optional[torch.Tensor] = None, eps: float = 1e-5,
                              out: Optional[torch.Tensor] = None, stream=None):
    """(Y fp16 [s,h], mean float32 [s], rstd float32 [s]) = layer norm of the
    rows of X (fp16 or fp32 [s,h]); gamma and beta [h] are fp16 or fp32 alike.
    out may be an fp16 X itself."""
    s, h = _matrix(X, "X")
    dev, ptype = X.device, gamma.dtype
    tx, tp = _ln_type(X, "X"), _ln_type(gamma, "gamma")
    args = (_tensor(X, "X", X.dtype, (s, h)), tx, s, h, _tensor(gamma, "gamma", ptype, (h,), dev),
            _optional(beta, "beta", ptype, (h,), dev), tp, eps)
    with _Launch(dev, stream) as st:
        if out is None:
            out = torch.empty((s, h), dtype=torch.float16, device=dev)
        mean, rstd = torch.empty((2, s), dtype=torch.float32, device=dev).unbind(0)
        _check("llmint8_layernorm_forward", load_library().llmint8_layernorm_forward(
            *args, _tensor(out, "out", torch.float16, (s, h), dev), mean.data_ptr(),
            rstd.data_ptr(), st))
    return out, mean, rstd


def llmint8_layernorm_backward(dY: torch.Tensor, X: torch.Tensor, gamma: torch.Tensor,
                               mean: torch.Tensor, rstd: torch.Tensor,
                               dX: Optional[torch.Tensor] = None,
                               workspace: Optional[LayerNormWorkspace] = None, stream=None):
    """(dX in X's type, dgamma float32 [h], dbeta float32 [h]) for dY fp16
    [s,h], with the forward call's mean and rstd. dX may be X itself, or dY
    where X is fp16.

    Without a workspace the call makes one of its own, whose status (a wait
    that ran out: llmint8_read_device_status) nobody can read afterwards."""
    s, h = _matrix(X, "X")
    dev, f32 = X.device, torch.float32
    tx, tp = _ln_type(X, "X"), _ln_type(gamma, "gamma")
    args = (_tensor(dY, "dY", torch.float16, (s, h), dev), _tensor(X, "X", X.dtype, (s, h)), tx,
            s, h, _tensor(gamma, "gamma", gamma.dtype, (h,), dev), tp,
            _tensor(mean, "mean", f32, (s,), dev), _tensor(rstd, "rstd", f32, (s,), dev))
    with _Launch(dev, stream) as st:
        if dX is None:
            dX = torch.empty_like(X)
        dgamma, dbeta = torch.empty((2, h), dtype=f32, device=dev).unbind(0)
        if workspace is None:
            workspace = LayerNormWorkspace(s, h, dev)
        _check("llmint8_layernorm_backward", load_library().llmint8_layernorm_backward(
            *args, _tensor(dX, "dX", X.dtype, (s, h), dev), dgamma.data_ptr(), dbeta.data_ptr(),
            *_ws(workspace, dev), st))
    return dX, dgamma, dbeta


def _address_ranges(tensors):
    """The addresses [begin, end) of contiguous tensors, merged and in order."""
    merged = []
    for begin, end in sorted((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size())
                             for t in tensors if t.numel()):
        if merged and begin <= merged[-1][1]:
            merged[-1] = (merged[-1][0], max(end, merged[-1][1]))
        else:
            merged.append((begin, end))
    return merged


def _overlaps(ranges, t: torch.Tensor) -> bool:
    """Whether t shares a byte with one of these merged ranges."""
    begin = t.data_ptr()
    end = begin + t.numel() * t.element_size()
    i = bisect.bisect_left(ranges, (end,))  # the ranges before i begin below end
    return i > 0 and begin < min(end, ranges[i - 1][1])


class GradList:
    """Gradients laid out once, on their device's current stream, for repeated
    llmint8_clip_grads: contiguous CUDA tensors (fp16, bf16 or fp32) on one
    device, none listed twice, clipped in place, or into `outs` (tensors of the
    same sizes and types). The tensors are kept, not copied."""

    def __init__(self, grads, outs=None, device=None):
        self.grads = list(grads)
        self.outs = self.grads if outs is None else list(outs)
        if len(self.grads) != len(self.outs):
            raise ValueError("outs must match grads one for one")
        device = self.grads[0].device if self.grads else torch.empty(
            0, device=device or "cuda").device
        if device.type != "cuda":
            raise ValueError(f"grads must be on a CUDA device, not on {device}")
        n = len(self.grads)
        items = (llmint8_grad * max(n, 1))()
        for i, (g, out) in enumerate(zip(self.grads, self.outs)):
            if g.dtype not in _TYPES:
                raise ValueError(f"grads[{i}] must be float16, bfloat16 or float32")
            items[i] = llmint8_grad(_tensor(g, f"grads[{i}]", g.dtype, g.shape, device),
                                    _tensor(out, f"outs[{i}]", g.dtype, g.shape, device),
                                    g.numel(), _TYPES[g.dtype])
        self.device = device
        self.ranges = _address_ranges(self.grads + self.outs)
        lib = load_library()
        nbytes = int(lib.llmint8_grad_list_size(n))
        with _Launch(device) as st:
            self.table = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=device)
            self.c = llmint8_grad_list(self.table.data_ptr(), nbytes, 0, 0)
            _check("llmint8_grad_list_init", lib.llmint8_grad_list_init(
                items, n, ctypes.byref(self.c), st))


def llmint8_clip_grads(grads: GradList, max_norm: float, norm: Optional[torch.Tensor] = None,
                       stream=None) -> torch.Tensor:
    """The global norm of a list's gradients (float32 [1], no part of them or
    of their outputs); they are scaled so that it does not exceed max_norm (inf:
    the norm alone)."""
    dev = grads.device
    if norm is not None and _overlaps(grads.ranges, norm):
        raise ValueError("norm lies in one of the list's gradients or outputs")
    with _Launch(dev, stream) as st:
        if norm is None:
            norm = torch.empty((1,), dtype=torch.float32, device=dev)
        _check("llmint8_clip_grads", load_library().llmint8_clip_grads(
            ctypes.byref(grads.c), max_norm, _tensor(norm, "norm", torch.float32, (1,), dev), st))
    return norm


_cudart = None


def event_elapsed_ms(start, stop) -> float:
    """Milliseconds between two torch.cuda.Event objects recorded by the
    library (torch's own elapsed_time only accepts events torch recorded)."""
    global _cudart
    if _cudart is None:
        cand = os.path.join(os.path.dirname(torch.__file__), "..", "nvidia",
                            "cuda_runtime", "lib", "libcudart.so.12")
        _cudart = ctypes.CDLL(cand if os.path.exists(cand) else "libcudart.so.12")
        _cudart.cudaEventElapsedTime.argtypes = [ctypes.POINTER(ctypes.c_float),
                                                 _vp, _vp]
        _cudart.cudaEventElapsedTime.restype = ctypes.c_int
    ms = ctypes.c_float(0.0)
    rc = _cudart.cudaEventElapsedTime(ctypes.byref(ms), _vp(start.cuda_event),
                                      _vp(stop.cuda_event))
    if rc != 0:
        raise RuntimeError(f"cudaEventElapsedTime failed ({rc})")
    return float(ms.value)


def effective_tops(s: int, h: int, o: int, seconds: float) -> float:
    return 2.0 * s * h * o / seconds / 1e12 if seconds > 0 else math.nan
