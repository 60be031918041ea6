"""Python binding of libaffqmm (include/affqmm.h): argument marshalling only.

Every step of the projection runs in the library's CUDA kernels; this module
turns torch tensors into pointers, sizes and the current CUDA stream, and
turns status codes into exceptions.  PyTorch supplies device memory and
streams.  There is no fallback: if libaffqmm.so is missing or cannot be
loaded, every call raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import os
import struct
from dataclasses import dataclass, field

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.environ.get("AFFQMM_LIB_PATH") or os.path.join(_PKG, "libaffqmm.so")   # the in-tree build unless overridden

MAX_STACK = 8
MAX_M = 1 << 20
NOALLOC_MAX_M = 16                   # rows affqmm_run_noalloc takes
WORKSPACE_ZEROED = 256 + 65536 * 4   # leading workspace bytes kept zero between calls

STATUS_NAMES = {
    0: "AFFQMM_OK", 1: "AFFQMM_E_NULL", 2: "AFFQMM_E_BITS", 3: "AFFQMM_E_GROUP",
    4: "AFFQMM_E_SHAPE", 5: "AFFQMM_E_ALIGN", 6: "AFFQMM_E_M", 7: "AFFQMM_E_WORKSPACE",
    8: "AFFQMM_E_TIMEOUT", 9: "AFFQMM_E_CUDA", 10: "AFFQMM_E_ARG", 11: "AFFQMM_E_DEVICE",
    12: "AFFQMM_E_SCRATCH",
}


class AffqmmError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        self.name = STATUS_NAMES.get(status, str(status))
        super().__init__(f"{what}: {self.name} ({strerror(status)})")


class CWeight(ctypes.Structure):
    _fields_ = [("bits", ctypes.c_int32), ("group", ctypes.c_int32), ("N", ctypes.c_int64),
                ("K", ctypes.c_int64), ("packed", ctypes.c_void_p)]


class CCache(ctypes.Structure):
    _fields_ = [("type", ctypes.c_int32), ("page", ctypes.c_int32), ("heads", ctypes.c_int32), ("dim", ctypes.c_int32),
                ("pages", ctypes.c_int64), ("page_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p)]


class CStep(ctypes.Structure):
    _fields_ = [("capacity", ctypes.c_int64), ("starts", ctypes.c_void_p), ("lens", ctypes.c_void_p),
                ("ring_state", ctypes.c_void_p), ("slots", ctypes.c_void_p), ("positions", ctypes.c_void_p),
                ("requests", ctypes.c_void_p), ("status", ctypes.c_void_p)]


class CRope(ctypes.Structure):
    _fields_ = [("turns", ctypes.c_void_p), ("axis", ctypes.c_void_p), ("rotary", ctypes.c_int32),
                ("neighbour", ctypes.c_int32), ("axes", ctypes.c_int32)]


class CRows(ctypes.Structure):
    _fields_ = [("p", ctypes.c_void_p), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class CLanes(ctypes.Structure):
    _fields_ = [("p", ctypes.c_void_p), ("batch_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64)]


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded libaffqmm.so (raises if it is not built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"libaffqmm.so is not built ({LIB_PATH}); run group_affine_bit_gb300.build.build()")
        L = ctypes.CDLL(LIB_PATH)
        vp, i64, i32, szp = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.POINTER(ctypes.c_size_t)
        wp = ctypes.POINTER(CWeight)
        sig = {
            "affqmm_strerror": (ctypes.c_char_p, [i32]),
            "affqmm_version": (i32, []),
            "affqmm_packed_bytes": (i32, [i32, i32, i64, i64, szp]),
            "affqmm_pack": (i32, [i32, i32, i64, i64, vp, vp, vp, vp, vp]),
            "affqmm_workspace_bytes": (i32, [wp, i64, szp]),
            "affqmm_workspace_bytes_stacked": (i32, [i32, wp, i64, szp]),
            "affqmm_run": (i32, [wp, vp, i64, vp, vp, ctypes.c_size_t, vp]),
            "affqmm_run_stacked": (i32, [i32, wp, vp, i64, ctypes.POINTER(vp), vp, ctypes.c_size_t, vp]),
            "affqmm_dequant": (i32, [wp, vp, vp]),
            "affqmm_workspace_status": (i32, [vp, vp]),
            "affqmm_run_noalloc": (i32, [wp, vp, i64, vp, vp]),
            "affqmm_run_host": (i32, [wp, vp, i64, vp, vp, vp, vp, ctypes.c_size_t, vp]),
            "affqmm_run_exact": (i32, [wp, vp, i64, vp, vp, ctypes.c_size_t, vp]),
            "affqmm_embed_rows": (i32, [wp, vp, i64, i32, ctypes.c_uint16, vp, vp, vp]),
            "affqmm_test_fault_wait": (i32, [i64]),
            "affqmm_run_exact_sums": (i32, [wp, vp, vp, i64, vp, vp, ctypes.c_size_t, vp]),
            "affqmm_run_geglu": (i32, [wp, vp, vp, i64, i32, vp, vp, ctypes.c_size_t, vp]),
            "affqmm_rows_bytes": (i32, [i32, i32, i64, i64, szp]),
            "affqmm_pack_rows": (i32, [wp, vp, vp]),
            "affqmm_embed_rows_copy": (i32, [wp, vp, vp, i64, i32, ctypes.c_uint16, vp, vp, vp]),
            "affqmm_paged_plan": (i32, [i64, vp, vp, vp, vp, i64, i64, vp, i64, vp, i32, vp, vp]),
            "affqmm_rope_append": (i32, [vp, vp, vp, vp, vp, vp, i64, i32, vp, i64, vp, vp, vp]),
            "affqmm_paged_attention_workspace_bytes": (i32, [vp, i32, i32, szp]),
            "affqmm_paged_attention": (i32, [vp, vp, vp, vp, i64, i32, i32, vp, i64, i64, vp, ctypes.c_float, i32, vp, vp,
                                             ctypes.c_size_t, vp]),
        }
        for name, (res, args) in sig.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def strerror(status: int) -> str:
    return lib().affqmm_strerror(int(status)).decode()


def _check(rc: int, what: str):
    if rc != 0:
        raise AffqmmError(rc, what)


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)   # cheap current-stream lookup, when present


def _stream_ptr(stream, device_index: int | None = None) -> int:
    if stream is None:
        if _raw_stream is not None:
            return int(_raw_stream(torch.cuda.current_device() if device_index is None else device_index))
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream)


def _under(stream, device):
    """Context in which torch allocates and fills for a call's stream: what is made there is ready when the call's
    kernel runs, and goes back to that stream's memory."""
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream.cuda_stream), device)
    return torch.cuda.stream(stream)


def _empty(shape, dtype, device, stream) -> torch.Tensor:
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with _under(stream, device):
        return torch.empty(shape, dtype=dtype, device=device)


def _status_ptr(status: torch.Tensor | None, device_index: int) -> int | None:
    """The address of a call's status word."""
    if status is None:
        return None
    if status.get_device() != device_index or status.dtype not in (torch.int32, torch.uint32) or status.numel() < 1:
        raise ValueError(f"status must be an int32 or uint32 tensor of one word on cuda:{device_index}")
    return status.data_ptr()


def _capture_id(stream_ptr: int) -> int:
    """Which capture a stream is in, 0 for none."""
    status, number = ctypes.c_int(0), ctypes.c_uint64(0)
    rc = ctypes.CDLL("libcuda.so.1").cuStreamGetCaptureInfo_v2(ctypes.c_void_p(stream_ptr), ctypes.byref(status),
                                                               ctypes.byref(number), None, None, None)
    if rc != 0:
        raise RuntimeError(f"cuStreamGetCaptureInfo: error {rc}")
    return number.value if status.value else 0


@dataclass
class PackedWeight:
    """A packed affine table (device memory owned by the torch tensor `packed`)."""
    bits: int
    group: int
    N: int
    K: int
    packed: torch.Tensor
    _c: CWeight | None = field(default=None, repr=False, compare=False)
    _ws: dict = field(default_factory=dict, repr=False, compare=False)   # (M, device) -> workspace bytes

    def cstruct(self) -> CWeight:
        """The C view of this weight (built once: the storage never moves)."""
        if self._c is None:
            self._c = CWeight(self.bits, self.group, self.N, self.K,
                              self.packed.data_ptr() if self.packed.numel() else None)
        return self._c


def packed_bytes(bits: int, group: int, N: int, K: int) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().affqmm_packed_bytes(bits, group, N, K, ctypes.byref(out)), "affqmm_packed_bytes")
    return out.value


def pack(codes: torch.Tensor, scales: torch.Tensor, biases: torch.Tensor, bits: int, group: int,
         stream=None) -> PackedWeight:
    """codes uint8 [N,K]; scales, biases bf16 [N,K/group]; all on one CUDA device."""
    N, K = codes.shape
    for t in (codes, scales, biases):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("pack wants contiguous CUDA tensors")
    if codes.dtype != torch.uint8 or scales.dtype != torch.bfloat16 or biases.dtype != torch.bfloat16:
        raise ValueError("pack wants uint8 codes and bf16 scales and biases")
    nbytes = packed_bytes(bits, group, N, K)
    packed = _empty(max(nbytes, 1), torch.uint8, codes.device, stream)
    _check(lib().affqmm_pack(bits, group, N, K, codes.data_ptr(), scales.data_ptr(), biases.data_ptr(),
                             packed.data_ptr(), _stream_ptr(stream)), "affqmm_pack")
    return PackedWeight(bits, group, N, K, packed)


def workspace_bytes(w: PackedWeight, M: int) -> int:
    key = (M, torch.cuda.current_device())
    got = w._ws.get(key)
    if got is None:
        out = ctypes.c_size_t(0)
        cw = w.cstruct()
        _check(lib().affqmm_workspace_bytes(ctypes.byref(cw), M, ctypes.byref(out)), "affqmm_workspace_bytes")
        got = w._ws[key] = out.value
    return got


def _warray(ws):
    arr = (CWeight * len(ws))()
    for i, w in enumerate(ws):
        arr[i] = w.cstruct()
    return arr


def workspace_bytes_stacked(ws, M: int) -> int:
    out = ctypes.c_size_t(0)
    arr = _warray(ws)
    _check(lib().affqmm_workspace_bytes_stacked(len(ws), arr, M, ctypes.byref(out)),
           "affqmm_workspace_bytes_stacked")
    return out.value


class Workspace:
    """A zero-filled device buffer that grows on demand.  The library leaves it
    zeroed after every call; calls sharing one must be stream-ordered.  It is
    made and filled on the stream of the call that needs it.  A captured graph
    keeps a buffer's address, so one that is outgrown is kept too (each is at
    least twice the last), and one made during a capture, which only a replay
    fills, serves that capture alone."""

    def __init__(self, device=None):
        self.device = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
        self.buf = torch.zeros(0, dtype=torch.uint8, device=self.device)
        self._kept: list = []        # outgrown buffers
        self._capture = 0            # the capture that fills `buf`, 0: it is filled

    def get(self, nbytes: int, stream=None) -> torch.Tensor:
        """The buffer for a call on `stream` (the current one if None)."""
        if self._capture or self.buf.numel() < nbytes:
            self._make(nbytes, stream)
        return self.buf

    def _make(self, nbytes: int, stream):
        with _under(stream, self.device):
            capture = _capture_id(_stream_ptr(stream, self.device.index)) if torch.cuda.is_current_stream_capturing() else 0
            if capture and capture == self._capture and self.buf.numel() >= nbytes:
                return
            if not self._capture:    # the memory of one made during a capture stays with its graph
                if self.buf.numel():
                    self._kept.append(self.buf)
                nbytes = max(nbytes, 2 * self.buf.numel())
            self.buf = torch.zeros(nbytes, dtype=torch.uint8, device=self.device)
            self._capture = capture


_workspaces: dict = {}


def default_workspace(device, stream_ptr: int | None = None) -> Workspace:
    """One workspace per (device, stream): calls on one stream never overlap."""
    index = torch.device(device).index if not isinstance(device, int) else device
    if stream_ptr is None:
        stream_ptr = _stream_ptr(None, index)
    key = (index, stream_ptr)
    ws = _workspaces.get(key)
    if ws is None:
        ws = _workspaces[key] = Workspace(torch.device("cuda", index))
    return ws


def _check_x(x: torch.Tensor, K: int):
    if not x.is_cuda or x.dtype != torch.bfloat16 or x.dim() != 2 or x.shape[1] != K or not x.is_contiguous():
        raise ValueError(f"x must be a contiguous CUDA bf16 [M, {K}] tensor")


def run(w: PackedWeight, x: torch.Tensor, y: torch.Tensor | None = None, workspace: Workspace | None = None,
        stream=None) -> torch.Tensor:
    """y[M, N] = bf16(x @ dequant(W)^T) with fp32 accumulation."""
    _check_x(x, w.K)
    M = x.shape[0]
    dev = x.get_device()
    if y is None:
        y = _empty((M, w.N), torch.bfloat16, x.device, stream)
    sp = _stream_ptr(stream, dev)
    ws = workspace or default_workspace(dev, sp)
    need = workspace_bytes(w, M)
    buf = ws.get(need, stream)
    cw = w.cstruct()
    _check(lib().affqmm_run(ctypes.byref(cw), x.data_ptr(), M, y.data_ptr(), buf.data_ptr() if need else None,
                            buf.numel(), sp), "affqmm_run")
    return y


def run_exact(w: PackedWeight, x: torch.Tensor, y: torch.Tensor | None = None, workspace: Workspace | None = None,
              stream=None) -> torch.Tensor:
    """affqmm_run_exact (M <= 16): y = bf16(sum_g s_g * sum q x + b_g * sum x), the
    exact-codes form (the weights are not rounded to bf16)."""
    _check_x(x, w.K)
    M = x.shape[0]
    dev = x.get_device()
    if y is None:
        y = _empty((M, w.N), torch.bfloat16, x.device, stream)
    sp = _stream_ptr(stream, dev)
    ws = workspace or default_workspace(dev, sp)
    need = workspace_bytes(w, M)
    buf = ws.get(need, stream)
    cw = w.cstruct()
    _check(lib().affqmm_run_exact(ctypes.byref(cw), x.data_ptr(), M, y.data_ptr(), buf.data_ptr() if need else None,
                                  buf.numel(), sp), "affqmm_run_exact")
    return y


FORM_ROUNDED, FORM_EXACT, FORM_EXACT_SUMS = 0, 1, 2


def _check_xsums(xsums: torch.Tensor, M: int, w: PackedWeight, x: torch.Tensor):
    G = w.K // w.group
    if (not xsums.is_cuda or xsums.dtype != torch.float32 or tuple(xsums.shape) != (M, G)
            or not xsums.is_contiguous() or xsums.device != x.device):
        raise ValueError(f"xsums must be a contiguous CUDA float32 [{M}, {G}] tensor on {x.device}")


def run_exact_sums(w: PackedWeight, x: torch.Tensor, xsums: torch.Tensor, y: torch.Tensor | None = None,
                   workspace: Workspace | None = None, stream=None) -> torch.Tensor:
    """affqmm_run_exact_sums (M <= 16): the exact-codes form with the group sums
    of x (float32 [M, K/group]) as the kernel that produced x wrote them."""
    _check_x(x, w.K)
    M = x.shape[0]
    _check_xsums(xsums, M, w, x)
    dev = x.get_device()
    if y is None:
        y = _empty((M, w.N), torch.bfloat16, x.device, stream)
    sp = _stream_ptr(stream, dev)
    ws = workspace or default_workspace(dev, sp)
    need = workspace_bytes(w, M)
    buf = ws.get(need, stream)
    cw = w.cstruct()
    _check(lib().affqmm_run_exact_sums(ctypes.byref(cw), x.data_ptr(), xsums.data_ptr(), M, y.data_ptr(),
                                       buf.data_ptr() if need else None, buf.numel(), sp), "affqmm_run_exact_sums")
    return y


def run_geglu(w: PackedWeight, x: torch.Tensor, form: int = FORM_ROUNDED, xsums: torch.Tensor | None = None,
              h: torch.Tensor | None = None, workspace: Workspace | None = None, stream=None) -> torch.Tensor:
    """affqmm_run_geglu (M <= 16): a gate/up stack (rows interleaved in 16-row
    blocks) with GeGLU as its epilogue; returns h bf16 [M, N/2]."""
    _check_x(x, w.K)
    M = x.shape[0]
    if form == FORM_EXACT_SUMS:
        _check_xsums(xsums, M, w, x)
    dev = x.get_device()
    if h is None:
        h = _empty((M, w.N // 2), torch.bfloat16, x.device, stream)
    sp = _stream_ptr(stream, dev)
    ws = workspace or default_workspace(dev, sp)
    need = workspace_bytes(w, M)
    buf = ws.get(need, stream)
    cw = w.cstruct()
    xs = xsums.data_ptr() if (form == FORM_EXACT_SUMS and xsums is not None) else None
    _check(lib().affqmm_run_geglu(ctypes.byref(cw), x.data_ptr(), xs, M, int(form), h.data_ptr(),
                                  buf.data_ptr() if need else None, buf.numel(), sp), "affqmm_run_geglu")
    return h


def run_host(w: PackedWeight, x: torch.Tensor, y: torch.Tensor, x_dev: torch.Tensor, y_dev: torch.Tensor,
             workspace: Workspace | None = None, stream=None) -> torch.Tensor:
    """affqmm_run_host: x (host, bf16 [M, K]) is copied into x_dev, the projection
    runs into y_dev, and y_dev is copied back into y (host, bf16 [M, N]), all on
    the stream.  Pinned host tensors keep the copies asynchronous; y is complete
    once the stream has passed the call."""
    M = x.shape[0]
    if (x.is_cuda or y.is_cuda or x.dtype != torch.bfloat16 or y.dtype != torch.bfloat16
            or tuple(x.shape) != (M, w.K) or tuple(y.shape) != (M, w.N)
            or not x.is_contiguous() or not y.is_contiguous()):
        raise ValueError(f"x and y must be contiguous host bf16 tensors [M, {w.K}] and [M, {w.N}]")
    _check_x(x_dev, w.K)
    if (x_dev.shape[0] != M or y_dev.dtype != torch.bfloat16 or tuple(y_dev.shape) != (M, w.N)
            or not y_dev.is_contiguous() or y_dev.device != x_dev.device):
        raise ValueError(f"x_dev and y_dev must be contiguous bf16 [M, {w.K}] and [M, {w.N}] on one device")
    dev = x_dev.get_device()
    sp = _stream_ptr(stream, dev)
    ws = workspace or default_workspace(dev, sp)
    need = workspace_bytes(w, M)
    buf = ws.get(need, stream)
    cw = w.cstruct()
    _check(lib().affqmm_run_host(ctypes.byref(cw), x.data_ptr(), M, y.data_ptr(), x_dev.data_ptr(), y_dev.data_ptr(),
                                 buf.data_ptr() if need else None, buf.numel(), sp), "affqmm_run_host")
    return y


def run_stacked(ws_list, x: torch.Tensor, ys=None, workspace: Workspace | None = None, stream=None):
    """Several projections of the same x in one launch; returns a list of y."""
    K = ws_list[0].K
    _check_x(x, K)
    M = x.shape[0]
    if ys is None:
        ys = [_empty((M, w.N), torch.bfloat16, x.device, stream) for w in ws_list]
    sp = _stream_ptr(stream, x.get_device())
    wsp = workspace or default_workspace(x.get_device(), sp)
    need = workspace_bytes_stacked(ws_list, M)
    buf = wsp.get(need, stream)
    arr = _warray(ws_list)
    yp = (ctypes.c_void_p * len(ys))(*[y.data_ptr() for y in ys])
    _check(lib().affqmm_run_stacked(len(ws_list), arr, x.data_ptr(), M, yp, buf.data_ptr() if need else None,
                                    buf.numel(), sp), "affqmm_run_stacked")
    return ys


def dequant(w: PackedWeight, stream=None) -> torch.Tensor:
    """The bf16 [N, K] weights as the run kernels dequantize them (test hook)."""
    out = _empty((w.N, w.K), torch.bfloat16, w.packed.device, stream)
    cw = w.cstruct()
    _check(lib().affqmm_dequant(ctypes.byref(cw), out.data_ptr(), _stream_ptr(stream)), "affqmm_dequant")
    return out


def workspace_status(buf: torch.Tensor, stream=None) -> int:
    """Read a workspace's device status word (0 = ok; after a timeout the
    library zeroes the status word and the merge counters again)."""
    return int(lib().affqmm_workspace_status(buf.data_ptr(), _stream_ptr(stream)))


def test_fault_wait(cycles: int) -> None:
    """Test hook: while cycles > 0, decode (M <= 16) and attention launches first wait, at
    most `cycles` SM clock cycles, on a barrier nothing completes, so the
    bounded wait runs out and the workspace status reports a timeout."""
    _check(lib().affqmm_test_fault_wait(int(cycles)), "affqmm_test_fault_wait")


def run_noalloc(w: PackedWeight, x: torch.Tensor, y: torch.Tensor, stream=None) -> torch.Tensor:
    """affqmm_run_noalloc: y = bf16(x @ dequant(W)^T) for M <= 16 rows, with no
    workspace.  For callers that cannot allocate device memory; the library
    works in its own fixed 8 MiB scratch array instead, shared by every call on
    the device, so calls must not overlap on the GPU.  `y` must be given: this
    wrapper allocates nothing either."""
    _check_x(x, w.K)
    M = x.shape[0]
    if y.dtype != torch.bfloat16 or tuple(y.shape) != (M, w.N) or not y.is_contiguous() or y.device != x.device:
        raise ValueError(f"y must be a contiguous bf16 [{M}, {w.N}] tensor on {x.device}")
    cw = w.cstruct()
    _check(lib().affqmm_run_noalloc(ctypes.byref(cw), x.data_ptr(), M, y.data_ptr(), _stream_ptr(stream)),
           "affqmm_run_noalloc")
    return y


def _embed_args(w: PackedWeight, ids: torch.Tensor, scale, out, stream):
    if not ids.is_cuda or ids.dtype != torch.int32 or ids.dim() != 1 or not ids.is_contiguous():
        raise ValueError("ids must be a contiguous int32 CUDA vector")
    T = ids.shape[0]
    if out is None:
        out = _empty((T, w.K), torch.bfloat16, ids.device, stream)
    if out.dtype != torch.bfloat16 or tuple(out.shape) != (T, w.K) or not out.is_contiguous():
        raise ValueError(f"out must be a contiguous bf16 [{T}, {w.K}] tensor")
    sbits = 0 if scale is None else int(torch.tensor([scale], dtype=torch.bfloat16).view(torch.int16).item()) & 0xFFFF
    return T, out, sbits


def embed_rows(w: PackedWeight, ids: torch.Tensor, scale: float | None = None, out: torch.Tensor | None = None,
               status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """out[t, k] = bf16(W[ids[t], k] * bf16(scale)) (or W's rows when scale is None),
    W = bf16(s*q + b): rows gathered from the packed table.  ids: int32 CUDA [T]."""
    T, out, sbits = _embed_args(w, ids, scale, out, stream)
    cw = w.cstruct()
    _check(lib().affqmm_embed_rows(ctypes.byref(cw), ids.data_ptr(), T, 0 if scale is None else 1, sbits,
                                   out.data_ptr(), _status_ptr(status, ids.get_device()),
                                   _stream_ptr(stream)), "affqmm_embed_rows")
    return out


def rows_bytes(bits: int, group: int, N: int, K: int) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().affqmm_rows_bytes(bits, group, N, K, ctypes.byref(out)), "affqmm_rows_bytes")
    return out.value


def pack_rows(w: PackedWeight, stream=None) -> torch.Tensor:
    """The row-contiguous copy of a packed table that embed_rows_copy gathers from."""
    nbytes = rows_bytes(w.bits, w.group, w.N, w.K)
    rows = _empty(max(nbytes, 1), torch.uint8, w.packed.device, stream)
    cw = w.cstruct()
    _check(lib().affqmm_pack_rows(ctypes.byref(cw), rows.data_ptr(), _stream_ptr(stream)), "affqmm_pack_rows")
    return rows


def embed_rows_copy(w: PackedWeight, rows: torch.Tensor, ids: torch.Tensor, scale: float | None = None,
                    out: torch.Tensor | None = None, status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """embed_rows, reading the rows from `rows` = pack_rows(w) (the same values)."""
    T, out, sbits = _embed_args(w, ids, scale, out, stream)
    if not rows.is_cuda or rows.dtype != torch.uint8 or rows.numel() < rows_bytes(w.bits, w.group, w.N, w.K):
        raise ValueError("rows must be the uint8 CUDA copy made by pack_rows(w)")
    cw = w.cstruct()
    _check(lib().affqmm_embed_rows_copy(ctypes.byref(cw), rows.data_ptr(), ids.data_ptr(), T,
                                        0 if scale is None else 1, sbits, out.data_ptr(),
                                        _status_ptr(status, ids.get_device()), _stream_ptr(stream)),
           "affqmm_embed_rows_copy")
    return out


# ----------------------------------------------------------------------------- the paged key-value cache
PAGED_MAX_BATCH = 16384              # requests of a call
PAGED_MAX_TOKENS = 64                # query tokens of a request
_KV_TYPES = {torch.bfloat16: 0, torch.float8_e4m3fn: 1}
_BF16, _I32, _F32, _BOOL = torch.bfloat16, torch.int32, torch.float32, torch.bool
# affqmm_rows and affqmm_lanes as bytes: a small part of what a ctypes structure costs a call
_ROWS, _LANES = struct.Struct("Pqq").pack, struct.Struct("Pqqq").pack


def _check_ints(t: torch.Tensor, name: str, shape: tuple, device=None, dtype=torch.int32, contiguous=True):
    if (not t.is_cuda or t.dtype != dtype or tuple(t.shape) != shape or (contiguous and not t.is_contiguous())
            or (device is not None and t.device != device)):
        raise ValueError(f"{name} must be a{' contiguous' if contiguous else ''} CUDA {dtype} {list(shape)} tensor"
                         + (f" on {device}" if device is not None else ""))


def _unstepped(rc: int, *rows: torch.Tensor):
    """After a call was refused for a misaligned stride: its tensors with stride 0 for the axes of one, which are never
    stepped along and whose torch strides may be anything; None if that changes nothing."""
    if STATUS_NAMES.get(rc) != "AFFQMM_E_ALIGN":
        return None
    plain = [[s if n > 1 else 0 for s, n in zip(t.stride()[:-1], t.shape)] + [1] for t in rows]
    if all(list(t.stride()) == p for t, p in zip(rows, plain)):
        return None
    return [t.as_strided(t.shape, p) for t, p in zip(rows, plain)]


class KVCache:
    """A pool of pages of keys and values: k and v [pages, page, heads, dim],
    bf16 or float8_e4m3fn, with the values of a head contiguous and the other
    axes in any order in memory (a head-major pool is a transposed view).  For
    float8, k_scale and v_scale (float32 [heads], or None for 1) are what a
    head's stored values are multiplied by.  The object keeps the tensors'
    addresses: build it once per pool."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor | None = None,
                 v_scale: torch.Tensor | None = None):
        if k.dim() != 4 or k.shape != v.shape or k.dtype != v.dtype or k.stride() != v.stride() or k.device != v.device:
            raise ValueError("k and v must be [pages, page, heads, dim] tensors of one type, shape, stride and device")
        if k.dtype not in _KV_TYPES or not k.is_cuda:
            raise ValueError("k and v must be CUDA bf16 or float8_e4m3fn tensors")
        if k.stride(3) != 1 and k.shape[3] > 1:
            raise ValueError("the values of a head must be contiguous")
        for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
            if t is not None:
                if k.dtype != torch.float8_e4m3fn:
                    raise ValueError(f"{name} belongs to a float8 cache")
                _check_ints(t, name, (k.shape[2],), k.device, torch.float32)
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.pages, self.page, self.heads, self.dim = k.shape
        self.device, self._dev = k.device, k.get_device()
        self._c = CCache(_KV_TYPES[k.dtype], self.page, self.heads, self.dim, self.pages, *k.stride()[:3],
                         k.data_ptr() if k.numel() else None, v.data_ptr() if v.numel() else None,
                         k_scale.data_ptr() if k_scale is not None else None,
                         v_scale.data_ptr() if v_scale is not None else None)
        self._ref = ctypes.addressof(self._c)
        self._ws: dict = {}          # (tokens, query heads) -> workspace bytes

    @classmethod
    def empty(cls, pages: int, page: int, heads: int, dim: int, dtype=torch.bfloat16, device="cuda", k_scale=None,
              v_scale=None) -> "KVCache":
        k, v = (torch.empty(pages, page, heads, dim, dtype=dtype, device=device) for _ in "kv")
        return cls(k, v, k_scale, v_scale)


class Rope:
    """Rotary positions: `turns` int64 [rotary / 2], pair i's turns a position
    as a 64-bit fraction of a turn (rope_turns makes them), and `axis` uint8
    [rotary / 2] or None, the axis of positions by which each pair turns (one
    beyond the positions' axes: the last, so that with [tokens] positions a
    rope of several axes turns every pair by them).
    neighbour=False pairs values i and i + rotary / 2, True 2i and 2i + 1."""

    def __init__(self, turns: torch.Tensor, axis: torch.Tensor | None = None, neighbour: bool = False):
        if turns.dim() != 1:
            raise ValueError("turns must be one-dimensional")
        _check_ints(turns, "turns", tuple(turns.shape), dtype=torch.int64)
        if axis is not None:
            _check_ints(axis, "axis", tuple(turns.shape), turns.device, torch.uint8)
        self.turns, self.axis, self.neighbour, self.device = turns, axis, bool(neighbour), turns.device
        self.rotary, self._dev = 2 * turns.numel(), turns.get_device()
        self._c: dict = {}           # axes of the positions -> the C view

    def cstruct(self, axes: int) -> int:
        """The address of the C view for positions of `axes` axes."""
        c = self._c.get(axes)
        if c is None:
            c = self._c[axes] = CRope(self.turns.data_ptr() if self.rotary else None,
                                      self.axis.data_ptr() if self.axis is not None else None, self.rotary,
                                      int(self.neighbour), axes)
        return ctypes.addressof(c)


def rope_turns(frequencies, device="cuda") -> torch.Tensor:
    """turns of a Rope from its frequencies in radians a position (a sequence
    or float64 tensor: base ** (-2i / rotary), scaled as the model scales it;
    0 for a pair that does not turn)."""
    f = torch.as_tensor(frequencies, dtype=torch.float64, device="cpu") / (2 * math.pi)
    whole = torch.floor((f - torch.floor(f)) * 2.0 ** 64).tolist()
    wrapped = [int(x) % (1 << 64) for x in whole]
    return torch.tensor([x - (1 << 64) if x >> 63 else x for x in wrapped], dtype=torch.int64, device=device)


class PagedStep:
    """What paged_plan writes: starts int32 [batch + 1], lens int32 [batch],
    ring_state int32 [2], slots / positions / requests int32 [capacity] and
    status int32 [1].  Build one (PagedStep.empty) and use it again: a captured
    step reads the same addresses every time."""

    def __init__(self, starts, lens, ring_state, slots, positions, requests, status):
        batch, capacity, device = lens.numel(), slots.numel(), lens.device
        _check_ints(starts, "starts", (batch + 1,), device)
        _check_ints(lens, "lens", (batch,))
        _check_ints(ring_state, "ring_state", (2,), device)
        for t, name in ((slots, "slots"), (positions, "positions"), (requests, "requests")):
            _check_ints(t, name, (capacity,), device)
        _check_ints(status, "status", (1,), device)
        self.starts, self.lens, self.ring_state, self.status = starts, lens, ring_state, status
        self.slots, self.positions, self.requests = slots, positions, requests
        self.batch, self.capacity, self.device, self._dev = batch, capacity, device, lens.get_device()
        ptr = lambda t: t.data_ptr() if t.numel() else None  # noqa: E731
        self._c = CStep(capacity, *[ptr(t) for t in (starts, lens, ring_state, slots, positions, requests, status)])
        self._ref = ctypes.addressof(self._c)

    @classmethod
    def empty(cls, batch: int, capacity: int, device="cuda") -> "PagedStep":
        make = lambda n: torch.empty(n, dtype=torch.int32, device=device)  # noqa: E731
        return cls(make(batch + 1), make(batch), make(2), make(capacity), make(capacity), make(capacity), make(1))


def paged_plan(lens: torch.Tensor, fresh: torch.Tensor, finished: torch.Tensor | None, table: torch.Tensor,
               ring: torch.Tensor, ring_state: torch.Tensor, page: int, out: PagedStep, stream=None) -> PagedStep:
    """affqmm_paged_plan: a step's block tables, slot maps, positions and
    lengths.  lens, fresh int32 [batch]; finished bool [batch] or None; table
    int32 [batch, wide] (rows may be strided), written where the step takes
    pages; ring int32 [pool] of free pages, ring_state int32 [2] its head and
    count.  out.lens and out.ring_state are the next step's lens and
    ring_state; they must be other tensors than this step's."""
    dev = out._dev
    shape, tshape, tstride = lens.shape, table.shape, table.stride()
    batch = out.batch
    if not (shape == (batch,) == fresh.shape and len(tshape) == 2 and tshape[0] == batch and ring.dim() == 1
            and ring_state.shape == (2,) and lens.dtype is fresh.dtype is table.dtype is ring.dtype is ring_state.dtype is _I32
            and lens.get_device() == fresh.get_device() == table.get_device() == ring.get_device()
            == ring_state.get_device() == dev
            and lens.is_contiguous() and fresh.is_contiguous() and ring.is_contiguous() and ring_state.is_contiguous()
            and (tstride[1] == 1 or tshape[1] <= 1)
            and (finished is None or (finished.dtype is _BOOL and finished.shape == shape
                                      and finished.get_device() == dev and finished.is_contiguous()))):
        raise ValueError(f"paged_plan wants contiguous CUDA int32 lens and fresh [{batch}] (the requests of out), ring "
                         f"[pool] and ring_state [2], table [{batch}, wide] with contiguous rows, and bool finished "
                         f"[{batch}] or None, all on {out.device}")
    _check((_lib or lib()).affqmm_paged_plan(
        batch, lens.data_ptr(), fresh.data_ptr(), finished.data_ptr() if finished is not None else None,
        table.data_ptr(), tstride[0], tshape[1], ring.data_ptr(), ring.shape[0], ring_state.data_ptr(), page, out._ref,
        _stream_ptr(stream, dev)), "affqmm_paged_plan")
    return out


def rope_append(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, positions: torch.Tensor, slots: torch.Tensor,
                rope: Rope, cache: KVCache, out: torch.Tensor | None = None, status: torch.Tensor | None = None,
                stream=None) -> torch.Tensor:
    """affqmm_rope_append: rotary positions on q and k, and k and v written to
    their slots of the cache.  q [tokens, query heads, dim], k and v [tokens,
    cache heads, dim], bf16, token and head strides multiples of 8 (views of the
    stacked projection's output serve); positions int32 [tokens] or [axes,
    tokens]; slots int32 [tokens], -1 for a token that is not kept.  Returns q turned,
    in `out` (which may be q)."""
    dev, dim = cache._dev, cache.dim
    shape, kshape, pshape = q.shape, k.shape, positions.shape
    if len(shape) != 3:
        raise ValueError("q must be [tokens, query heads, dim]")
    T = shape[0]
    if out is None:
        out = _empty(shape, _BF16, cache.device, stream)
    sq, sk, sv, so, sp = q.stride(), k.stride(), v.stride(), out.stride(), positions.stride()
    if not (shape[2] == dim and out.shape == shape and kshape == (T, cache.heads, dim) == v.shape
            and q.dtype is k.dtype is v.dtype is out.dtype is _BF16 and sq[2] == sk[2] == sv[2] == so[2] == 1
            and q.get_device() == k.get_device() == v.get_device() == out.get_device() == positions.get_device()
            == slots.get_device() == rope._dev == dev
            and positions.dtype is slots.dtype is _I32 and len(pshape) in (1, 2) and pshape[-1] == T
            and (sp[-1] == 1 or T <= 1) and slots.shape == (T,) and slots.is_contiguous()):
        raise ValueError(f"rope_append wants CUDA bf16 q and out [tokens, query heads, {dim}], k and v [tokens, "
                         f"{cache.heads}, {dim}], the values of a head contiguous, int32 positions [tokens] or [axes, "
                         f"tokens] and slots [tokens], and the rope, all on {cache.device}")
    if T == 0:
        return out
    axes = pshape[0] if len(pshape) == 2 else 1
    rc = (_lib or lib()).affqmm_rope_append(
        cache._ref, rope.cstruct(axes), _ROWS(q.data_ptr(), sq[0], sq[1]), _ROWS(k.data_ptr(), sk[0], sk[1]),
        _ROWS(v.data_ptr(), sv[0], sv[1]), _ROWS(out.data_ptr(), so[0], so[1]), T, shape[1], positions.data_ptr(),
        sp[0] if axes > 1 else 0, slots.data_ptr(), _status_ptr(status, dev),
        _stream_ptr(stream, dev))
    if rc:
        rows = _unstepped(rc, q, k, v, out)
        if rows is None:
            raise AffqmmError(rc, "affqmm_rope_append")
        rope_append(*rows[:3], positions, slots, rope, cache, rows[3], status, stream)
    return out


def paged_attention_workspace_bytes(cache: KVCache, tokens: int, heads: int) -> int:
    need = cache._ws.get((tokens, heads))
    if need is None:
        got = ctypes.c_size_t(0)
        with torch.cuda.device(cache.device):
            _check(lib().affqmm_paged_attention_workspace_bytes(cache._ref, tokens, heads, ctypes.byref(got)),
                   "affqmm_paged_attention_workspace_bytes")
        need = cache._ws[(tokens, heads)] = got.value
    return need


def paged_attention(q: torch.Tensor, cache: KVCache, table: torch.Tensor, lens: torch.Tensor, scale: float | None = None,
                    window: int = 0, out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                    status: torch.Tensor | None = None, workspace: Workspace | None = None, stream=None) -> torch.Tensor:
    """affqmm_paged_attention: each request's newest tokens against its pages.
    q bf16 [batch, query heads, dim] (one new token) or [batch, tokens, query
    heads, dim], strides multiples of 8; table int32 [batch, wide]; lens int32 [batch], the
    step's own tokens included; scale defaults to dim ** -0.5; window > 0 keeps
    the last `window` keys of each token.  `lse` (float32, q's shape without its
    last axis) gets the log of each row's sum of exponentials.  Returns `out`,
    of q's shape."""
    dev, dim, shape = cache._dev, cache.dim, q.shape
    if len(shape) == 4:
        batch, tokens, heads, d = shape
    elif len(shape) == 3:
        (batch, heads, d), tokens = shape, 1
    else:
        raise ValueError("q must be [batch, query heads, dim] or [batch, tokens, query heads, dim]")
    if not -1 << 31 <= window < 1 << 31:         # the ABI's int; ctypes would drop the upper bits
        raise ValueError("window must fit 32 bits")
    if out is None:
        out = _empty(shape, _BF16, cache.device, stream)
    sq, so, st, tshape = q.stride(), out.stride(), table.stride(), table.shape
    if not (d == dim and out.shape == shape and q.dtype is out.dtype is _BF16 and sq[-1] == so[-1] == 1
            and q.get_device() == out.get_device() == table.get_device() == lens.get_device() == dev
            and table.dtype is lens.dtype is _I32 and len(tshape) == 2 and tshape[0] == batch
            and (st[1] == 1 or tshape[1] <= 1) and lens.shape == (batch,) and lens.is_contiguous()
            and (lse is None or (lse.dtype is _F32 and lse.shape == shape[:-1] and lse.get_device() == dev
                                 and lse.is_contiguous()))):
        raise ValueError(f"paged_attention wants CUDA bf16 q and out of one shape, {dim} contiguous values a head, int32 "
                         f"table [{batch}, wide] with contiguous rows and lens [{batch}], and float32 lse {list(shape[:-1])} "
                         f"or None, all on {cache.device}")
    sp = _stream_ptr(stream, dev)
    buf = (workspace or default_workspace(dev, sp)).get(
        cache._ws.get((tokens, heads)) or paged_attention_workspace_bytes(cache, tokens, heads), stream)
    rc = (_lib or lib()).affqmm_paged_attention(
        cache._ref, _LANES(q.data_ptr(), sq[0], sq[-3], sq[-2]), _LANES(out.data_ptr(), so[0], so[-3], so[-2]),
        lse.data_ptr() if lse is not None else None, batch, tokens, heads, table.data_ptr(), st[0], tshape[1],
        lens.data_ptr(), dim ** -0.5 if scale is None else scale, window,
        _status_ptr(status, dev), buf.data_ptr(), buf.numel(), sp)
    if rc:
        lanes = _unstepped(rc, q, out)
        if lanes is None:
            raise AffqmmError(rc, "affqmm_paged_attention")
        paged_attention(lanes[0], cache, table, lens, scale, window, lanes[1], lse, status, workspace, stream)
    return out
