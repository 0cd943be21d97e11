"""ctypes binding of libtwell.so: argument marshalling only.

Torch tensors supply device memory (``data_ptr()``) and the stream
(``torch.cuda.current_stream().cuda_stream``); every step of the layer runs in
the library's HIP kernels. There is no fallback: if the library is missing
the calls raise.
"""
from __future__ import annotations

import ctypes
import os
import struct
from dataclasses import dataclass

import torch

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libtwell.so")

TWELL_F32, TWELL_BF16 = 0, 1
TILE_C = 128
DEV_TILE_OVERFLOW, DEV_OVF_CAPACITY, DEV_BAD_INDEX = 1, 2, 4

# every extern "C" symbol include/twell.h declares
EXPORTS = ("twell_gate_pack", "twell_gate_workspace_bytes", "twell_ffn_fwd", "twell_fwd_workspace_bytes", "twell_decode_fwd",
           "twell_decode_workspace_bytes", "twell_to_hybrid", "hybrid_ffn_fwd",
           "hybrid_fwd_workspace_bytes", "hybrid_ffn_bwd", "hybrid_bwd_workspace_bytes",
           "twell_status_str", "twell_decode_fwd_noalloc", "twell_rmsnorm_fwd",
           "twell_rmsnorm_bwd", "twell_rmsnorm_bwd_workspace_bytes", "twell_fp8_quant",
           "twell_fp8_matmul", "twell_fp8_matmul_workspace_bytes", "twell_fp4_quant",
           "twell_fp4_dequant", "twell_fp4_matmul", "twell_fp4_matmul_workspace_bytes",
           "twell_fp4_matmul_dx", "twell_fp4_matmul_dx_workspace_bytes", "twell_fp4_decode_fwd",
           "twell_fp4_decode_workspace_bytes")
STATIC_SCRATCH_BYTES = 12 << 20  # twell_decode_fwd_noalloc's scratch per GPU
DECODE_T = 64  # most tokens twell_decode_fwd takes (few-token kernels up to here)
FP8_BLOCK = 128  # columns that share a scale of an 8-bit matrix
FP4_BLOCK = 128  # columns that a row of a 4-bit matrix is padded to
FP4_GROUPS = (32, 64, 128)  # columns that may share a scale of a 4-bit matrix
NORM_COLS = 16384  # widest row the norm takes
SUMS_F32, SUMS_FP8 = 0, 1  # how twell_fp8_matmul adds products
E_WORKSPACE = -5  # status: the call needs (more) workspace

c_i32, c_sz, c_p = ctypes.c_int32, ctypes.c_size_t, ctypes.c_void_p


class TwellC(ctypes.Structure):
    _fields_ = [("T", c_i32), ("d_ff", c_i32), ("width", c_i32), ("dtype", ctypes.c_int),
                ("count", c_p), ("col", c_p), ("val", c_p)]


TIMING_MAX = 24


class TimingC(ctypes.Structure):
    _fields_ = [("events", c_p * (TIMING_MAX + 1)), ("n_events", c_i32), ("n_used", c_i32),
                ("names", ctypes.c_char_p * TIMING_MAX)]


class KernelTimer:
    """Per-kernel HIP-event timing of library calls on the current stream.

    ``timer.arg()`` gives the struct to pass to one call; after the stream is
    synchronised, ``timer.collect()`` returns [(kernel name, ms), ...] of the
    last call and ``timer.add(totals)`` accumulates them into a dict.
    """

    def __init__(self):
        self.ev = [torch.cuda.Event(enable_timing=True) for _ in range(TIMING_MAX + 1)]
        for e in self.ev:  # materialise the underlying events
            e.record()
        torch.cuda.synchronize()
        self.c = TimingC()
        for k, e in enumerate(self.ev):
            self.c.events[k] = e.cuda_event
        self.c.n_events = TIMING_MAX + 1

    def arg(self):
        return ctypes.byref(self.c)

    def collect(self):
        out = []
        for k in range(self.c.n_used - 1):
            out.append((self.c.names[k].decode(), self.ev[k].elapsed_time(self.ev[k + 1])))
        return out

    def add(self, totals: dict):
        for name, ms in self.collect():
            totals[name] = totals.get(name, 0.0) + ms


class HybridC(ctypes.Structure):
    _fields_ = [("T", c_i32), ("d_ff", c_i32), ("K", c_i32), ("max_ovf", c_i32),
                ("dtype", ctypes.c_int), ("row_nnz", c_p), ("row_slot", c_p), ("ell_col", c_p),
                ("ell_val", c_p), ("ovf_rows", c_p), ("dense", c_p), ("n_ovf", c_p)]


class MatC(ctypes.Structure):
    _fields_ = [("rows", c_i32), ("cols", c_i32), ("ld", ctypes.c_int64),
                ("dtype", ctypes.c_int), ("data", c_p)]


class Fp8C(ctypes.Structure):
    _fields_ = [("rows", c_i32), ("cols", c_i32), ("block_rows", c_i32), ("q", c_p),
                ("scale", c_p)]


class Fp4C(ctypes.Structure):
    _fields_ = [("rows", c_i32), ("cols", c_i32), ("group", c_i32), ("q", c_p), ("scale", c_p)]


_lib = None


class TwellError(RuntimeError):
    pass


def load() -> ctypes.CDLL:
    """Load libtwell.so (built by __graft_entry__.build()); raise if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise TwellError(f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                         "(the HIP library is the only implementation; there is no fallback)")
    L = ctypes.CDLL(LIB_PATH)
    P, I, S = c_p, c_i32, c_sz
    L.twell_gate_pack.argtypes = [ctypes.c_int, P, P, I, I, ctypes.POINTER(TwellC), P, S, P, P,
                                  P]
    L.twell_gate_workspace_bytes.argtypes = [ctypes.c_int, I, I, I]
    L.twell_gate_workspace_bytes.restype = S
    L.twell_ffn_fwd.argtypes = [ctypes.c_int, P, ctypes.POINTER(TwellC), P, P, I, P, P, S, P, P,
                                P]
    L.twell_fwd_workspace_bytes.argtypes = [ctypes.c_int, I, I, I, I]
    L.twell_fwd_workspace_bytes.restype = S
    L.twell_decode_fwd.argtypes = [ctypes.c_int, P, P, P, P, I, ctypes.POINTER(TwellC), P, P,
                                   S, P, P, P]
    L.twell_decode_fwd_noalloc.argtypes = [ctypes.c_int, P, P, P, P, I,
                                           ctypes.POINTER(TwellC), P, P, P, P]
    L.twell_decode_workspace_bytes.argtypes = [ctypes.c_int, I, I, I, I]
    L.twell_decode_workspace_bytes.restype = S
    L.twell_to_hybrid.argtypes = [ctypes.POINTER(TwellC), ctypes.POINTER(HybridC), P, P, P]
    L.hybrid_ffn_bwd.argtypes = [ctypes.c_int, P, P, ctypes.POINTER(HybridC), P, P, P, I,
                                 ctypes.c_float, P, P, P, P, P, S, P, P, P]
    L.hybrid_ffn_fwd.argtypes = [ctypes.c_int, P, ctypes.POINTER(HybridC), P, P, I, P, P, S, P,
                                 P, P]
    L.hybrid_fwd_workspace_bytes.argtypes = [ctypes.c_int, I, I, I, I, I]
    L.hybrid_fwd_workspace_bytes.restype = S
    L.hybrid_bwd_workspace_bytes.argtypes = [ctypes.c_int, I, I, I, I, I]
    L.hybrid_bwd_workspace_bytes.restype = S
    M, Q, F = P, P, ctypes.c_float  # structures as packed bytes (_pack_mat, _pack_fp8)
    L.twell_rmsnorm_fwd.argtypes = [M, M, P, ctypes.c_int, F, M, M, Q, P, P]
    L.twell_rmsnorm_bwd.argtypes = [M, M, P, ctypes.c_int, F, M, M, P, P, S, P, P]
    L.twell_rmsnorm_bwd_workspace_bytes.argtypes = [I, I]
    L.twell_rmsnorm_bwd_workspace_bytes.restype = S
    L.twell_fp8_quant.argtypes = [M, Q, Q, P, P]
    L.twell_fp8_matmul.argtypes = [Q, Q, M, I, P, S, P, P]
    L.twell_fp8_matmul_workspace_bytes.argtypes = [I, I, I]
    L.twell_fp8_matmul_workspace_bytes.restype = S
    L.twell_fp4_quant.argtypes = [M, Q, P, P]
    L.twell_fp4_dequant.argtypes = [Q, M, P, P]
    for f in ("twell_fp4_matmul", "twell_fp4_matmul_dx"):
        getattr(L, f).argtypes = [M, Q, M, P, S, P, P]
        getattr(L, f).restype = ctypes.c_int
        getattr(L, f + "_workspace_bytes").argtypes = [ctypes.c_int, I, I, I]
        getattr(L, f + "_workspace_bytes").restype = S
    L.twell_fp4_decode_fwd.argtypes = [M, Q, Q, Q, P, P, S, P, P]
    L.twell_fp4_decode_workspace_bytes.argtypes = [ctypes.c_int, I, I, I]
    L.twell_fp4_decode_workspace_bytes.restype = S
    L.twell_status_str.argtypes = [ctypes.c_int]
    L.twell_status_str.restype = ctypes.c_char_p
    for f in ("twell_gate_pack", "twell_ffn_fwd", "twell_decode_fwd", "twell_to_hybrid",
              "hybrid_ffn_fwd", "hybrid_ffn_bwd", "twell_decode_fwd_noalloc", "twell_rmsnorm_fwd",
              "twell_rmsnorm_bwd", "twell_fp8_quant", "twell_fp8_matmul", "twell_fp4_quant",
              "twell_fp4_dequant", "twell_fp4_decode_fwd"):
        getattr(L, f).restype = ctypes.c_int
    _lib = L
    return L


def _check(rc: int, what: str):
    if rc != 0:
        raise TwellError(f"{what}: {load().twell_status_str(rc).decode()} (status {rc})")


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return TWELL_BF16
    if t.dtype == torch.float32:
        return TWELL_F32
    raise TwellError(f"unsupported dtype {t.dtype}")


def _ptr(t):
    return None if t is None else c_p(t.data_ptr())


# ---- argument checks: the C-ABI sees only pointers, so every tensor's shape,
# dtype, layout and device is checked here, before any call reaches the GPU
def _req(t, name, shape, dtype, device=None):
    """t must be a contiguous tensor of `shape` and `dtype` (on `device` if
    given); raises TwellError otherwise."""
    if not isinstance(t, torch.Tensor):
        raise TwellError(f"{name}: expected a tensor, got {type(t).__name__}")
    if tuple(t.shape) != tuple(shape):
        raise TwellError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise TwellError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if not t.is_contiguous():
        raise TwellError(f"{name}: must be contiguous (row-major), e.g. not a transposed view")
    if device is not None and t.device != torch.device(device):
        raise TwellError(f"{name}: on {t.device}, expected {device}")


def _ws_form(workspace):
    if workspace is not None and (not isinstance(workspace, torch.Tensor)
                                  or workspace.dtype != torch.uint8 or workspace.dim() != 1
                                  or not workspace.is_contiguous()):
        raise TwellError("workspace: expected a contiguous 1-D uint8 tensor")


def _on_gpu(*named):
    """Every given tensor lives on one GPU; returns that device. (The
    workspace's form is checked first: it is the one argument whose shape the
    other checks do not cover.)"""
    for name, t in named:
        if name == "workspace":
            _ws_form(t)
    dev = None
    for name, t in named:
        if t is None:
            continue
        if t.device.type != "cuda":
            raise TwellError(f"{name}: on {t.device}; the library runs on the GPU only")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise TwellError(f"{name}: on {t.device}, other arguments on {dev}")
    return dev


def _ws(workspace, need, device):
    """The caller's workspace, checked, or a new one of `need` bytes."""
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=device) if need else None
    _ws_form(workspace)
    if workspace.numel() < need:
        raise TwellError(f"workspace: {workspace.numel()} bytes, need {need}")
    return workspace


def _status(status, device):
    if status is not None:
        _req(status, "status", (1,), torch.int32)
    return status


def _check_weights(d_ff, d_model, dtype, **w):
    for name, t in w.items():
        _req(t, name, (d_ff, d_model), dtype)


def _check_twell(tw, T, dtype):
    if not isinstance(tw, Twell):
        raise TwellError("expected a Twell")
    nt = tw.count.shape[1] if tw.count.dim() == 2 else -1
    if tw.count.dim() != 2 or tw.col.dim() != 3:
        raise TwellError("twell: count must be [T][d_ff/128], col/val [T][d_ff/128][width]")
    W = tw.col.shape[2]
    _req(tw.count, "twell.count", (T, nt), torch.int32)
    _req(tw.col, "twell.col", (T, nt, W), torch.int16)
    _req(tw.val, "twell.val", (T, nt, W), dtype)


def _check_hybrid(hy, T, dtype):
    if not isinstance(hy, Hybrid):
        raise TwellError("expected a Hybrid")
    if hy.ell_col.dim() != 2 or hy.dense.dim() != 2:
        raise TwellError("hybrid: ell_col/ell_val must be [T][K], dense [max_ovf][d_ff]")
    K, mo, dff = hy.ell_col.shape[1], hy.dense.shape[0], hy.dense.shape[1]
    _req(hy.row_nnz, "hybrid.row_nnz", (T,), torch.int32)
    _req(hy.row_slot, "hybrid.row_slot", (T,), torch.int32)
    _req(hy.ell_col, "hybrid.ell_col", (T, K), torch.int16)
    _req(hy.ell_val, "hybrid.ell_val", (T, K), dtype)
    _req(hy.ovf_rows, "hybrid.ovf_rows", (mo,), torch.int32)
    _req(hy.dense, "hybrid.dense", (mo, dff), dtype)
    _req(hy.n_ovf, "hybrid.n_ovf", (1,), torch.int32)


def _twell_tensors(tw):
    return [("twell.count", tw.count), ("twell.col", tw.col), ("twell.val", tw.val)]


def _hybrid_tensors(hy):
    return [("hybrid.row_nnz", hy.row_nnz), ("hybrid.row_slot", hy.row_slot),
            ("hybrid.ell_col", hy.ell_col), ("hybrid.ell_val", hy.ell_val),
            ("hybrid.ovf_rows", hy.ovf_rows), ("hybrid.dense", hy.dense),
            ("hybrid.n_ovf", hy.n_ovf)]


def _x2(x, name="x"):
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise TwellError(f"{name}: expected a [T][d_model] tensor")
    _dt(x)
    return x.shape


def _stream(device) -> c_p:
    return c_p(torch.cuda.current_stream(device).cuda_stream)


# the same stream's handle for a device's number, without building a Stream
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


@dataclass
class Twell:
    """TwELL arrays (device tensors) of h = ReLU(x W_g)."""

    count: torch.Tensor  # [T][d_ff/128] int32
    col: torch.Tensor    # [T][d_ff/128][width] int16
    val: torch.Tensor    # [T][d_ff/128][width] dtype

    @property
    def T(self):
        return self.count.shape[0]

    @property
    def d_ff(self):
        return self.count.shape[1] * TILE_C

    @property
    def width(self):
        return self.col.shape[2]

    def c(self) -> TwellC:
        return TwellC(self.T, self.d_ff, self.width, _dt(self.val), self.count.data_ptr(),
                      self.col.data_ptr(), self.val.data_ptr())


@dataclass
class Hybrid:
    """Hybrid ELL + dense-backup arrays (device tensors)."""

    row_nnz: torch.Tensor   # [T] int32
    row_slot: torch.Tensor  # [T] int32
    ell_col: torch.Tensor   # [T][K] int16
    ell_val: torch.Tensor   # [T][K] dtype
    ovf_rows: torch.Tensor  # [max_ovf] int32
    dense: torch.Tensor     # [max_ovf][d_ff] dtype
    n_ovf: torch.Tensor     # [1] int32

    @property
    def T(self):
        return self.row_nnz.shape[0]

    @property
    def K(self):
        return self.ell_col.shape[1]

    @property
    def max_ovf(self):
        return self.dense.shape[0]

    @property
    def d_ff(self):
        return self.dense.shape[1]

    def c(self) -> HybridC:
        return HybridC(self.T, self.d_ff, self.K, self.max_ovf, _dt(self.ell_val),
                       self.row_nnz.data_ptr(), self.row_slot.data_ptr(),
                       self.ell_col.data_ptr(), self.ell_val.data_ptr(),
                       self.ovf_rows.data_ptr(), self.dense.data_ptr(), self.n_ovf.data_ptr())


def empty_twell(T, d_ff, width, dtype, device) -> Twell:
    nt = d_ff // TILE_C
    return Twell(torch.empty((T, nt), dtype=torch.int32, device=device),
                 torch.empty((T, nt, width), dtype=torch.int16, device=device),
                 torch.empty((T, nt, width), dtype=dtype, device=device))


def empty_hybrid(T, d_ff, K, max_ovf, dtype, device) -> Hybrid:
    return Hybrid(torch.empty(T, dtype=torch.int32, device=device),
                  torch.empty(T, dtype=torch.int32, device=device),
                  torch.empty((T, K), dtype=torch.int16, device=device),
                  torch.empty((T, K), dtype=dtype, device=device),
                  torch.empty(max_ovf, dtype=torch.int32, device=device),
                  torch.empty((max_ovf, d_ff), dtype=dtype, device=device),
                  torch.zeros(1, dtype=torch.int32, device=device))


def _timing(t):
    return None if t is None else t.arg()


def gate_workspace_bytes(dtype, T, d_model, d_ff) -> int:
    return int(load().twell_gate_workspace_bytes(dtype, T, d_model, d_ff))


def gate_pack(x, wg_t, width=TILE_C, out: Twell | None = None, status=None,
              timing: KernelTimer | None = None, workspace=None) -> Twell:
    T, dm = _x2(x)
    _req(x, "x", (T, dm), x.dtype)
    if not isinstance(wg_t, torch.Tensor) or wg_t.dim() != 2:
        raise TwellError("wg_t: expected a [d_ff][d_model] tensor")
    d_ff = wg_t.shape[0]
    _req(wg_t, "wg_t", (d_ff, dm), x.dtype)
    if out is None:
        out = empty_twell(T, d_ff, width, x.dtype, x.device)
    _check_twell(out, T, x.dtype)
    if out.d_ff != d_ff:
        raise TwellError(f"out: d_ff {out.d_ff}, wg_t has {d_ff} rows")
    dev = _on_gpu(("x", x), ("wg_t", wg_t), *_twell_tensors(out), ("status", status),
                  ("workspace", workspace))
    _status(status, dev)
    need = gate_workspace_bytes(_dt(x), T, dm, d_ff)
    workspace = _ws(workspace, need, dev)
    nbytes = 0 if workspace is None else workspace.numel()
    c = out.c()
    _check(load().twell_gate_pack(_dt(x), _ptr(x), _ptr(wg_t), T, dm, ctypes.byref(c),
                                  _ptr(workspace), nbytes, _ptr(status), _timing(timing),
                                  _stream(x.device)), "twell_gate_pack")
    return out


def fwd_workspace_bytes(dtype, T, d_model, d_ff, width) -> int:
    return int(load().twell_fwd_workspace_bytes(dtype, T, d_model, d_ff, width))


def ffn_fwd(x, tw: Twell, wu_t, wd, y=None, workspace=None, status=None,
            timing: KernelTimer | None = None):
    T, dm = _x2(x)
    _req(x, "x", (T, dm), x.dtype)
    _check_twell(tw, T, x.dtype)
    _check_weights(tw.d_ff, dm, x.dtype, wu_t=wu_t, wd=wd)
    if y is None:
        y = torch.empty((T, dm), dtype=torch.float32, device=x.device)
    _req(y, "y", (T, dm), torch.float32)
    dev = _on_gpu(("x", x), *_twell_tensors(tw), ("wu_t", wu_t), ("wd", wd), ("y", y),
                  ("status", status), ("workspace", workspace))
    _status(status, dev)
    need = fwd_workspace_bytes(_dt(x), T, dm, tw.d_ff, tw.width)
    workspace = _ws(workspace, need, dev)
    nbytes = 0 if workspace is None else workspace.numel()
    c = tw.c()
    _check(load().twell_ffn_fwd(_dt(x), _ptr(x), ctypes.byref(c), _ptr(wu_t), _ptr(wd), dm,
                                _ptr(y), _ptr(workspace), nbytes, _ptr(status),
                                _timing(timing), _stream(x.device)), "twell_ffn_fwd")
    return y


def decode_workspace_bytes(dtype, T, d_model, d_ff, width) -> int:
    return int(load().twell_decode_workspace_bytes(dtype, T, d_model, d_ff, width))


def decode_fwd(x, wg_t, wu_t, wd, width=TILE_C, out: Twell | None = None, y=None,
               workspace=None, status=None, timing: KernelTimer | None = None):
    """The whole layer for T <= DECODE_T tokens in one call (three launches
    on the current stream); returns (TwELL of h, y float32)."""
    T, dm = _x2(x)
    _req(x, "x", (T, dm), x.dtype)
    if not isinstance(wg_t, torch.Tensor) or wg_t.dim() != 2:
        raise TwellError("wg_t: expected a [d_ff][d_model] tensor")
    d_ff = wg_t.shape[0]
    _check_weights(d_ff, dm, x.dtype, wg_t=wg_t, wu_t=wu_t, wd=wd)
    if T > DECODE_T:
        raise TwellError(f"decode_fwd takes at most {DECODE_T} tokens, got {T}")
    if out is None:
        out = empty_twell(T, d_ff, width, x.dtype, x.device)
    _check_twell(out, T, x.dtype)
    if out.d_ff != d_ff:
        raise TwellError(f"out: d_ff {out.d_ff}, wg_t has {d_ff} rows")
    if y is None:
        y = torch.empty((T, dm), dtype=torch.float32, device=x.device)
    _req(y, "y", (T, dm), torch.float32)
    dev = _on_gpu(("x", x), ("wg_t", wg_t), ("wu_t", wu_t), ("wd", wd), *_twell_tensors(out),
                  ("y", y), ("status", status), ("workspace", workspace))
    _status(status, dev)
    need = decode_workspace_bytes(_dt(x), T, dm, d_ff, out.width)
    workspace = _ws(workspace, need, dev)
    nbytes = 0 if workspace is None else workspace.numel()
    c = out.c()
    _check(load().twell_decode_fwd(_dt(x), _ptr(x), _ptr(wg_t), _ptr(wu_t), _ptr(wd), dm,
                                   ctypes.byref(c), _ptr(y), _ptr(workspace), nbytes,
                                   _ptr(status), _timing(timing), _stream(x.device)),
           "twell_decode_fwd")
    return out, y


def decode_fwd_noalloc(x, wg_t, wu_t, wd, out: Twell, y, status=None,
                       timing: KernelTimer | None = None):
    """decode_fwd for callers that cannot allocate: the caller passes the
    outputs (out, y), the library's static per-GPU scratch replaces the
    workspace, and nothing is allocated. Overlapping calls on one GPU race."""
    T, dm = _x2(x)
    _req(x, "x", (T, dm), x.dtype)
    if not isinstance(wg_t, torch.Tensor) or wg_t.dim() != 2:
        raise TwellError("wg_t: expected a [d_ff][d_model] tensor")
    d_ff = wg_t.shape[0]
    _check_weights(d_ff, dm, x.dtype, wg_t=wg_t, wu_t=wu_t, wd=wd)
    if T > DECODE_T:
        raise TwellError(f"decode_fwd_noalloc takes at most {DECODE_T} tokens, got {T}")
    _check_twell(out, T, x.dtype)
    if out.d_ff != d_ff:
        raise TwellError(f"out: d_ff {out.d_ff}, wg_t has {d_ff} rows")
    _req(y, "y", (T, dm), torch.float32)
    dev = _on_gpu(("x", x), ("wg_t", wg_t), ("wu_t", wu_t), ("wd", wd), *_twell_tensors(out),
                  ("y", y), ("status", status))
    _status(status, dev)
    c = out.c()
    _check(load().twell_decode_fwd_noalloc(_dt(x), _ptr(x), _ptr(wg_t), _ptr(wu_t), _ptr(wd), dm,
                                           ctypes.byref(c), _ptr(y), _ptr(status),
                                           _timing(timing), _stream(x.device)),
           "twell_decode_fwd_noalloc")
    return out, y


def to_hybrid(tw: Twell, K, max_ovf, out: Hybrid | None = None, status=None,
              timing: KernelTimer | None = None) -> Hybrid:
    if not isinstance(tw, Twell):
        raise TwellError("expected a Twell")
    _check_twell(tw, tw.T, tw.val.dtype)
    _dt(tw.val)
    if out is None:
        out = empty_hybrid(tw.T, tw.d_ff, K, max_ovf, tw.val.dtype, tw.val.device)
    _check_hybrid(out, tw.T, tw.val.dtype)
    if (out.K, out.max_ovf, out.d_ff) != (K, max_ovf, tw.d_ff):
        raise TwellError(f"out: (K, max_ovf, d_ff) = {(out.K, out.max_ovf, out.d_ff)}, "
                         f"expected {(K, max_ovf, tw.d_ff)}")
    dev = _on_gpu(*_twell_tensors(tw), *_hybrid_tensors(out), ("status", status))
    _status(status, dev)
    ct, ch = tw.c(), out.c()
    _check(load().twell_to_hybrid(ctypes.byref(ct), ctypes.byref(ch), _ptr(status),
                                  _timing(timing), _stream(tw.val.device)), "twell_to_hybrid")
    return out


def hybrid_fwd_workspace_bytes(dtype, T, d_model, d_ff, K, max_ovf) -> int:
    return int(load().hybrid_fwd_workspace_bytes(dtype, T, d_model, d_ff, K, max_ovf))


def hybrid_fwd(x, hy: Hybrid, wu_t, wd, y=None, workspace=None, status=None,
               timing: KernelTimer | None = None):
    """Training forward over a hybrid; returns y (float32)."""
    T, dm = _x2(x)
    _req(x, "x", (T, dm), x.dtype)
    _check_hybrid(hy, T, x.dtype)
    _check_weights(hy.d_ff, dm, x.dtype, wu_t=wu_t, wd=wd)
    if y is None:
        y = torch.empty((T, dm), dtype=torch.float32, device=x.device)
    _req(y, "y", (T, dm), torch.float32)
    dev = _on_gpu(("x", x), *_hybrid_tensors(hy), ("wu_t", wu_t), ("wd", wd), ("y", y),
                  ("status", status), ("workspace", workspace))
    _status(status, dev)
    need = hybrid_fwd_workspace_bytes(_dt(x), T, dm, hy.d_ff, hy.K, hy.max_ovf)
    workspace = _ws(workspace, need, dev)
    nbytes = 0 if workspace is None else workspace.numel()
    ch = hy.c()
    _check(load().hybrid_ffn_fwd(_dt(x), _ptr(x), ctypes.byref(ch), _ptr(wu_t), _ptr(wd), dm,
                                 _ptr(y), _ptr(workspace), nbytes, _ptr(status), _timing(timing),
                                 _stream(x.device)), "hybrid_ffn_fwd")
    return y


def bwd_workspace_bytes(dtype, T, d_model, d_ff, K, max_ovf) -> int:
    return int(load().hybrid_bwd_workspace_bytes(dtype, T, d_model, d_ff, K, max_ovf))


def ffn_bwd(x, dy, hy: Hybrid, wg_t, wu_t, wd, out=None, workspace=None, status=None,
            timing: KernelTimer | None = None, l1: float = 0.0):
    """Returns (dx, dwg_t, dwu_t, dwd), all float32; l1 weights an activation
    penalty l1 * sum(h) whose gradient is included."""
    T, dm = _x2(x)
    _req(x, "x", (T, dm), x.dtype)
    _req(dy, "dy", (T, dm), x.dtype)
    _check_hybrid(hy, T, x.dtype)
    d_ff = hy.d_ff
    _check_weights(d_ff, dm, x.dtype, wg_t=wg_t, wu_t=wu_t, wd=wd)
    if out is None:
        f = dict(dtype=torch.float32, device=x.device)
        out = (torch.empty((T, dm), **f), torch.empty((d_ff, dm), **f),
               torch.empty((d_ff, dm), **f), torch.empty((d_ff, dm), **f))
    if len(out) != 4:
        raise TwellError("out: expected (dx, dwg_t, dwu_t, dwd)")
    dx, dwg, dwu, dwd = out
    _req(dx, "dx", (T, dm), torch.float32)
    for name, t in (("dwg_t", dwg), ("dwu_t", dwu), ("dwd", dwd)):
        _req(t, name, (d_ff, dm), torch.float32)
    dev = _on_gpu(("x", x), ("dy", dy), *_hybrid_tensors(hy), ("wg_t", wg_t), ("wu_t", wu_t),
                  ("wd", wd), ("dx", dx), ("dwg_t", dwg), ("dwu_t", dwu), ("dwd", dwd),
                  ("status", status), ("workspace", workspace))
    _status(status, dev)
    need = bwd_workspace_bytes(_dt(x), T, dm, d_ff, hy.K, hy.max_ovf)
    workspace = _ws(workspace, need, dev)
    nbytes = 0 if workspace is None else workspace.numel()
    ch = hy.c()
    _check(load().hybrid_ffn_bwd(_dt(x), _ptr(x), _ptr(dy), ctypes.byref(ch), _ptr(wg_t),
                                 _ptr(wu_t), _ptr(wd), dm, float(l1), _ptr(dx), _ptr(dwg),
                                 _ptr(dwu),
                                 _ptr(dwd), _ptr(workspace), nbytes, _ptr(status),
                                 _timing(timing), _stream(x.device)), "hybrid_ffn_bwd")
    return out


# ---- the residual stream's norm and the 8-bit products around the layer
@dataclass
class Fp8:
    """A matrix [rows][cols] in 8 bits: element (r, c) stands for
    q[r][c] * scale[c // 128][r // block_rows]."""

    q: torch.Tensor      # [rows][cols rounded up to 128] float8_e4m3fn, zeros past cols
    scale: torch.Tensor  # [ceil(cols / 128)][ceil(rows / block_rows)] float32
    cols: int
    block_rows: int = 1

    @property
    def rows(self):
        return self.q.shape[0]

    def float(self) -> torch.Tensor:
        """The float32 values the matrix stands for."""
        s = self.scale.t().repeat_interleave(self.block_rows, 0)[:self.rows]
        return (self.q.float() * s.repeat_interleave(FP8_BLOCK, 1))[:, :self.cols]


def empty_fp8(rows, cols, block_rows, device) -> Fp8:
    nb = -(-cols // FP8_BLOCK)
    return Fp8(torch.empty(rows, nb * FP8_BLOCK, dtype=_E4, device=device),
               torch.empty(nb, -(-rows // block_rows), dtype=_F32, device=device),
               cols, block_rows)


# These calls are short enough on the GPU for their arguments' checks to be
# what they cost: the structures are packed as bytes (MatC and Fp8C, a third of
# the time of building them), and the usual case of every check is one test.
_pack_mat = struct.Struct("iiqi4xP").pack
_pack_fp8 = struct.Struct("iii4xPP").pack
assert struct.calcsize("iiqi4xP") == ctypes.sizeof(MatC)
assert struct.calcsize("iii4xPP") == ctypes.sizeof(Fp8C)
_F32, _E4 = torch.float32, torch.float8_e4m3fn
_DT = {torch.float32: TWELL_F32, torch.bfloat16: TWELL_BF16}


def _check_fp8(m, name, rows=None, cols=None):
    """(structure, rows) of a well-formed Fp8 [rows][cols]."""
    if not isinstance(m, Fp8):
        raise TwellError(f"{name}: expected an Fp8")
    q, s, br, mc = m.q, m.scale, m.block_rows, m.cols
    if br not in (1, FP8_BLOCK):
        raise TwellError(f"{name}.block_rows: {br}, expected 1 or {FP8_BLOCK}")
    if not isinstance(q, torch.Tensor) or q.dim() != 2:
        raise TwellError(f"{name}.q: expected a [rows][cols up to 128] tensor")
    r, pitch = q.shape
    nb = -(-mc // FP8_BLOCK)
    sshape = (nb, r if br == 1 else -(-r // FP8_BLOCK))
    if not (isinstance(s, torch.Tensor) and pitch == nb * FP8_BLOCK and s.shape == sshape
            and q.dtype == _E4 and s.dtype == _F32 and q.is_contiguous() and s.is_contiguous()
            and (cols is None or (mc == cols and r == rows))):
        if cols is not None and mc != cols:
            raise TwellError(f"{name}: {mc} columns, expected {cols}")
        if rows is None:
            rows = r
        _req(q, f"{name}.q", (rows, nb * FP8_BLOCK), _E4)
        _req(s, f"{name}.scale", sshape, _F32)
    return _pack_fp8(r, mc, br, q.data_ptr(), s.data_ptr()), r


def _mat(t, name, rows=None, cols=None, dtype=None):
    """(structure, rows, cols) of a [rows][cols] float32 or bfloat16 tensor
    whose columns are consecutive; its rows may be any stride apart (a slice
    of columns)."""
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise TwellError(f"{name}: expected a [rows][cols] tensor")
    r, c = t.shape
    ld, sc = t.stride()
    tdt = t.dtype
    dt = _DT.get(tdt)
    if rows is not None and (r != rows or c != cols):
        raise TwellError(f"{name}: shape {(r, c)}, expected {(rows, cols)}")
    if dt is None:
        raise TwellError(f"unsupported dtype {tdt}")
    if dtype is not None and tdt != dtype:
        raise TwellError(f"{name}: dtype {tdt}, expected {dtype}")
    if (sc != 1 and c > 1) or (r > 1 and ld < c):
        raise TwellError(f"{name}: columns must be consecutive and rows must not overlap")
    return _pack_mat(r, c, ld if r > 1 else c, dt, t.data_ptr()), r, c


def _new_mat(rows, cols, dtype, device):
    """A new contiguous tensor and its structure."""
    dt = _DT.get(dtype)
    if dt is None:
        raise TwellError(f"unsupported dtype {dtype}")
    t = torch.empty(rows, cols, dtype=dtype, device=device)
    return t, _pack_mat(rows, cols, cols, dt, t.data_ptr())


def _new_fp8(rows, cols, block_rows, device):
    m = empty_fp8(rows, cols, block_rows, device)
    return m, _pack_fp8(rows, cols, block_rows, m.q.data_ptr(), m.scale.data_ptr())


def _gain(gain, d):
    if not isinstance(gain, torch.Tensor):
        raise TwellError("gain: expected a tensor")
    dt = _DT.get(gain.dtype)
    if dt is None or gain.shape != (d,) or not gain.is_contiguous():
        _req(gain, "gain", (d,), gain.dtype)
        raise TwellError(f"unsupported dtype {gain.dtype}")
    return dt


def _gpu(named: dict) -> int:
    """The number of the one GPU that every given tensor lives on."""
    dev = -1
    for t in named.values():
        if t is not None:
            i = t.get_device()
            if i < 0 or (dev >= 0 and i != dev):
                _on_gpu(*named.items())  # names the tensor
            dev = i
    return dev


def _at(t):
    return None if t is None else t.data_ptr()


def rmsnorm_fwd(x, gain, residual=None, eps: float = 1e-6, out_dtype=torch.bfloat16, h=None,
                out=None, timing: KernelTimer | None = None):
    """h = residual + x and its root-mean-square norm n times gain; returns
    (n, h). n is a tensor of out_dtype (float32 or bfloat16), or an Fp8 for
    float8_e4m3fn; h has residual's dtype (without a residual h is x). h and
    out, if given, are written (h may be residual or x, out may be x, in place)."""
    mx, T, d = _mat(x, "x")
    gdt = _gain(gain, d)
    mr = mh = mn = m8 = None
    on = {"x": x, "gain": gain}
    if residual is not None:
        mr = _mat(residual, "residual", T, d)[0]
        on["residual"] = residual
        if h is None:
            h, mh = _new_mat(T, d, residual.dtype, x.device)
        else:
            mh = _mat(h, "h", T, d, residual.dtype)[0]
            on["h"] = h
    elif h is not None:
        raise TwellError("h: written only with a residual")
    if out_dtype == torch.float8_e4m3fn:
        if out is None:
            out, m8 = _new_fp8(T, d, 1, x.device)
        else:
            m8 = _check_fp8(out, "out", T, d)[0]
            on["out.q"], on["out.scale"] = out.q, out.scale
    elif out is None:
        out, mn = _new_mat(T, d, out_dtype, x.device)
    else:
        mn = _mat(out, "out", T, d, out_dtype)[0]
        on["out"] = out
    dev = _gpu(on)
    _check(load().twell_rmsnorm_fwd(mx, mr, gain.data_ptr(), gdt, eps, mh, mn, m8,
                                    _timing(timing), _raw_stream(dev)), "twell_rmsnorm_fwd")
    return out, (x if residual is None else h)


def rmsnorm_bwd_workspace_bytes(T, d) -> int:
    return int(load().twell_rmsnorm_bwd_workspace_bytes(T, d))


def rmsnorm_bwd(dn, h, gain, dres=None, eps: float = 1e-6, dh_dtype=torch.float32, dh=None,
                dgain=None, workspace=None, timing: KernelTimer | None = None):
    """Gradients of rmsnorm_fwd from dn: (dh, dgain). h is the stream the
    forward normed (its h), dres the gradient reaching h past the norm."""
    md, T, d = _mat(dn, "dn")
    mh = _mat(h, "h", T, d)[0]
    gdt = _gain(gain, d)
    mr = None if dres is None else _mat(dres, "dres", T, d)[0]
    if dh is None:
        dh, mo = _new_mat(T, d, dh_dtype, dn.device)
    else:
        mo = _mat(dh, "dh", T, d)[0]
    if dgain is None:
        dgain = torch.empty(d, dtype=torch.float32, device=dn.device)
    else:
        _req(dgain, "dgain", (d,), torch.float32)
    if workspace is not None:
        _ws_form(workspace)
    dev = _gpu({"dn": dn, "h": h, "gain": gain, "dres": dres, "dh": dh, "dgain": dgain,
                "workspace": workspace})
    workspace = _ws(workspace, rmsnorm_bwd_workspace_bytes(T, d), dn.device)
    _check(load().twell_rmsnorm_bwd(md, mh, gain.data_ptr(), gdt, eps, mr, mo, dgain.data_ptr(),
                                    _at(workspace), 0 if workspace is None else workspace.numel(),
                                    _timing(timing), _raw_stream(dev)), "twell_rmsnorm_bwd")
    return dh, dgain


def fp8_quant(x, block_rows: int = 1, layout: str = "rows", out: Fp8 | None = None,
              out_t: Fp8 | None = None, timing: KernelTimer | None = None):
    """x in 8 bits with block scales; returns (of x, of its transpose), None
    for the one that layout ("rows", "cols" or "both") leaves out."""
    mx, R, C = _mat(x, "x")
    if layout not in ("rows", "cols", "both"):
        raise TwellError(f"layout: {layout!r}, expected 'rows', 'cols' or 'both'")
    if block_rows not in (1, FP8_BLOCK):
        raise TwellError(f"block_rows: {block_rows}, expected 1 or {FP8_BLOCK}")
    on, m = {"x": x}, {}
    for name, t, skip, shape in (("out", out, "cols", (R, C)), ("out_t", out_t, "rows", (C, R))):
        if layout == skip:
            if t is not None:
                raise TwellError(f"{name}: not written with layout {layout!r}")
            m[name] = None, None
        elif t is None:
            m[name] = _new_fp8(*shape, block_rows, x.device)
        else:
            m[name] = t, _check_fp8(t, name, *shape)[0]
            if t.block_rows != block_rows:
                raise TwellError(f"{name}: block_rows {t.block_rows}, expected {block_rows}")
            on[name + ".q"], on[name + ".scale"] = t.q, t.scale
    (out, mo), (out_t, mt) = m["out"], m["out_t"]
    dev = _gpu(on)
    _check(load().twell_fp8_quant(mx, mo, mt, _timing(timing), _raw_stream(dev)),
           "twell_fp8_quant")
    return out, out_t


def fp8_matmul_workspace_bytes(M, N, K) -> int:
    return int(load().twell_fp8_matmul_workspace_bytes(M, N, K))


def fp8_matmul(a: Fp8, b: Fp8, out=None, out_dtype=torch.bfloat16, fast_sums: bool = False,
               workspace=None, timing: KernelTimer | None = None):
    """out [a.rows][b.rows] = a b^T of two 8-bit matrices, out in float32 or
    bfloat16. Products are added in float32, or, with fast_sums, by the 8-bit
    matrix instruction at up to twice the rate. Those lose less than 2^-10 of the
    sum of a result's terms' sizes; typically 1e-5 to 3e-5 of the results' norm,
    far below a bfloat16 result's rounding unless large terms cancel."""
    (ma, M), (mb, N) = _check_fp8(a, "a"), _check_fp8(b, "b")
    K = a.cols
    if b.cols != K:
        raise TwellError(f"b: {b.cols} columns, a has {K}")
    on = {"a.q": a.q, "a.scale": a.scale, "b.q": b.q, "b.scale": b.scale}
    if out is None:
        out, mo = _new_mat(M, N, out_dtype, a.q.device)
    else:
        mo = _mat(out, "out", M, N, out_dtype)[0]
        on["out"] = out
    if workspace is not None:
        _ws_form(workspace)
        on["workspace"] = workspace
    args = ma, mb, mo, SUMS_FP8 if fast_sums else SUMS_F32
    end = _timing(timing), _raw_stream(_gpu(on))
    # most sizes need no workspace, and the call says which do
    rc = load().twell_fp8_matmul(*args, _at(workspace),
                                 0 if workspace is None else workspace.numel(), *end)
    if rc == E_WORKSPACE:
        workspace = _ws(workspace, fp8_matmul_workspace_bytes(M, N, K), out.device)
        rc = load().twell_fp8_matmul(*args, _at(workspace),
                                     0 if workspace is None else workspace.numel(), *end)
    _check(rc, "twell_fp8_matmul")
    return out


# ---- weights in 4 bits
@dataclass
class Fp4:
    """A matrix [rows][cols] in 4 bits: element (r, c) stands for
    value(code) * scale[c // group][r], the code of column 2b in the low half
    of byte b of q's row."""

    q: torch.Tensor      # [rows][cols rounded up to 128, / 2] uint8, zeros past cols
    scale: torch.Tensor  # [cols rounded up to 128, / group][rows] bfloat16
    cols: int
    group: int = 128

    @property
    def rows(self):
        return self.q.shape[0]

    def float(self) -> torch.Tensor:
        """The float32 values the matrix stands for (on any device)."""
        v = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), device=self.q.device)
        c = torch.stack((self.q & 15, self.q >> 4), 2).flatten(1)
        s = self.scale.float().t().repeat_interleave(self.group, 1)
        return (v[c.int()] * s)[:, :self.cols]


_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
_U8, _BF = torch.uint8, torch.bfloat16


def empty_fp4(rows, cols, group, device) -> Fp4:
    nb = -(-cols // FP4_BLOCK)
    return Fp4(torch.empty(rows, nb * (FP4_BLOCK // 2), dtype=_U8, device=device),
               torch.empty(nb * (FP4_BLOCK // group), rows, dtype=_BF, device=device), cols, group)


def _check_fp4(m, name, rows=None, cols=None):
    """(structure, rows) of a well-formed Fp4 [rows][cols]."""
    if not isinstance(m, Fp4):
        raise TwellError(f"{name}: expected an Fp4")
    q, s, g, mc = m.q, m.scale, m.group, m.cols
    if g not in FP4_GROUPS:
        raise TwellError(f"{name}.group: {g}, expected one of {FP4_GROUPS}")
    if not isinstance(q, torch.Tensor) or q.dim() != 2:
        raise TwellError(f"{name}.q: expected a [rows][cols up to 128, / 2] tensor")
    r, pitch = q.shape
    nb = -(-mc // FP4_BLOCK)
    sshape = (nb * (FP4_BLOCK // g), r)
    if not (isinstance(s, torch.Tensor) and pitch == nb * (FP4_BLOCK // 2) and s.shape == sshape
            and q.dtype == _U8 and s.dtype == _BF and q.is_contiguous() and s.is_contiguous()
            and (cols is None or (mc == cols and r == rows))):
        if cols is not None and mc != cols:
            raise TwellError(f"{name}: {mc} columns, expected {cols}")
        if rows is None:
            rows = r
        _req(q, f"{name}.q", (rows, nb * (FP4_BLOCK // 2)), _U8)
        _req(s, f"{name}.scale", sshape, _BF)
    return _pack_fp8(r, mc, g, q.data_ptr(), s.data_ptr()), r  # Fp4C: the same fields


assert ctypes.sizeof(Fp4C) == ctypes.sizeof(Fp8C)


def fp4_quant(w, group: int = 128, out: Fp4 | None = None,
              timing: KernelTimer | None = None) -> Fp4:
    """w in 4 bits, one scale for each `group` (32, 64 or 128) columns of a row."""
    mw, R, C = _mat(w, "w")
    if group not in FP4_GROUPS:
        raise TwellError(f"group: {group}, expected one of {FP4_GROUPS}")
    if out is None:
        out = empty_fp4(R, C, group, w.device)
    mo = _check_fp4(out, "out", R, C)[0]
    if out.group != group:
        raise TwellError(f"out: group {out.group}, expected {group}")
    dev = _gpu({"w": w, "out.q": out.q, "out.scale": out.scale})
    _check(load().twell_fp4_quant(mw, mo, _timing(timing), _raw_stream(dev)), "twell_fp4_quant")
    return out


def fp4_dequant(w: Fp4, out=None, out_dtype=torch.bfloat16, timing: KernelTimer | None = None):
    """The matrix that w stands for, in bfloat16 (exact for fp4_quant's scales)
    or float32."""
    mw, R = _check_fp4(w, "w")
    on = {"w.q": w.q, "w.scale": w.scale}
    if out is None:
        out, mo = _new_mat(R, w.cols, out_dtype, w.q.device)
    else:
        mo = _mat(out, "out", R, w.cols, out_dtype)[0]
        on["out"] = out
    _check(load().twell_fp4_dequant(mw, mo, _timing(timing), _raw_stream(_gpu(on))),
           "twell_fp4_dequant")
    return out


def fp4_matmul_workspace_bytes(dtype, T, N, K) -> int:
    return int(load().twell_fp4_matmul_workspace_bytes(dtype, T, N, K))


def fp4_matmul_dx_workspace_bytes(dtype, T, N, K) -> int:
    return int(load().twell_fp4_matmul_dx_workspace_bytes(dtype, T, N, K))


def _fp4_mm(name, x, xname, w, out, out_dtype, workspace, timing):
    mw, N = _check_fp4(w, "w")
    mx, T, C = _mat(x, xname)
    fwd = name == "twell_fp4_matmul"
    take, give = (w.cols, N) if fwd else (N, w.cols)
    if C != take:
        raise TwellError(f"{xname}: {C} columns, w has {take} {'columns' if fwd else 'rows'}")
    on = {xname: x, "w.q": w.q, "w.scale": w.scale}
    if out is None:
        out, mo = _new_mat(T, give, out_dtype, x.device)
    else:
        mo = _mat(out, "out", T, give, out_dtype)[0]
        on["out"] = out
    if workspace is not None:
        _ws_form(workspace)
        on["workspace"] = workspace
    L = load()
    call = getattr(L, name)
    end = _timing(timing), _raw_stream(_gpu(on))
    # few tokens need no workspace, and the call says which do
    rc = call(mx, mw, mo, _at(workspace), 0 if workspace is None else workspace.numel(), *end)
    if rc == E_WORKSPACE:
        need = getattr(L, name + "_workspace_bytes")(_dt(x), T, N, w.cols)
        workspace = _ws(workspace, need, x.device)
        rc = call(mx, mw, mo, workspace.data_ptr(), workspace.numel(), *end)
    _check(rc, name)
    return out


def fp4_matmul(x, w: Fp4, out=None, out_dtype=torch.bfloat16, workspace=None,
               timing: KernelTimer | None = None):
    """out [T][w.rows] = x w^T, x [T][w.cols] and out each float32 or bfloat16.
    Products are exact, sums float32; any number of tokens, one upwards."""
    return _fp4_mm("twell_fp4_matmul", x, "x", w, out, out_dtype, workspace, timing)


def fp4_matmul_dx(dy, w: Fp4, out=None, out_dtype=torch.bfloat16, workspace=None,
                  timing: KernelTimer | None = None):
    """fp4_matmul's gradient for x: out [T][w.cols] = dy w, dy [T][w.rows]."""
    return _fp4_mm("twell_fp4_matmul_dx", dy, "dy", w, out, out_dtype, workspace, timing)


def fp4_decode_workspace_bytes(dtype, T, d_model, d_ff) -> int:
    return int(load().twell_fp4_decode_workspace_bytes(dtype, T, d_model, d_ff))


def fp4_decode_fwd(x, wg_t: Fp4, wu_t: Fp4, wd: Fp4, y=None, workspace=None,
                   timing: KernelTimer | None = None):
    """The sparse layer for T <= DECODE_T tokens from 4-bit weights [d_ff][d_model]
    of one group: y [T][d_model] float32, (relu(x Wg) * (x Wu)) Wd with g and u
    in float32."""
    mx, T, dm = _mat(x, "x")
    if T > DECODE_T:
        raise TwellError(f"fp4_decode_fwd takes at most {DECODE_T} tokens, got {T}")
    mg, f = _check_fp4(wg_t, "wg_t")
    on = {"x": x, "wg_t.q": wg_t.q, "wg_t.scale": wg_t.scale}
    ms = []
    for name, m in (("wu_t", wu_t), ("wd", wd)):
        ms.append(_check_fp4(m, name, f, dm)[0])
        if m.group != wg_t.group:
            raise TwellError(f"{name}: group {m.group}, wg_t has {wg_t.group}")
        on[name + ".q"], on[name + ".scale"] = m.q, m.scale
    if wg_t.cols != dm:
        raise TwellError(f"wg_t: {wg_t.cols} columns, expected {dm}")
    if y is None:
        y = torch.empty(T, dm, dtype=torch.float32, device=x.device)
    else:
        _req(y, "y", (T, dm), torch.float32)
        on["y"] = y
    if workspace is not None:
        _ws_form(workspace)
        on["workspace"] = workspace
    dev = _gpu(on)
    workspace = _ws(workspace, fp4_decode_workspace_bytes(_dt(x), T, dm, f), x.device)
    _check(load().twell_fp4_decode_fwd(mx, mg, *ms, y.data_ptr(), _at(workspace),
                                       0 if workspace is None else workspace.numel(),
                                       _timing(timing), _raw_stream(dev)),
           "twell_fp4_decode_fwd")
    return y
