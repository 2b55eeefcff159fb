"""Thin ctypes binding of liblstm.so (include/lstm.h).

Argument marshalling only: every step of the forward and backward pass runs
in the library's HIP kernels.  torch is used for device memory and streams
(it is imported before the library so that both share one HIP runtime).
There is no fallback: if liblstm.so is missing or cannot be loaded, importing
this module raises.
"""
from __future__ import annotations

import ctypes
import math
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "liblstm.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is not built; run `python -m layer_lstm_amd.build`")
_lib = ctypes.CDLL(LIB_PATH)

# --- constants restated from include/lstm.h ---------------------------------
ABI_VERSION = 3
REVERSE = 1  # lstm_shape.flags: the reverse direction of time
GATES_IJFO = 2  # lstm_shape.flags: W/b/dW/db row blocks in the gate order i, g, f, o
TWO_BIAS = 4  # lstm_shape.flags: b and db are [2][4H] (b_ih, b_hh)
BIDIRECTIONAL = 8  # lstm_shape.flags: both directions of time, outputs side by side
GATE_I, GATE_F, GATE_G, GATE_O = 0, 1, 2, 3
I32, I64 = 0, 1  # id_type of token ids
MAX_TOP = 32  # LSTM_MAX_TOP
LINATTN_STEP = 8  # LSTM_LINATTN_STEP: the most steps whose state may be moved on in place
ADAMW_BLOCK = 256  # LSTM_ADAMW_BLOCK: values of an 8-bit state that share a scale
F32, BF16, F16 = 0, 1, 2
OK = 0
STATUS = {0: "OK", -1: "ERR_NULL", -2: "ERR_DIMS", -3: "ERR_DTYPE", -4: "ERR_ALIGN",
          -5: "ERR_WORKSPACE", -6: "ERR_UNSUPPORTED", -7: "ERR_COOP", -8: "ERR_LAUNCH",
          -9: "ERR_TIMEOUT", -10: "ERR_DEVICE", -11: "ERR_SCRATCH", -12: "ERR_PLACEMENT",
          -13: "ERR_STATE"}
DEBUG_FAIL_STEP, DEBUG_MISPLACE, DEBUG_XCD_LOCAL = 1, 2, 3  # lstm_debug_inject
PROBE_READS, PROBE_READS_AHEAD, PROBE_BARRIER, PROBE_DMA = 1, 2, 4, 8  # lstm_probe_mfma_stage
PROBE_SCRATCH_BYTES = 1 << 20  # LSTM_PROBE_SCRATCH_BYTES
SCRATCH_BYTES = 64 << 20  # LSTM_SCRATCH_BYTES
EXPORTS = ("lstm_abi_version", "lstm_status_string", "lstm_query", "lstm_query_plan", "lstm_fwd_train",
           "lstm_fwd_train_scratch", "lstm_bwd", "lstm_check_workspace", "lstm_timing_enable", "lstm_timing_read",
           "lstm_stamps_set", "lstm_probe_exchange", "lstm_probe_mfma_stage", "lstm_debug_inject", "lstm_stack_query",
           "lstm_stack_fwd_train", "lstm_stack_bwd", "lstm_embed_query", "lstm_embed_fwd", "lstm_embed_bwd",
           "lstm_attend_query", "lstm_attend_fwd", "lstm_attend_bwd", "lstm_logprob_query", "lstm_logprob_fwd", "lstm_logprob_bwd",
           "lstm_linattn_query", "lstm_linattn_fwd", "lstm_linattn_bwd", "lstm_penalty", "lstm_adamw_query",
           "lstm_adamw_norm", "lstm_adamw_step")
STAMP_WGS, STAMP_POINTS = 8, 6
KERNEL_KINDS = ("input_projection", "forward_recurrence", "backward_recurrence", "dW_product",
                "dx_product", "direction_copy", "state_copy", "embedding", "cross_attention", "log_probability",
                "linear_attention", "penalty", "adamw")


class Shape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("B", ctypes.c_int64), ("I", ctypes.c_int64),
                ("H", ctypes.c_int64), ("dtype", ctypes.c_int32), ("flags", ctypes.c_int32)]


class PlanInfo(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("rows_per_group", "units_per_group", "groups", "units_groups",
                                               "grid", "waves", "xcd_local", "fwd_valu", "bwd_valu",
                                               "inproj_tiles_per_wg", "directions_concurrent", "fwd_tagged")] + \
               [("reserved", ctypes.c_int32 * 4)]


class EmbedShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("N", "V", "D", "ld_table", "ld_out", "padding")] + \
               [("scale", ctypes.c_float), ("dtype", ctypes.c_int32), ("id_type", ctypes.c_int32)]


class LogprobShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("N", "V", "ld", "ld_grad")] + \
               [("scale", ctypes.c_float)] + [(n, ctypes.c_int32) for n in ("top", "dtype", "id_type")]


class Stride(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("t", "b", "h")]


class AttendShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("Tq", "Tk", "B", "Hq", "Hk", "D")] + \
               [(n, Stride) for n in ("q", "k", "v", "o", "dout", "dq", "dk", "dv")] + \
               [("mask_b", ctypes.c_int64), ("scale", ctypes.c_float), ("dtype", ctypes.c_int32)]


class LinattnShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("T", "B", "Hq", "Hk", "D", "Dv")] + \
               [(n, Stride) for n in ("q", "k", "v", "o", "dout", "dq", "dk", "dv")] + \
               [("scale", ctypes.c_float), ("dtype", ctypes.c_int32)]


class PenaltyShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("N", "V", "ld", "ld_out", "L", "history_n", "history_t", "ld_bias", "ld_mask")] + \
               [("dtype", ctypes.c_int32), ("id_type", ctypes.c_int32)]


class AdamwTensor(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("param", "grad", "master", "m", "v", "m_scale", "v_scale")] + \
               [("n", ctypes.c_int64), ("weight_decay", ctypes.c_double)]


class AdamwShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_double) for n in ("lr", "beta1", "beta2", "eps")] + \
               [("step", ctypes.c_int64), ("dtype", ctypes.c_int32), ("bits", ctypes.c_int32)]


class AdamwControl(ctypes.Structure):  # in device memory
    _fields_ = [("step", ctypes.c_int64)] + [(n, ctypes.c_float) for n in ("scale", "norm", "rate", "root")] + \
               [("skip", ctypes.c_int32), ("reserved", ctypes.c_int32)]


_P = ctypes.c_void_p
_lib.lstm_abi_version.restype = ctypes.c_int
_lib.lstm_status_string.restype = ctypes.c_char_p
_lib.lstm_status_string.argtypes = [ctypes.c_int]
_lib.lstm_query.restype = ctypes.c_int
_lib.lstm_query.argtypes = [ctypes.POINTER(Shape), ctypes.POINTER(ctypes.c_size_t)]
_lib.lstm_query_plan.restype = ctypes.c_int
_lib.lstm_query_plan.argtypes = [ctypes.POINTER(Shape), ctypes.POINTER(PlanInfo)]
_lib.lstm_fwd_train.restype = ctypes.c_int
_lib.lstm_fwd_train.argtypes = [ctypes.POINTER(Shape)] + [_P] * 9 + [_P, ctypes.c_size_t, _P]
_lib.lstm_fwd_train_scratch.restype = ctypes.c_int
_lib.lstm_fwd_train_scratch.argtypes = [ctypes.POINTER(Shape)] + [_P] * 9 + [_P]
_lib.lstm_bwd.restype = ctypes.c_int
_lib.lstm_bwd.argtypes = [ctypes.POINTER(Shape)] + [_P] * 9 + [_P, ctypes.c_size_t] + [_P] * 5 + [_P]
_lib.lstm_check_workspace.restype = ctypes.c_int
_lib.lstm_check_workspace.argtypes = [_P, ctypes.c_size_t, _P]
_lib.lstm_timing_enable.restype = ctypes.c_int
_lib.lstm_timing_enable.argtypes = [ctypes.c_int]
_lib.lstm_timing_read.restype = ctypes.c_int
_lib.lstm_timing_read.argtypes = [ctypes.c_int, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_int64)]
_lib.lstm_probe_exchange.restype = ctypes.c_int
_lib.lstm_probe_exchange.argtypes = [ctypes.POINTER(Shape), ctypes.c_int, _P, ctypes.c_size_t,
                                     ctypes.POINTER(ctypes.c_double), _P]
_lib.lstm_probe_mfma_stage.restype = ctypes.c_int
_lib.lstm_probe_mfma_stage.argtypes = [ctypes.c_int, ctypes.c_int64, _P, ctypes.c_size_t,
                                       ctypes.POINTER(ctypes.c_double), _P]
_lib.lstm_stack_query.restype = ctypes.c_int
_lib.lstm_stack_query.argtypes = [ctypes.POINTER(Shape), ctypes.c_int64, ctypes.c_int64,
                                  ctypes.POINTER(ctypes.c_size_t), ctypes.POINTER(ctypes.c_int32)]
_lib.lstm_stack_fwd_train.restype = ctypes.c_int
_lib.lstm_stack_fwd_train.argtypes = [ctypes.POINTER(Shape), ctypes.c_int64, ctypes.c_int64] + [_P] * 8 + \
    [_P, ctypes.c_size_t, _P]
_lib.lstm_stack_bwd.restype = ctypes.c_int
_lib.lstm_stack_bwd.argtypes = [ctypes.POINTER(Shape), ctypes.c_int64, ctypes.c_int64] + [_P] * 8 + \
    [_P, ctypes.c_size_t] + [_P] * 5 + [_P]
for _n, _a in (("lstm_embed_query", [ctypes.POINTER(EmbedShape), ctypes.POINTER(ctypes.c_size_t)]),
               ("lstm_embed_fwd", [ctypes.POINTER(EmbedShape)] + [_P] * 4),
               ("lstm_embed_bwd", [ctypes.POINTER(EmbedShape)] + [_P] * 3 + [ctypes.c_size_t] + [_P] * 2),
               ("lstm_attend_query", [ctypes.POINTER(AttendShape)] + [ctypes.POINTER(ctypes.c_size_t)] * 2),
               ("lstm_attend_fwd", [ctypes.POINTER(AttendShape)] + [_P] * 6 + [ctypes.c_size_t] + [_P] * 3),
               ("lstm_attend_bwd", [ctypes.POINTER(AttendShape)] + [_P] * 9 + [ctypes.c_size_t] + [_P] * 4),
               ("lstm_logprob_query", [ctypes.POINTER(LogprobShape), ctypes.POINTER(ctypes.c_size_t)]),
               ("lstm_logprob_fwd", [ctypes.POINTER(LogprobShape)] + [_P] * 3 + [ctypes.c_size_t] + [_P] * 7),
               ("lstm_logprob_bwd", [ctypes.POINTER(LogprobShape)] + [_P] * 10),
               ("lstm_linattn_query", [ctypes.POINTER(LinattnShape)] + [ctypes.POINTER(ctypes.c_size_t)] * 2),
               ("lstm_linattn_fwd", [ctypes.POINTER(LinattnShape)] + [_P] * 7 + [ctypes.c_size_t] + [_P] * 3),
               ("lstm_linattn_bwd", [ctypes.POINTER(LinattnShape)] + [_P] * 9 + [ctypes.c_size_t] + [_P] * 5),
               ("lstm_penalty", [ctypes.POINTER(PenaltyShape)] + [_P] * 10),
               ("lstm_adamw_query", [ctypes.POINTER(AdamwShape), ctypes.POINTER(AdamwTensor), ctypes.c_int64,
                                     ctypes.POINTER(ctypes.c_size_t)]),
               ("lstm_adamw_norm", [ctypes.POINTER(AdamwShape), ctypes.POINTER(AdamwTensor), ctypes.c_int64,
                                    ctypes.c_double, ctypes.c_double, _P, ctypes.c_size_t, _P, _P]),
               ("lstm_adamw_step", [ctypes.POINTER(AdamwShape), ctypes.POINTER(AdamwTensor), ctypes.c_int64, _P, _P])):
    getattr(_lib, _n).restype = ctypes.c_int
    getattr(_lib, _n).argtypes = _a
_lib.lstm_debug_inject.restype = ctypes.c_int
_lib.lstm_debug_inject.argtypes = [ctypes.c_int, ctypes.c_int64]
_lib.lstm_stamps_set.restype = ctypes.c_int
_lib.lstm_stamps_set.argtypes = [_P, ctypes.c_size_t, ctypes.c_int64]


class LstmError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        msg = _lib.lstm_status_string(code).decode()
        super().__init__(f"{where}: {STATUS.get(code, code)} ({msg})")


def lib():
    return _lib


def abi_version() -> int:
    return _lib.lstm_abi_version()


def status_string(code: int) -> str:
    return _lib.lstm_status_string(code).decode()


def torch_dtype(dtype: int):
    return {F32: torch.float32, BF16: torch.bfloat16, F16: torch.float16}[dtype]


def make_shape(T, B, I, H, dtype, reverse=False, gate_order="ifjo", two_bias=False, bidirectional=False) -> Shape:
    if gate_order not in ("ifjo", "ijfo"):
        raise ValueError(f"gate_order {gate_order!r}: 'ifjo' or 'ijfo'")
    flags = (REVERSE if reverse else 0) | (GATES_IJFO if gate_order == "ijfo" else 0) | \
        (TWO_BIAS if two_bias else 0) | (BIDIRECTIONAL if bidirectional else 0)
    return Shape(int(T), int(B), int(I), int(H), int(dtype), flags)


def query(shape: Shape) -> int:
    n = ctypes.c_size_t(0)
    rc = _lib.lstm_query(ctypes.byref(shape), ctypes.byref(n))
    if rc != OK:
        raise LstmError(rc, "lstm_query")
    return n.value


def query_plan(shape: Shape) -> dict:
    """Layout of the persistent recurrences for `shape` (lstm_query_plan)."""
    info = PlanInfo()
    rc = _lib.lstm_query_plan(ctypes.byref(shape), ctypes.byref(info))
    if rc != OK:
        raise LstmError(rc, "lstm_query_plan")
    return {n: getattr(info, n) for n, _ in PlanInfo._fields_ if n != "reserved"}


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr() if t.numel() > 0 else None


# The current stream's handle without a Stream object built for it (3 us a
# call, which is a third of a small operator's).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream):
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is None:
        return torch.cuda.current_stream().cuda_stream
    return _raw_stream(torch.cuda.current_device())


def fwd_train(shape, x, W, b, h0, c0, y, hT, cT, workspace, ws_bytes=None, stream=None, check=True,
              seq_length=None):
    """lstm_fwd_train on torch tensors (None = NULL; seq_length: int32 [B]
    device tensor of sequence lengths).  Returns the status."""
    if ws_bytes is None:
        ws_bytes = workspace.numel() * workspace.element_size()
    rc = _lib.lstm_fwd_train(ctypes.byref(shape), _ptr(x), _ptr(W), _ptr(b), _ptr(h0), _ptr(c0),
                             _ptr(seq_length), _ptr(y), _ptr(hT), _ptr(cT), _ptr(workspace), ws_bytes,
                             _stream(stream))
    if check and rc != OK:
        raise LstmError(rc, "lstm_fwd_train")
    return rc


def fwd_train_scratch(shape, x, W, b, h0, c0, y, hT, cT, stream=None, check=True, seq_length=None):
    """lstm_fwd_train_scratch on torch tensors (None = NULL): the forward
    pass with the library's own device array as the workspace.  Returns the
    status."""
    rc = _lib.lstm_fwd_train_scratch(ctypes.byref(shape), _ptr(x), _ptr(W), _ptr(b), _ptr(h0), _ptr(c0),
                                     _ptr(seq_length), _ptr(y), _ptr(hT), _ptr(cT), _stream(stream))
    if check and rc != OK:
        raise LstmError(rc, "lstm_fwd_train_scratch")
    return rc


def bwd(shape, dy, dhT, dcT, x, W, h0, c0, y, workspace, dx, dW, db, dh0, dc0, ws_bytes=None,
        stream=None, check=True, seq_length=None):
    """lstm_bwd on torch tensors (None = NULL).  Returns the status."""
    if ws_bytes is None:
        ws_bytes = workspace.numel() * workspace.element_size()
    rc = _lib.lstm_bwd(ctypes.byref(shape), _ptr(dy), _ptr(dhT), _ptr(dcT), _ptr(x), _ptr(W),
                       _ptr(h0), _ptr(c0), _ptr(seq_length), _ptr(y), _ptr(workspace), ws_bytes, _ptr(dx),
                       _ptr(dW), _ptr(db), _ptr(dh0), _ptr(dc0), _stream(stream))
    if check and rc != OK:
        raise LstmError(rc, "lstm_bwd")
    return rc


def check_workspace(workspace, stream=None) -> int:
    return _lib.lstm_check_workspace(_ptr(workspace), workspace.numel() * workspace.element_size(),
                                     _stream(stream))


def timing_enable(on: bool) -> None:
    _lib.lstm_timing_enable(1 if on else 0)


def timing_read() -> dict:
    """{kind name: (total ms, launches)} of the per-kernel event timing."""
    out = {}
    for k, name in enumerate(KERNEL_KINDS):
        ms, n = ctypes.c_double(0), ctypes.c_int64(0)
        rc = _lib.lstm_timing_read(k, ctypes.byref(ms), ctypes.byref(n))
        if rc != OK:
            raise LstmError(rc, "lstm_timing_read")
        out[name] = (ms.value, n.value)
    return out


def probe_exchange(shape: Shape, workspace, layout: int = 0, stream=None) -> float:
    """lstm_probe_exchange: microseconds per step of the forward
    recurrence's exchange alone (layout 0: the plan's own; 1: spread over
    the XCDs)."""
    us = ctypes.c_double(0)
    rc = _lib.lstm_probe_exchange(ctypes.byref(shape), int(layout), _ptr(workspace),
                                  workspace.numel() * workspace.element_size(), ctypes.byref(us), _stream(stream))
    if rc != OK:
        raise LstmError(rc, "lstm_probe_exchange")
    return us.value


def probe_mfma_stage(parts: int, scratch, iters: int = 4000, stream=None) -> float:
    """lstm_probe_mfma_stage: fraction of the bf16 dense peak of 32 MFMAs
    per wave and iteration with the stage parts `parts` (PROBE_* bits);
    scratch: device memory of at least PROBE_SCRATCH_BYTES."""
    frac = ctypes.c_double(0)
    rc = _lib.lstm_probe_mfma_stage(int(parts), int(iters), _ptr(scratch), scratch.numel() * scratch.element_size(),
                                    ctypes.byref(frac), _stream(stream))
    if rc != OK:
        raise LstmError(rc, "lstm_probe_mfma_stage")
    return frac.value


def debug_inject(what: int, value: int) -> None:
    """lstm_debug_inject: the test hooks of the failure paths."""
    rc = _lib.lstm_debug_inject(int(what), int(value))
    if rc != OK:
        raise LstmError(rc, "lstm_debug_inject")


def stamps_set(buf, T) -> None:
    """Point the recurrent kernels' phase stamps at a device tensor of at
    least 2*8*T*6 int64 values (None disables)."""
    if buf is None:
        _lib.lstm_stamps_set(None, 0, 0)
        return
    rc = _lib.lstm_stamps_set(_ptr(buf), buf.numel() * buf.element_size(), int(T))
    if rc != OK:
        raise LstmError(rc, "lstm_stamps_set")


class Lstm:
    """One problem shape with its workspace and output buffers on the current
    device.  ``forward``/``backward`` take device tensors and return device
    tensors; nothing is synchronised."""

    def __init__(self, T, B, I, H, dtype=F32, device="cuda", reverse=False, gate_order="ifjo", two_bias=False,
                 bidirectional=False):
        self.shape = make_shape(T, B, I, H, dtype, reverse, gate_order, two_bias, bidirectional)
        self.T, self.B, self.I, self.H, self.dtype = T, B, I, H, dtype
        self.tdtype = torch_dtype(dtype)
        self.ws_bytes = query(self.shape)
        self.workspace = torch.empty(self.ws_bytes, dtype=torch.uint8, device=device)
        dev, td = device, self.tdtype
        nd = (2,) if bidirectional else ()
        self.y = torch.empty((T, B, 2 * H if bidirectional else H), dtype=td, device=dev)
        self.hT = torch.empty(nd + (B, H), dtype=td, device=dev)
        self.cT = torch.empty(nd + (B, H), dtype=td, device=dev)
        self.dx = torch.empty((T, B, I), dtype=td, device=dev)
        self.dW = torch.empty(nd + (4 * H, H + I), dtype=td, device=dev)
        self.db = torch.empty(nd + ((2, 4 * H) if two_bias else (4 * H,)), dtype=td, device=dev)
        self.dh0 = torch.empty(nd + (B, H), dtype=td, device=dev)
        self.dc0 = torch.empty(nd + (B, H), dtype=td, device=dev)

    def forward(self, x, W, b=None, h0=None, c0=None, stream=None, seq_length=None):
        fwd_train(self.shape, x, W, b, h0, c0, self.y, self.hT, self.cT, self.workspace,
                  self.ws_bytes, stream, seq_length=seq_length)
        return self.y, self.hT, self.cT

    def backward(self, dy, dhT, dcT, x, W, h0=None, c0=None, want_db=True, stream=None, seq_length=None):
        bwd(self.shape, dy, dhT, dcT, x, W, h0, c0, self.y, self.workspace, self.dx, self.dW,
            self.db if want_db else None, self.dh0, self.dc0, self.ws_bytes, stream, seq_length=seq_length)
        return self.dx, self.dW, self.db, self.dh0, self.dc0

    def check(self, stream=None):
        rc = check_workspace(self.workspace, stream)
        if rc != OK:
            raise LstmError(rc, "lstm_check_workspace")


def stack_query(shape: Shape, layers: int, chunks: int = 0):
    """lstm_stack_query: (workspace bytes, the most layers whose
    recurrences share one launch; 1: one after the other)."""
    n, conc = ctypes.c_size_t(0), ctypes.c_int32(0)
    rc = _lib.lstm_stack_query(ctypes.byref(shape), int(layers), int(chunks), ctypes.byref(n), ctypes.byref(conc))
    if rc != OK:
        raise LstmError(rc, "lstm_stack_query")
    return n.value, conc.value


class Stack:
    """An L-layer stack (lstm_stack_*) of one problem shape with its
    workspace and output buffers on the current device.  W is the layers'
    weights back to back (layer 0 [4H][H+I], the others [4H][2H]); b, h0, c0,
    dhT, dcT have a leading layer axis."""

    def __init__(self, T, B, I, H, layers, dtype=F32, chunks=0, device="cuda", gate_order="ifjo", two_bias=False):
        self.shape = make_shape(T, B, I, H, dtype, False, gate_order, two_bias)
        self.T, self.B, self.I, self.H, self.L, self.chunks = T, B, I, H, layers, chunks
        self.tdtype = torch_dtype(dtype)
        self.ws_bytes, self.concurrent = stack_query(self.shape, layers, chunks)
        self.workspace = torch.empty(self.ws_bytes, dtype=torch.uint8, device=device)
        dev, td, L = device, self.tdtype, layers
        self.w_elems = 4 * H * (H + I) + (L - 1) * 4 * H * 2 * H
        self.y = torch.empty((T, B, H), dtype=td, device=dev)
        self.hT = torch.empty((L, B, H), dtype=td, device=dev)
        self.cT = torch.empty((L, B, H), dtype=td, device=dev)
        self.dx = torch.empty((T, B, I), dtype=td, device=dev)
        self.dW = torch.empty((self.w_elems,), dtype=td, device=dev)
        self.db = torch.empty((L, 2, 4 * H) if two_bias else (L, 4 * H), dtype=td, device=dev)
        self.dh0 = torch.empty((L, B, H), dtype=td, device=dev)
        self.dc0 = torch.empty((L, B, H), dtype=td, device=dev)

    def forward(self, x, W, b=None, h0=None, c0=None, stream=None):
        rc = _lib.lstm_stack_fwd_train(ctypes.byref(self.shape), self.L, self.chunks, _ptr(x), _ptr(W), _ptr(b),
                                       _ptr(h0), _ptr(c0), _ptr(self.y), _ptr(self.hT), _ptr(self.cT),
                                       _ptr(self.workspace), self.ws_bytes, _stream(stream))
        if rc != OK:
            raise LstmError(rc, "lstm_stack_fwd_train")
        return self.y, self.hT, self.cT

    def backward(self, dy, dhT, dcT, x, W, h0=None, c0=None, want_db=True, stream=None):
        rc = _lib.lstm_stack_bwd(ctypes.byref(self.shape), self.L, self.chunks, _ptr(dy), _ptr(dhT), _ptr(dcT),
                                 _ptr(x), _ptr(W), _ptr(h0), _ptr(c0), _ptr(self.y), _ptr(self.workspace),
                                 self.ws_bytes, _ptr(self.dx), _ptr(self.dW), _ptr(self.db if want_db else None),
                                 _ptr(self.dh0), _ptr(self.dc0), _stream(stream))
        if rc != OK:
            raise LstmError(rc, "lstm_stack_bwd")
        return self.dx, self.dW, self.db, self.dh0, self.dc0

    def check(self, stream=None):
        rc = check_workspace(self.workspace, stream)
        if rc != OK:
            raise LstmError(rc, "lstm_check_workspace")


# --- sequence-to-sequence operators -------------------------------------------
_ID_TYPES = {torch.int64: I64, torch.int32: I32}
_STORAGE = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}


# A kernel that is given the address of host memory, or of another device's,
# faults: the operators take tensors of the device that their buffers are on,
# and launch while it is the current one.
def _device_index(device):
    d = torch.device(device)
    if d.type != "cuda":
        raise ValueError(f"device {device}: a GPU")
    return torch.cuda.current_device() if d.index is None else d.index


def _on_device(index, *tensors):
    for t in tensors:
        if t is not None and t.get_device() != index:
            raise ValueError(f"every tensor on cuda:{index}, where the operator's buffers are (one is on {t.device})")


def _row_stride(name, x, width):
    """Elements between the rows of x [n, width], which the kernels take to be
    at least width (the stride of one row alone means nothing)."""
    st = x.stride(0)
    if st >= width:
        return st
    if x.shape[0] > 1:
        raise ValueError(f"{name}: rows {st} elements apart, at least {width} (an expanded tensor has to be copied)")
    return width


def _buffer(shape, dtype, device, stream):
    """An output made when it is first needed, from the memory of the stream
    that writes it: memory of the current stream may still be in use there."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _stream_on(index, stream):
    if torch.cuda.current_device() != index or (stream is not None and stream.device_index != index):
        raise ValueError(f"cuda:{index} has to be the current device, and the stream's")
    return _raw_stream(index) if stream is None and _raw_stream is not None else _stream(stream)


def _capturing(stream):
    with torch.cuda.stream(stream):
        return torch.cuda.is_current_stream_capturing()


def _settle(index):
    torch.cuda.current_stream(index).synchronize()


def _workspace(fn, name, shape, device):
    n = ctypes.c_size_t(0)
    rc = fn(ctypes.byref(shape), ctypes.byref(n))
    if rc != OK:
        raise LstmError(rc, name)
    return torch.empty(n.value, dtype=torch.uint8, device=device)


class Embedding:
    """The embedding of N tokens by a [V, D] table (lstm_embed_*), with its
    workspace and output buffers on the current device.  `ids`: N tokens,
    int32 or int64, of any shape, contiguous; the rows of `table` and `dout`
    may be strided (D contiguous).  `padding`: an id whose row takes no
    gradient."""

    def __init__(self, N, V, D, dtype=F32, scale=1.0, padding=None, device="cuda"):
        self.N, self.V, self.D, self.dtype, self.device = N, V, D, dtype, device
        self.shape = EmbedShape(N, V, D, D, D, -1 if padding is None else int(padding), float(scale), int(dtype), I64)
        self._ref = ctypes.byref(self.shape)
        self.workspace = _workspace(_lib.lstm_embed_query, "lstm_embed_query", self.shape, device)
        self._dev = _device_index(device)
        self.tdtype = torch_dtype(dtype)
        self.out = self.dtable = None

    def _ids(self, ids):
        if ids.numel() != self.N or not ids.is_contiguous() or ids.dtype not in _ID_TYPES:
            raise ValueError(f"ids: {self.N} contiguous tokens, int32 or int64")
        self.shape.id_type = _ID_TYPES[ids.dtype]

    def forward(self, ids, table, stream=None):
        """out [*ids.shape, D] = scale * table[ids]."""
        self._ids(ids)
        _on_device(self._dev, ids, table)
        if table.dtype != self.tdtype or table.shape != (self.V, self.D) or (self.D > 1 and table.stride(1) != 1):
            raise ValueError(f"table: [{self.V}, {self.D}] of {self.tdtype}, rows contiguous")
        if self.out is None or self.out.shape[:-1] != ids.shape:
            self.out = _buffer((*ids.shape, self.D), self.tdtype, self.device, stream)
        self.shape.ld_table, self.shape.ld_out = _row_stride("table", table, self.D), self.D
        rc = _lib.lstm_embed_fwd(self._ref, _ptr(ids), _ptr(table), _ptr(self.out), _stream_on(self._dev, stream))
        if rc != OK:
            raise LstmError(rc, "lstm_embed_fwd")
        return self.out

    def backward(self, ids, dout, stream=None):
        """dtable [V, D] of dout [*ids.shape, D]."""
        self._ids(ids)
        _on_device(self._dev, ids, dout)
        if dout.dtype != self.tdtype or dout.shape != (*ids.shape, self.D):
            raise ValueError(f"dout: {[*ids.shape, self.D]} of {self.tdtype}")
        try:
            rows = dout if dout.dim() == 2 else dout.view(self.N, self.D)
        except RuntimeError:
            raise ValueError("dout: rows at one stride") from None
        if self.D > 1 and rows.stride(1) != 1:
            raise ValueError("dout: rows contiguous")
        if self.dtable is None:
            self.dtable = _buffer((self.V, self.D), self.tdtype, self.device, stream)
        self.shape.ld_table, self.shape.ld_out = self.D, _row_stride("dout", rows, self.D)
        rc = _lib.lstm_embed_bwd(self._ref, _ptr(ids), _ptr(rows), _ptr(self.workspace), self.workspace.numel(),
                                 _ptr(self.dtable), _stream_on(self._dev, stream))
        if rc != OK:
            raise LstmError(rc, "lstm_embed_bwd")
        return self.dtable


class Attention:
    """Cross attention of Tq queries to Tk states of an encoder
    (lstm_attend_*), with its workspace and output buffers on the current
    device.  q [Tq, B, Hq, D], k and v [Tk, B, Hk, D] (any strides >= 0, D
    contiguous; an expanded k or v gets the gradient of its expanded form);
    k_length: int32 [B] valid keys of each sequence; key_mask: bool or uint8
    [B, Tk], zero = not a key.  o, dq, dk, dv are dense, lse fp32 [B, Hq,
    Tq]."""

    def __init__(self, Tq, Tk, B, Hq, Hk, D, dtype=F32, scale=None, device="cuda"):
        self.Tq, self.Tk, self.B, self.Hq, self.Hk, self.D, self.dtype, self.device = Tq, Tk, B, Hq, Hk, D, dtype, device
        dense_q, dense_k = Stride(B * Hq * D, Hq * D, D), Stride(B * Hk * D, Hk * D, D)
        self.shape = AttendShape(Tq, Tk, B, Hq, Hk, D, dense_q, dense_k, dense_k, dense_q, dense_q, dense_q, dense_k,
                                 dense_k, Tk, float(max(D, 1) ** -0.5 if scale is None else scale), int(dtype))
        nf, nb = ctypes.c_size_t(0), ctypes.c_size_t(0)
        rc = _lib.lstm_attend_query(ctypes.byref(self.shape), ctypes.byref(nf), ctypes.byref(nb))
        if rc != OK:
            raise LstmError(rc, "lstm_attend_query")
        self._ref = ctypes.byref(self.shape)
        self._dev = _device_index(device)
        self.ws_bytes = max(nf.value, nb.value)
        self.workspace = torch.empty(self.ws_bytes, dtype=torch.uint8, device=device)
        self.tdtype = torch_dtype(dtype)
        self.o = torch.empty((Tq, B, Hq, D), dtype=self.tdtype, device=device)
        self.lse = torch.empty((B, Hq, Tq), dtype=torch.float32, device=device)
        self.dq = self.dk = self.dv = None

    def _strides(self, name, s, x, T, H):
        if x.dtype != self.tdtype or x.shape != (T, self.B, H, self.D) or (self.D > 1 and x.stride(3) != 1):
            raise ValueError(f"{name}: {[T, self.B, H, self.D]} of {self.tdtype}, last dimension contiguous")
        s.t, s.b, s.h = x.stride()[:3]

    def _inputs(self, q, k, v, k_length, key_mask):
        self._strides("q", self.shape.q, q, self.Tq, self.Hq)
        self._strides("k", self.shape.k, k, self.Tk, self.Hk)
        self._strides("v", self.shape.v, v, self.Tk, self.Hk)
        if k_length is not None and (k_length.dtype != torch.int32 or k_length.shape != (self.B,) or
                                     not k_length.is_contiguous()):
            raise ValueError(f"k_length: int32 [{self.B}], contiguous")
        if key_mask is not None:
            if key_mask.dtype not in (torch.bool, torch.uint8) or key_mask.shape != (self.B, self.Tk) or \
                    (self.Tk > 1 and key_mask.stride(1) != 1):
                raise ValueError(f"key_mask: bool or uint8 {[self.B, self.Tk]}, rows contiguous")
            self.shape.mask_b = key_mask.stride(0)
        _on_device(self._dev, q, k, v, k_length, key_mask)

    def forward(self, q, k, v, k_length=None, key_mask=None, stream=None):
        """o [Tq, B, Hq, D] and lse [B, Hq, Tq]."""
        self._inputs(q, k, v, k_length, key_mask)
        rc = _lib.lstm_attend_fwd(self._ref, _ptr(q), _ptr(k), _ptr(v), _ptr(k_length), _ptr(key_mask),
                                  _ptr(self.workspace), self.ws_bytes, _ptr(self.o), _ptr(self.lse),
                                  _stream_on(self._dev, stream))
        if rc != OK:
            raise LstmError(rc, "lstm_attend_fwd")
        return self.o, self.lse

    def backward(self, dout, q, k, v, k_length=None, key_mask=None, stream=None):
        """dq, dk, dv after a forward on the same inputs."""
        self._inputs(q, k, v, k_length, key_mask)
        self._strides("dout", self.shape.dout, dout, self.Tq, self.Hq)
        _on_device(self._dev, dout)
        if self.dq is None:
            self.dq = _buffer((self.Tq, self.B, self.Hq, self.D), self.tdtype, self.device, stream)
            self.dk, self.dv = (_buffer((self.Tk, self.B, self.Hk, self.D), self.tdtype, self.device, stream)
                                for _ in range(2))
        rc = _lib.lstm_attend_bwd(self._ref, _ptr(dout), _ptr(q), _ptr(k), _ptr(v), _ptr(k_length),
                                  _ptr(key_mask), _ptr(self.o), _ptr(self.lse), _ptr(self.workspace), self.ws_bytes,
                                  _ptr(self.dq), _ptr(self.dk), _ptr(self.dv), _stream_on(self._dev, stream))
        if rc != OK:
            raise LstmError(rc, "lstm_attend_bwd")
        return self.dq, self.dk, self.dv


class LogProb:
    """Log probabilities of given tokens under N rows of V logits, entropies
    and the `top` best alternatives (lstm_logprob_*), with workspace and
    output buffers on the current device.  logits [N, V] (rows may be
    strided), targets [N] int32 or int64."""

    def __init__(self, N, V, dtype=F32, top=0, scale=1.0, device="cuda"):
        self.N, self.V, self.top, self.dtype, self.device = N, V, int(top), dtype, device
        self.shape = LogprobShape(N, V, V, V, float(scale), int(top), int(dtype), I64)
        self._ref = ctypes.byref(self.shape)
        self.workspace = _workspace(_lib.lstm_logprob_query, "lstm_logprob_query", self.shape, device)
        self._dev = _device_index(device)
        self.tdtype = torch_dtype(dtype)
        self.record = torch.empty((N, 2), dtype=torch.float32, device=device)
        self.lse, self.logp, self.entropy = (torch.empty(N, dtype=torch.float32, device=device) for _ in range(3))
        self.top_logp = torch.empty((N, self.top), dtype=torch.float32, device=device)
        self.top_ids = self.dlogits = None

    def _rows(self, logits, targets):
        if logits.dtype != self.tdtype or logits.shape != (self.N, self.V) or (self.V > 1 and logits.stride(1) != 1):
            raise ValueError(f"logits: [{self.N}, {self.V}] of {self.tdtype}, rows contiguous")
        if targets.shape != (self.N,) or not targets.is_contiguous() or targets.dtype not in _ID_TYPES:
            raise ValueError(f"targets: [{self.N}] int32 or int64, contiguous")
        _on_device(self._dev, logits, targets)
        self.shape.id_type = _ID_TYPES[targets.dtype]
        self.shape.ld = _row_stride("logits", logits, self.V)

    def forward(self, logits, targets, stream=None):
        """logp [N], entropy [N] and, with alternatives, top_logp and top_ids [N, top] (ids of targets' type)."""
        self._rows(logits, targets)
        if self.top_ids is None or self.top_ids.dtype != targets.dtype:
            self.top_ids = _buffer((self.N, self.top), targets.dtype, self.device, stream)
        rc = _lib.lstm_logprob_fwd(self._ref, _ptr(logits), _ptr(targets), _ptr(self.workspace),
                                   self.workspace.numel(), _ptr(self.record), _ptr(self.lse), _ptr(self.logp),
                                   _ptr(self.entropy), _ptr(self.top_logp), _ptr(self.top_ids),
                                   _stream_on(self._dev, stream))
        if rc != OK:
            raise LstmError(rc, "lstm_logprob_fwd")
        if not self.top:
            return self.logp, self.entropy
        return self.logp, self.entropy, self.top_logp, self.top_ids

    def backward(self, logits, targets, dlogp=None, dentropy=None, dtop=None, stream=None):
        """dlogits [N, V] after a forward on the same logits and targets; cotangents fp32, contiguous, None = zero."""
        self._rows(logits, targets)
        for name, g, shape in (("dlogp", dlogp, (self.N,)), ("dentropy", dentropy, (self.N,)),
                               ("dtop", dtop, (self.N, self.top))):
            if g is not None and (g.dtype != torch.float32 or g.shape != shape or not g.is_contiguous()):
                raise ValueError(f"{name}: {list(shape)} of float32, contiguous")
        _on_device(self._dev, dlogp, dentropy, dtop)
        if dtop is not None and self.top and (self.top_ids is None or self.top_ids.dtype != targets.dtype):
            raise ValueError("backward follows a forward on the same targets")
        if self.dlogits is None:
            self.dlogits = _buffer((self.N, self.V), self.tdtype, self.device, stream)
        rc = _lib.lstm_logprob_bwd(self._ref, _ptr(logits), _ptr(targets), _ptr(self.record),
                                   _ptr(self.entropy), _ptr(self.top_ids), _ptr(dlogp), _ptr(dentropy),
                                   _ptr(dtop) if self.top else None, _ptr(self.dlogits),
                                   _stream_on(self._dev, stream))
        if rc != OK:
            raise LstmError(rc, "lstm_logprob_bwd")
        return self.dlogits


class LinearAttention:
    """Linear attention with a decay for each head (lstm_linattn_*) of T steps
    of B sequences, with workspace and output buffers on the current device.
    q [T, B, Hq, D], k [T, B, Hk, D], v [T, B, Hk, Dv] (any strides >= 0, the
    last dimension contiguous; an expanded k or v gets the gradient of its
    expanded form), log_decay fp32 [Hk], states fp32 [B, Hk, D, Dv], length:
    int32 [B] steps of each sequence.  o, dq, dk, dv are dense."""

    def __init__(self, T, B, Hq, Hk, D, Dv=None, dtype=F32, scale=None, device="cuda"):
        Dv = D if Dv is None else Dv
        self.T, self.B, self.Hq, self.Hk, self.D, self.Dv, self.dtype, self.device = T, B, Hq, Hk, D, Dv, dtype, device
        rows = [Stride(B * h * d, h * d, d) for h, d in ((Hq, D), (Hk, D), (Hk, Dv), (Hq, Dv))]
        q, k, v, o = rows
        self.shape = LinattnShape(T, B, Hq, Hk, D, Dv, q, k, v, o, o, q, k, v,
                                  float(max(D, 1) ** -0.5 if scale is None else scale), int(dtype))
        # shapes of q, k, v, dout and the states, and the strides of those last seen
        self._shapes = [torch.Size(i) for i in ((T, B, Hq, D), (T, B, Hk, D), (T, B, Hk, Dv), (T, B, Hq, Dv), (B, Hk, D, Dv))]
        self._at = [None] * 4
        nf, nb = ctypes.c_size_t(0), ctypes.c_size_t(0)
        rc = _lib.lstm_linattn_query(ctypes.byref(self.shape), ctypes.byref(nf), ctypes.byref(nb))
        if rc != OK:
            raise LstmError(rc, "lstm_linattn_query")
        self._ref = ctypes.byref(self.shape)
        self._dev = _device_index(device)
        self.tdtype = torch_dtype(dtype)
        self._fwd_bytes, self._bwd_bytes = nf.value, nb.value
        self.workspace = torch.empty(self._fwd_bytes, dtype=torch.uint8, device=device)
        self.o = torch.empty((T, B, Hq, Dv), dtype=self.tdtype, device=device)
        self.state = self.dq = self.dk = self.dv = self.dstate = self.bwd_workspace = None

    def _rows(self, name, i, x):
        shape, at = self._shapes[i], x.stride()
        if x.dtype is not self.tdtype or x.shape != shape or (at[3] != 1 and shape[3] > 1 and x.numel()):
            raise ValueError(f"{name}: {list(shape)} of {self.tdtype}, last dimension contiguous")
        if at != self._at[i]:
            self._at[i] = at
            if x.numel():
                s = getattr(self.shape, name)
                s.t, s.b, s.h = at[:3]

    def _state(self, name, x):
        if x.dtype is not torch.float32 or x.shape != self._shapes[4] or not x.is_contiguous():
            raise ValueError(f"{name}: float32 {list(self._shapes[4])}, contiguous")

    def _inputs(self, q, k, v, log_decay, state, length):
        self._rows("q", 0, q)
        self._rows("k", 1, k)
        self._rows("v", 2, v)
        if log_decay.dtype is not torch.float32 or log_decay.dim() != 1 or log_decay.shape[0] != self.Hk or \
                not log_decay.is_contiguous():
            raise ValueError(f"log_decay: float32 [{self.Hk}], contiguous")
        if state is not None:
            self._state("state", state)
        if length is not None and (length.dtype is not torch.int32 or length.shape != (self.B,) or not length.is_contiguous()):
            raise ValueError(f"length: int32 [{self.B}], contiguous")
        _on_device(self._dev, q, k, v, log_decay, state, length)

    def _forward(self, q, k, v, log_decay, state, length, out, stream):
        rc = _lib.lstm_linattn_fwd(self._ref, q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(),
                                   None if length is None else length.data_ptr(), None if state is None else state.data_ptr(),
                                   self.workspace.data_ptr(), self._fwd_bytes, self.o.data_ptr(), out.data_ptr(),
                                   _stream_on(self._dev, stream))
        if rc != OK:
            raise LstmError(rc, "lstm_linattn_fwd")

    def forward(self, q, k, v, log_decay, state=None, length=None, stream=None):
        """o [T, B, Hq, Dv] and the state after the last step (a buffer of its own: pass a copy of it as the next
        call's `state`)."""
        self._inputs(q, k, v, log_decay, state, length)
        if self.state is None:
            self.state = _buffer((self.B, self.Hk, self.D, self.Dv), torch.float32, self.device, stream)
        if state is not None and state.numel() and state.data_ptr() == self.state.data_ptr():
            raise ValueError("state: not the buffer that the new state is written to")
        self._forward(q, k, v, log_decay, state, length, self.state, stream)
        return self.o, self.state

    def step(self, q, k, v, log_decay, state, length=None, stream=None):
        """o [T, B, Hq, Dv] of at most LINATTN_STEP steps; `state` is moved on in place."""
        if self.T > LINATTN_STEP:
            raise ValueError(f"step: at most {LINATTN_STEP} steps")
        self._inputs(q, k, v, log_decay, state, length)
        self._forward(q, k, v, log_decay, state, length, state, stream)
        return self.o

    def backward(self, dout, q, k, v, log_decay, state=None, length=None, dstate=None, stream=None):
        """dq, dk, dv and the gradient of `state`; dstate: the gradient of the state after the last step."""
        self._inputs(q, k, v, log_decay, state, length)
        self._rows("dout", 3, dout)
        if dstate is not None:
            self._state("dstate", dstate)
        _on_device(self._dev, dout, dstate)
        if self.bwd_workspace is None:  # beside the forward's, which a captured forward goes on using
            self.bwd_workspace = self.workspace if self.workspace.numel() >= self._bwd_bytes else \
                _buffer((self._bwd_bytes,), torch.uint8, self.device, stream)
        if self.dq is None:
            self.dq = _buffer((self.T, self.B, self.Hq, self.D), self.tdtype, self.device, stream)
            self.dk = _buffer((self.T, self.B, self.Hk, self.D), self.tdtype, self.device, stream)
            self.dv = _buffer((self.T, self.B, self.Hk, self.Dv), self.tdtype, self.device, stream)
            self.dstate = _buffer((self.B, self.Hk, self.D, self.Dv), torch.float32, self.device, stream)
        if dstate is not None and dstate.numel() and dstate.data_ptr() == self.dstate.data_ptr():
            raise ValueError("dstate: not the buffer that the gradient of the state before is written to")
        rc = _lib.lstm_linattn_bwd(self._ref, _ptr(dout), _ptr(q), _ptr(k), _ptr(v), _ptr(log_decay), _ptr(length),
                                   _ptr(state), _ptr(dstate), _ptr(self.bwd_workspace), self.bwd_workspace.numel(),
                                   _ptr(self.dq), _ptr(self.dk), _ptr(self.dv), _ptr(self.dstate),
                                   _stream_on(self._dev, stream))
        if rc != OK:
            raise LstmError(rc, "lstm_linattn_bwd")
        return self.dq, self.dk, self.dv, self.dstate


class Penalty:
    """Penalties for repeated tokens, biases and masks on N rows of V logits
    (lstm_penalty), with an output buffer on the current device."""

    def __init__(self, N, V, dtype=F32, device="cuda"):
        self.N, self.V, self.dtype, self.device = N, V, dtype, device
        self._n, self._rows = torch.Size((N,)), torch.Size((N, V))
        self.shape = PenaltyShape(N, V, V, V, 0, 0, 0, 0, 0, int(dtype), I64)
        self._ref = ctypes.byref(self.shape)
        self._dev = _device_index(device)
        self.tdtype = torch_dtype(dtype)
        self.out = None

    def forward(self, logits, history=None, length=None, repetition=None, presence=None, frequency=None, bias=None,
                mask=None, out=None, stream=None):
        """logits [N, V] changed by what its row says: history [N, L] of int32 or int64 ids (any strides >= 0: time-major
        ids as ids.t()), the first length [N] (int32) of them counting; repetition, presence, frequency fp32 [N]; bias
        fp32 [V] or [N, V]; mask int32 [N, >= ceil(V / 32)], bit v % 32 of word v / 32 zero = not allowed.  `out`: where
        to (logits itself or memory that is not theirs); None: the operator's own buffer."""
        N, V, s, td, dev = self.N, self.V, self.shape, self.tdtype, self._dev
        if logits.dtype is not td or logits.shape != self._rows or (V > 1 and logits.stride(1) != 1):
            raise ValueError(f"logits: [{N}, {V}] of {td}, rows contiguous")
        s.ld = _row_stride("logits", logits, V)
        if out is None:
            if self.out is None:
                self.out = _buffer((N, V), td, self.device, stream)
            out, s.ld_out = self.out, V
        else:
            if out.dtype is not td or out.shape != self._rows or (V > 1 and out.stride(1) != 1):
                raise ValueError(f"out: [{N}, {V}] of {td}, rows contiguous")
            s.ld_out = _row_stride("out", out, V)
        row = self._row
        rep, pre, fre = row("repetition", repetition), row("presence", presence), row("frequency", frequency)
        s.L = 0
        if history is not None:
            if history.dim() != 2 or history.shape[0] != N or history.dtype not in _ID_TYPES:
                raise ValueError(f"history: [{N}, L] of int32 or int64")
            s.L = history.shape[1]
            s.history_n, s.history_t = history.stride()
            s.id_type = _ID_TYPES[history.dtype]
        elif rep or pre or fre:
            raise ValueError("history: the tokens that the penalties are for")
        if length is not None and (length.dtype is not torch.int32 or length.shape != self._n or not length.is_contiguous()):
            raise ValueError(f"length: int32 [{N}], contiguous")
        if bias is not None:
            if bias.dtype is not torch.float32 or bias.shape not in ((V,), self._rows) or (V > 1 and bias.stride(-1) != 1):
                raise ValueError(f"bias: float32 [{V}] or [{N}, {V}], rows contiguous")
            s.ld_bias = 0 if bias.dim() == 1 or N == 1 or bias.stride(0) == 0 else _row_stride("bias", bias, V)
        if mask is not None:
            words = (V + 31) // 32
            if mask.dtype is not torch.int32 or mask.dim() != 2 or mask.shape[0] != N or mask.shape[1] < words or \
                    (words > 1 and mask.stride(1) != 1):
                raise ValueError(f"mask: int32 [{N}, {words}], rows contiguous")
            s.ld_mask = _row_stride("mask", mask, words)
        _on_device(dev, logits, history, length, bias, mask, out)
        rc = _lib.lstm_penalty(self._ref, logits.data_ptr(), None if history is None else history.data_ptr(),
                               None if length is None else length.data_ptr(), rep, pre, fre,
                               None if bias is None else bias.data_ptr(), None if mask is None else mask.data_ptr(),
                               out.data_ptr(), _stream_on(dev, stream))
        if rc != OK:
            raise LstmError(rc, "lstm_penalty")
        return out

    def _row(self, name, x):
        if x is None:
            return None
        if x.dtype is not torch.float32 or x.shape != self._n or not x.is_contiguous():
            raise ValueError(f"{name}: float32 [{self.N}], contiguous")
        if x.get_device() != self._dev:
            _on_device(self._dev, x)
        return x.data_ptr()


class AdamW:
    """AdamW steps over `params` (contiguous tensors of one storage type on the
    current device, which do not overlap), all of them in one launch
    (lstm_adamw_*).  bits: 32 or 8, of the states m and v; 16-bit parameters
    have an fp32 copy, `master`, unless master=False.  weight_decay: one number
    or one for each parameter.  clip: the norm that the gradients are held to
    (math.inf: none); it, or loss_scale (gradients are divided by it), puts the
    number of the step on the device, leaves out steps whose gradients are not
    finite, and is what a step captured into a graph needs.

    The states of all tensors lie in one buffer each (m, v, master; 8 bits: of
    torch.float8_e4m3fn, with m_scale and v_scale), tensor i's at
    places[i]..., a multiple of ADAMW_BLOCK values.  They are filled when the
    constructor returns, whatever stream the steps go to; what is written into
    them later is for the caller to order before a step.  lr may be changed between
    steps (a captured step keeps the one it was captured with); the parameters
    stay where they are in memory."""

    def __init__(self, params, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, bits=32, clip=None,
                 loss_scale=None, master=None, device="cuda"):
        self.params = list(params)
        kinds = {p.dtype for p in self.params}
        if len(kinds) != 1 or next(iter(kinds)) not in _STORAGE:
            raise ValueError("params: tensors of one type, float32, bfloat16 or float16")
        if bits not in (8, 32):
            raise ValueError("bits: 8 or 32")
        self.tdtype = kinds.pop()
        self.lr, self.betas, self.eps, self.bits, self.device = lr, betas, eps, bits, device
        self._dev = _device_index(device)
        n = len(self.params)
        decay = [float(weight_decay)] * n if isinstance(weight_decay, (int, float)) else [float(x) for x in weight_decay]
        if len(decay) != n:
            raise ValueError(f"weight_decay: one number, or {n}")
        if any(not p.is_contiguous() for p in self.params):
            raise ValueError("params: contiguous tensors")
        _on_device(self._dev, *self.params)
        spans = sorted((p.data_ptr(), p.data_ptr() + p.numel() * p.element_size()) for p in self.params if p.numel())
        if any(a[1] > b[0] for a, b in zip(spans, spans[1:])):
            raise ValueError("params: tensors that do not overlap (one was given twice?)")
        self.places, end = [], 0
        for p in self.params:
            self.places.append(end)
            end += -(-p.numel() // ADAMW_BLOCK) * ADAMW_BLOCK
        state = torch.float32 if bits == 32 else torch.float8_e4m3fn
        self.m, self.v = (torch.zeros(end, dtype=state, device=device) for _ in range(2))
        self.m_scale = self.v_scale = self.master = None
        if bits == 8:
            self.m_scale, self.v_scale = (torch.zeros(end // ADAMW_BLOCK, dtype=torch.float32, device=device) for _ in range(2))
        if self.tdtype != torch.float32 and master is not False:
            self.master = torch.zeros(end, dtype=torch.float32, device=device)
            for p, at in zip(self.params, self.places):
                self.master[at : at + p.numel()].copy_(p.detach().reshape(-1))
        self._table = (AdamwTensor * n)()
        each = self.m.element_size()
        for t, p, at, w in zip(self._table, self.params, self.places, decay):
            t.n, t.weight_decay = p.numel(), w
            if t.n == 0:
                continue
            t.param = p.data_ptr()
            t.m, t.v = self.m.data_ptr() + at * each, self.v.data_ptr() + at * each
            if bits == 8:
                t.m_scale, t.v_scale = (x.data_ptr() + at // ADAMW_BLOCK * 4 for x in (self.m_scale, self.v_scale))
            if self.master is not None:
                t.master = self.master.data_ptr() + at * 4
        self._entries = [(p, p.shape, p.data_ptr(), t) for p, t in zip(self.params, self._table)]
        self.shape = AdamwShape(lr, betas[0], betas[1], eps, 0, _STORAGE[self.tdtype], bits)
        self._ref = ctypes.byref(self.shape)
        self.clip = self.loss_scale = self.control = self.workspace = None
        if clip is not None or loss_scale is not None:
            self.clip = math.inf if clip is None else float(clip)
            self.loss_scale = 1.0 if loss_scale is None else float(loss_scale)
            size = ctypes.c_size_t(0)
            rc = _lib.lstm_adamw_query(self._ref, self._table, n, ctypes.byref(size))
            if rc != OK:
                raise LstmError(rc, "lstm_adamw_query")
            self.workspace = torch.empty(size.value, dtype=torch.uint8, device=device)
            self.control = torch.zeros(ctypes.sizeof(AdamwControl) // 8, dtype=torch.int64, device=device)
        _settle(self._dev)  # the states are filled before a step on any stream reads them

    def set_step(self, t, stream=None):
        """t steps have been taken (0 at the start); `stream`: the one that the next step goes to."""
        self.shape.step = int(t)
        if self.control is not None:
            with torch.cuda.stream(stream):
                self.control[0] = int(t)

    @property
    def norm(self):
        """The last step's gradient norm, a view of device memory (with clip or loss_scale)."""
        return None if self.control is None else self.control.view(torch.float32)[3]

    def step(self, grads, stream=None):
        """One step by the gradients, one for each parameter (contiguous, of its shape and type)."""
        n, table, dev, td = len(self.params), self._table, self._dev, self.tdtype
        if len(grads) != n:
            raise ValueError(f"grads: {n} tensors")
        for g, (p, shape, at, entry) in zip(grads, self._entries):
            if p.data_ptr() != at:
                raise ValueError("params: their memory is no longer the one that this optimiser was made for")
            if g.shape != shape or g.dtype is not td or not g.is_contiguous() or g.get_device() != dev:
                raise ValueError(f"grads: {list(shape)} of {td} on cuda:{dev}, contiguous")
            entry.grad = g.data_ptr()
        s, st = self.shape, _stream_on(dev, stream)
        s.lr, s.beta1, s.beta2, s.eps = self.lr, self.betas[0], self.betas[1], self.eps
        control = None
        if self.control is not None:
            control = self.control.data_ptr()
            rc = _lib.lstm_adamw_norm(self._ref, table, n, self.clip, 1.0 / self.loss_scale,
                                      _ptr(self.workspace), self.workspace.numel(), control, st)
            if rc != OK:
                raise LstmError(rc, "lstm_adamw_norm")
        elif _capturing(stream):
            raise ValueError("a step in a graph needs clip (math.inf: none): its number has to be on the device")
        else:
            s.step += 1
        rc = _lib.lstm_adamw_step(self._ref, table, n, control, st)
        if rc != OK:
            if control is None:
                s.step -= 1
            raise LstmError(rc, "lstm_adamw_step")
