"""NVFP4 linear layers for B200 (sm_100a): Python binding of libnvfp4.so.

NVFP4 two-level microblock quantization (FP32 per-tensor scale + E4M3 scale
per 16 elements, E2M1 elements) and the tcgen05 block-scaled FP4 GEMM, as
used for the linear layers of FLUX diffusion transformers ("英伟达B200狂飙
10.2倍！AI绘图告别龟速！", section "NVFP4量化"; "Scaling NVFP4 Inference for
FLUX.2 on NVIDIA Blackwell Data Center GPUs", section "Key Questions
Answered").

This module only marshals arguments: every step runs in the CUDA kernels of
libnvfp4.so through its C ABI (include/nvfp4.h).  PyTorch supplies device
memory and the current stream.  There is no CPU fallback: if the library is
missing or the device is not sm_100, calls raise.

A call with stream= works on that stream, and the tensors it makes belong to it:
they may be dropped at any time, and used on the caller's current stream once
that waits for the given one; on a third stream they need record_stream.
"""
from __future__ import annotations

import ctypes
import os
import struct
from dataclasses import dataclass
from typing import NamedTuple

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libnvfp4.so")

STATUS = {0: "ok", 1: "invalid argument", 2: "misaligned", 3: "unsupported device",
          4: "launch error", 5: "device wait timed out"}


class NVFP4Error(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn}: {STATUS.get(status, status)} (status {status})")
        self.status = status


class FusedOut(ctypes.Structure):
    _fields_ = [("s_enc_y", ctypes.c_void_p), ("yq", ctypes.c_void_p),
                ("ysf", ctypes.c_void_p), ("amax_y", ctypes.c_void_p),
                ("s_dec_y", ctypes.c_void_p), ("activation", ctypes.c_int)]


ACT_NONE = 0   # nvfp4_activation values
ACT_GELU = 1


class LinearWorkspace(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("xq", ctypes.c_void_p), ("xsf", ctypes.c_void_p),
                ("amax", ctypes.c_void_p), ("s_dec", ctypes.c_void_p), ("y", ctypes.c_void_p),
                ("dyn_ws", ctypes.c_void_p)]


class ResidualNormArgs(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int64) for n in ("rows", "cols")] +
                [f for n in ("residual", "y", "h", "out")
                 for f in ((n, ctypes.c_void_p), (n + "_stride", ctypes.c_int64))] +
                [(n, ctypes.c_void_p) for n in ("post_weight", "post_bias", "pre_weight", "pre_bias")] +
                [f for n in ("gate", "scale", "shift")
                 for f in ((n, ctypes.c_void_p), (n + "_stride", ctypes.c_int64))] +
                [("row_group", ctypes.c_void_p), ("groups", ctypes.c_int64)] +
                [(n, ctypes.c_void_p) for n in ("q", "sf", "s_dec_rows", "amax_rows")] +
                [(n, ctypes.c_float) for n in ("residual_scale", "branch_scale", "post_eps", "pre_eps")] +
                [(n, ctypes.c_int) for n in ("post_norm", "pre_norm", "stream_dtype", "vector_dtype")])


class LoraArgs(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int64) for n in ("rows", "k", "n", "rank", "slots")] +
                [f for n in ("x", "y", "out")
                 for f in ((n, ctypes.c_void_p), (n + "_stride", ctypes.c_int64))] +
                [(n, ctypes.c_void_p) for n in ("a", "b", "scale", "row_slot", "workspace")])


def _packer(args) -> struct.Struct:
    """Packs the fields of an argument structure in order, as C lays it out
    (several times quicker than setting them one by one)."""
    codes = {ctypes.c_int64: "q", ctypes.c_void_p: "P", ctypes.c_float: "f", ctypes.c_int: "i"}
    packer = struct.Struct("@" + "".join(codes[t] for _, t in args._fields_))
    assert packer.size == ctypes.sizeof(args)
    return packer


_pack_residual_norm = _packer(ResidualNormArgs).pack
_pack_lora = _packer(LoraArgs).pack

_lib = None


def lib() -> ctypes.CDLL:
    """The loaded C-ABI library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with "
                              "`python -m nvfp4_block_scaled_19_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        vp, i64, st = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
        L.nvfp4_packed_bytes.restype = ctypes.c_size_t
        L.nvfp4_packed_bytes.argtypes = [i64, i64]
        L.nvfp4_sf_bytes.restype = ctypes.c_size_t
        L.nvfp4_sf_bytes.argtypes = [i64, i64]
        L.nvfp4_status_string.restype = ctypes.c_char_p
        L.nvfp4_status_string.argtypes = [st]
        L.nvfp4_tensor_amax.restype = st
        L.nvfp4_tensor_amax.argtypes = [vp, i64, vp, vp]
        L.nvfp4_quantize.restype = st
        L.nvfp4_quantize.argtypes = [vp, i64, i64, vp, vp, vp, vp, vp]
        L.nvfp4_quantize_with_scale.restype = st
        L.nvfp4_quantize_with_scale.argtypes = [vp, i64, i64, vp, vp, vp, vp, vp]
        L.nvfp4_quantize_one_pass.restype = st
        L.nvfp4_quantize_one_pass.argtypes = [vp, i64, i64, vp, vp, vp, vp, vp, vp]
        L.nvfp4_quantize_dynamic_workspace_bytes.restype = ctypes.c_size_t
        L.nvfp4_quantize_dynamic_workspace_bytes.argtypes = []
        L.nvfp4_quantize_dynamic.restype = st
        L.nvfp4_quantize_dynamic.argtypes = [vp, i64, i64, vp, vp, vp, vp, vp, vp]
        L.nvfp4_quantize_dynamic_noalloc.restype = st
        L.nvfp4_quantize_dynamic_noalloc.argtypes = [vp, i64, i64, vp, vp, vp, vp, vp]
        L.nvfp4_gemm.restype = st
        L.nvfp4_gemm.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, vp,
                                 ctypes.POINTER(FusedOut), vp]
        L.nvfp4_gemm_rowscale.restype = st
        L.nvfp4_gemm_rowscale.argtypes = list(L.nvfp4_gemm.argtypes)
        L.nvfp4_quantize_rowwise.restype = st
        L.nvfp4_quantize_rowwise.argtypes = [vp, i64, i64, vp, vp, vp, vp, vp]
        L.nvfp4_fp8_quantize.restype = st
        L.nvfp4_fp8_quantize.argtypes = [vp, i64, i64, vp, vp, vp, vp]
        L.nvfp4_fp8_gemm.restype = st
        L.nvfp4_fp8_gemm.argtypes = [vp, vp, vp, vp, i64, i64, i64, vp, vp, vp]
        L.nvfp4_residual_norm.restype = st
        L.nvfp4_residual_norm.argtypes = [vp, vp]  # an nvfp4_residual_norm_args
        L.nvfp4_lora_workspace_bytes.restype = ctypes.c_size_t
        L.nvfp4_lora_workspace_bytes.argtypes = [i64, i64, i64, i64]
        L.nvfp4_lora.restype = st
        L.nvfp4_lora.argtypes = [vp, vp]  # an nvfp4_lora_args
        L.nvfp4_selftest_wait_timeout.restype = st
        L.nvfp4_selftest_wait_timeout.argtypes = [i64, vp]
        L.nvfp4_linear_host.restype = st
        L.nvfp4_linear_host.argtypes = [vp, i64, i64, vp, vp, vp, i64, vp,
                                        ctypes.POINTER(LinearWorkspace), vp]
        L.nvfp4_device_error.restype = st
        L.nvfp4_device_error.argtypes = [ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_int)]
        _lib = L
    return _lib


def _check(fn: str, status: int) -> None:
    if status != 0:
        raise NVFP4Error(fn, status)


def _stream(stream=None) -> int:
    """The given stream's handle, or that of the current device's current stream
    (asked for by its handle: building a Stream object costs several us a call)."""
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


def _empty(dtype, device, stream, *shape) -> torch.Tensor:
    """A new tensor that a call writes on the given stream (or the current one).
    It comes from the memory of the stream that writes it, where no other work
    can still hold it, and is not given out again before what the caller's
    stream has read of it by then is done."""
    if stream is None:
        return torch.empty(*shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(*shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(t.device))
    return t


def _ptr(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


def packed_bytes(rows: int, cols: int) -> int:
    return int(lib().nvfp4_packed_bytes(rows, cols))


def sf_bytes(rows: int, cols: int) -> int:
    return int(lib().nvfp4_sf_bytes(rows, cols))


def _require(x: torch.Tensor, dtype, name: str) -> None:
    if not x.is_cuda or x.dtype != dtype or not x.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA {dtype} tensor")


@dataclass
class NVFP4Tensor:
    """A quantized [rows, cols] tensor: packed codes, tiled scales, decode scale."""
    q: torch.Tensor       # uint8 [rows, cols/2]
    sf: torch.Tensor      # uint8 [sf_bytes(rows, cols)]
    s_dec: torch.Tensor   # float32 [1] = 1 / S_enc, or [rows] with per-row scales
    rows: int
    cols: int


def empty_nvfp4(rows: int, cols: int, device=None, row_scales: bool = False, stream=None) -> NVFP4Tensor:
    dev = torch.device("cuda") if device is None else device
    return NVFP4Tensor(_empty(torch.uint8, dev, stream, rows, cols // 2),
                       _empty(torch.uint8, dev, stream, sf_bytes(rows, cols)),
                       _empty(torch.float32, dev, stream, rows if row_scales else 1),
                       rows, cols)


def tensor_amax(x: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """max |x| of a bf16 CUDA tensor into a 1-element fp32 CUDA tensor."""
    _require(x, torch.bfloat16, "x")
    if out is None:
        out = _empty(torch.float32, x.device, stream, 1)
    _check("nvfp4_tensor_amax", lib().nvfp4_tensor_amax(x.data_ptr(), x.numel(), out.data_ptr(),
                                                        _stream(stream)))
    return out


def quantize(x: torch.Tensor, amax: torch.Tensor, out: NVFP4Tensor | None = None,
             stream=None) -> NVFP4Tensor:
    """Dynamic NVFP4 quantization of bf16 x[rows, cols] given its amax (device)."""
    _require(x, torch.bfloat16, "x")
    rows, cols = x.shape
    out = empty_nvfp4(rows, cols, x.device, stream=stream) if out is None else out
    _check("nvfp4_quantize", lib().nvfp4_quantize(
        x.data_ptr(), rows, cols, amax.data_ptr(), out.q.data_ptr(), out.sf.data_ptr(),
        out.s_dec.data_ptr(), _stream(stream)))
    return out


def quantize_with_scale(x: torch.Tensor, s_enc: torch.Tensor, out: NVFP4Tensor | None = None,
                        stream=None) -> NVFP4Tensor:
    """NVFP4 quantization with a static per-tensor scale S_enc (device fp32)."""
    _require(x, torch.bfloat16, "x")
    rows, cols = x.shape
    out = empty_nvfp4(rows, cols, x.device, stream=stream) if out is None else out
    _check("nvfp4_quantize_with_scale", lib().nvfp4_quantize_with_scale(
        x.data_ptr(), rows, cols, s_enc.data_ptr(), out.q.data_ptr(), out.sf.data_ptr(),
        out.s_dec.data_ptr(), _stream(stream)))
    return out


def quantize_one_pass(x: torch.Tensor, amax_prev: torch.Tensor, amax_out: torch.Tensor,
                      out: NVFP4Tensor | None = None, stream=None) -> NVFP4Tensor:
    """One pass over x with the tensor scale derived from an earlier amax
    (amax_prev, device fp32); writes this tensor's amax into amax_out (a
    different device fp32) for the next call."""
    _require(x, torch.bfloat16, "x")
    rows, cols = x.shape
    out = empty_nvfp4(rows, cols, x.device, stream=stream) if out is None else out
    _check("nvfp4_quantize_one_pass", lib().nvfp4_quantize_one_pass(
        x.data_ptr(), rows, cols, amax_prev.data_ptr(), out.q.data_ptr(), out.sf.data_ptr(),
        out.s_dec.data_ptr(), amax_out.data_ptr(), _stream(stream)))
    return out


_dyn_workspaces: dict = {}


def dynamic_workspace(device=None) -> torch.Tensor:
    """A zero-filled workspace for nvfp4_quantize_dynamic (one per device,
    shared by calls on one stream; give concurrent streams their own)."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    ws = _dyn_workspaces.get(dev)
    if ws is None:
        n = int(lib().nvfp4_quantize_dynamic_workspace_bytes())
        ws = torch.zeros((n + 15) // 16 * 16, dtype=torch.uint8, device=dev)
        _dyn_workspaces[dev] = ws
    return ws


def quantize_dynamic(x: torch.Tensor, out: NVFP4Tensor | None = None,
                     amax: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                     stream=None) -> NVFP4Tensor:
    """Per-call activation path in one launch: amax, S_enc, block quantize."""
    _require(x, torch.bfloat16, "x")
    rows, cols = x.shape
    out = empty_nvfp4(rows, cols, x.device, stream=stream) if out is None else out
    ws = dynamic_workspace(x.device) if workspace is None else workspace
    _check("nvfp4_quantize_dynamic", lib().nvfp4_quantize_dynamic(
        x.data_ptr(), rows, cols, out.q.data_ptr(), out.sf.data_ptr(), out.s_dec.data_ptr(),
        _ptr(amax), ws.data_ptr(), _stream(stream)))
    return out


def quantize_rowwise(x: torch.Tensor, out: NVFP4Tensor | None = None,
                     amax_rows: torch.Tensor | None = None, stream=None) -> NVFP4Tensor:
    """Per-token activation scales: each row quantized with its own tensor
    scale 2688 / amax(row); out.s_dec holds one decode scale per row."""
    _require(x, torch.bfloat16, "x")
    rows, cols = x.shape
    out = empty_nvfp4(rows, cols, x.device, True, stream) if out is None else out
    if out.s_dec.numel() != rows:
        raise ValueError("out.s_dec must hold one scale per row")
    _check("nvfp4_quantize_rowwise", lib().nvfp4_quantize_rowwise(
        x.data_ptr(), rows, cols, out.q.data_ptr(), out.sf.data_ptr(), out.s_dec.data_ptr(),
        _ptr(amax_rows), _stream(stream)))
    return out


@dataclass
class FusedQuant:
    """Fused next-layer quantization outputs of a GEMM.  out is a complete
    NVFP4Tensor afterwards (out.s_dec = 1/s_enc is written by the GEMM), so it
    can feed the next GEMM directly."""
    s_enc: torch.Tensor           # fp32 [1], read
    out: NVFP4Tensor              # q [M, N/2], sf tiled, s_dec written
    amax: torch.Tensor | None     # fp32 [1], written with max|Y|
    activation: int = ACT_NONE    # ACT_GELU: Y = bf16(GELU(alpha * acc))


def gemm(a: NVFP4Tensor, b: NVFP4Tensor, y: torch.Tensor | None = None,
         fused: FusedQuant | None = None, want_y: bool = True, stream=None) -> torch.Tensor | None:
    """Y[M,N] = A[M,K] . B[N,K]^T on tcgen05 block-scaled FP4 tensor cores."""
    M, K = a.rows, a.cols
    N = b.rows
    if b.cols != K:
        raise ValueError("K mismatch")
    if y is None and want_y:
        y = _empty(torch.bfloat16, a.q.device, stream, M, N)
    fo = None
    if fused is not None:
        fo = FusedOut(fused.s_enc.data_ptr(), fused.out.q.data_ptr(), fused.out.sf.data_ptr(),
                      _ptr(fused.amax), fused.out.s_dec.data_ptr(), int(fused.activation))
    if b.s_dec.numel() != 1:
        raise ValueError("per-row scales are supported for A (activations) only")
    row_scaled = a.s_dec.numel() != 1
    if row_scaled and a.s_dec.numel() != M:
        raise ValueError("a.s_dec must hold 1 or M decode scales")
    fn = lib().nvfp4_gemm_rowscale if row_scaled else lib().nvfp4_gemm
    _check("nvfp4_gemm", fn(
        a.q.data_ptr(), a.sf.data_ptr(), a.s_dec.data_ptr(), b.q.data_ptr(), b.sf.data_ptr(),
        b.s_dec.data_ptr(), M, N, K, _ptr(y), ctypes.byref(fo) if fo is not None else None,
        _stream(stream)))
    return y


@dataclass
class FP8Tensor:
    """The FP8 variant's quantized [rows, cols] tensor: E4M3 codes and one
    decode scale."""
    q: torch.Tensor       # uint8 [rows, cols]
    s_dec: torch.Tensor   # float32 [1] = 1 / S_enc = amax / 448
    rows: int
    cols: int


def quantize_fp8(x: torch.Tensor, amax: torch.Tensor | None = None,
                 out: FP8Tensor | None = None, stream=None) -> FP8Tensor:
    """FP8 (E4M3) with one FP32 per-tensor scale 448 / amax; amax computed
    here (dynamic) unless given (static)."""
    _require(x, torch.bfloat16, "x")
    rows, cols = x.shape
    amax = tensor_amax(x, stream=stream) if amax is None else amax
    if out is None:
        out = FP8Tensor(_empty(torch.uint8, x.device, stream, rows, cols),
                        _empty(torch.float32, x.device, stream, 1), rows, cols)
    _check("nvfp4_fp8_quantize", lib().nvfp4_fp8_quantize(
        x.data_ptr(), rows, cols, amax.data_ptr(), out.q.data_ptr(), out.s_dec.data_ptr(),
        _stream(stream)))
    return out


def gemm_fp8(a: FP8Tensor, b: FP8Tensor, y: torch.Tensor | None = None,
             fused: FusedQuant | None = None, want_y: bool = True, stream=None):
    """Y[M,N] = A[M,K] . B[N,K]^T on tcgen05 FP8 (E4M3) tensor cores."""
    M, K, N = a.rows, a.cols, b.rows
    if b.cols != K:
        raise ValueError("K mismatch")
    if y is None and want_y:
        y = _empty(torch.bfloat16, a.q.device, stream, M, N)
    fo = None
    if fused is not None:
        fo = FusedOut(fused.s_enc.data_ptr(), fused.out.q.data_ptr(), fused.out.sf.data_ptr(),
                      _ptr(fused.amax), fused.out.s_dec.data_ptr(), int(fused.activation))
    _check("nvfp4_fp8_gemm", lib().nvfp4_fp8_gemm(
        a.q.data_ptr(), a.s_dec.data_ptr(), b.q.data_ptr(), b.s_dec.data_ptr(), M, N, K, _ptr(y),
        ctypes.byref(fo) if fo is not None else None, _stream(stream)))
    return y


class FP8Linear:
    """nn.Linear-shaped FP8 variant: weights quantized once (static scale),
    activations with a dynamic per-tensor scale on every call."""

    def __init__(self, weight: torch.Tensor):
        _require(weight, torch.bfloat16, "weight")
        self.N, self.K = weight.shape
        self.w = quantize_fp8(weight)

    def __call__(self, x: torch.Tensor, y: torch.Tensor | None = None,
                 fused: FusedQuant | None = None, want_y: bool = True,
                 adapters: LoraAdapters | None = None, row_slot: torch.Tensor | None = None):
        _adapters_need_y(adapters, row_slot, y, fused, want_y)
        y = gemm_fp8(quantize_fp8(x), self.w, y, fused, want_y)
        return y if adapters is None else lora(x, y, adapters, row_slot, out=y)


def _adapters_need_y(adapters, row_slot, y, fused, want_y) -> None:
    if adapters is None:
        if row_slot is not None:
            raise ValueError("row_slot needs adapters")
    elif fused is not None or (y is None and not want_y):
        raise ValueError("adapters are added to the bf16 output: fused codes would miss them")


SELFTEST_TAG = 90


def selftest_wait_timeout(timeout_us: int = 50_000, stream=None) -> None:
    """Failure-detection self-test: two kernels (the GEMM's waits, and those of the
    kernels around a projection) whose bounded waits can never be satisfied each
    give up after timeout_us; read the result with device_error()."""
    _check("nvfp4_selftest_wait_timeout",
           lib().nvfp4_selftest_wait_timeout(int(timeout_us), _stream(stream)))


class NVFP4Linear:
    """An nn.Linear-shaped NVFP4 layer: weights quantized once with a static
    per-tensor scale (from the weight amax, or a given one), activations
    quantized dynamically on every call.  adapters (with row_slot, one int32
    per row) adds the low-rank adapters of the rows' requests to the output;
    x may be given quantized already (xq, as residual_norm's quant), x itself
    then being read by the adapters only."""

    def __init__(self, weight: torch.Tensor, w_amax: torch.Tensor | None = None):
        _require(weight, torch.bfloat16, "weight")
        self.N, self.K = weight.shape
        amax = tensor_amax(weight) if w_amax is None else w_amax
        self.w = quantize(weight, amax)
        self._x = None

    def _xbuf(self, M: int, device) -> tuple[NVFP4Tensor, torch.Tensor]:
        if self._x is None or self._x[0].rows != M:
            self._x = (empty_nvfp4(M, self.K, device),
                       torch.empty(1, dtype=torch.float32, device=device))
        return self._x

    def __call__(self, x: torch.Tensor | None, y: torch.Tensor | None = None,
                 fused: FusedQuant | None = None, want_y: bool = True, *,
                 xq: NVFP4Tensor | None = None, adapters: LoraAdapters | None = None,
                 row_slot: torch.Tensor | None = None) -> torch.Tensor | None:
        _adapters_need_y(adapters, row_slot, y, fused, want_y)
        if xq is None:
            xq, amax = self._xbuf(x.shape[0], x.device)
            quantize_dynamic(x, xq, amax)
        elif x is None and adapters is not None:
            raise ValueError("adapters need x in bf16")
        y = gemm(xq, self.w, y, fused, want_y)
        return y if adapters is None else lora(x, y, adapters, row_slot, out=y)

    def forward_host(self, x_host: torch.Tensor, y_host: torch.Tensor, ws: dict,
                     stream=None, single_launch: bool = True) -> None:
        """Host bf16 X -> host bf16 Y through nvfp4_linear_host (copies included).
        single_launch=False passes no dynamic-quantize workspace, so the call
        quantizes X with nvfp4_tensor_amax + nvfp4_quantize."""
        M = x_host.shape[0]
        dyn = ws.get("dyn")
        if dyn is None:
            dyn = dynamic_workspace(ws["x"].device)
        w = LinearWorkspace(ws["x"].data_ptr(), ws["xq"].data_ptr(), ws["xsf"].data_ptr(),
                            ws["amax"].data_ptr(), ws["s_dec"].data_ptr(), ws["y"].data_ptr(),
                            dyn.data_ptr() if single_launch else None)
        _check("nvfp4_linear_host", lib().nvfp4_linear_host(
            x_host.data_ptr(), M, self.K, self.w.q.data_ptr(), self.w.sf.data_ptr(),
            self.w.s_dec.data_ptr(), self.N, y_host.data_ptr(), ctypes.byref(w),
            _stream(stream)))

    def host_workspace(self, M: int, device=None) -> dict:
        """Device buffers for forward_host, including a dynamic-quantize
        workspace of its own, so calls with different workspaces may run on
        different streams at the same time."""
        dev = torch.device("cuda") if device is None else device
        n = int(lib().nvfp4_quantize_dynamic_workspace_bytes())
        return {"dyn": torch.zeros((n + 15) // 16 * 16, dtype=torch.uint8, device=dev),
                "x": torch.empty(M, self.K, dtype=torch.bfloat16, device=dev),
                "xq": torch.empty(M, self.K // 2, dtype=torch.uint8, device=dev),
                "xsf": torch.empty(sf_bytes(M, self.K), dtype=torch.uint8, device=dev),
                "amax": torch.empty(1, dtype=torch.float32, device=dev),
                "s_dec": torch.empty(1, dtype=torch.float32, device=dev),
                "y": torch.empty(M, self.N, dtype=torch.bfloat16, device=dev)}


def _launch(name: str, args: bytes, index: int, stream) -> None:
    """Calls an entry point that takes a packed argument structure, on the
    tensors' device and its current stream (or the given one)."""
    raw = torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream
    fn = getattr(lib(), name)
    if index == torch.cuda.current_device():
        status = fn(args, raw)
    else:
        with torch.cuda.device(index):
            status = fn(args, raw)
    if status != 0:
        raise NVFP4Error(name, status)


def _row_stride(t: torch.Tensor, name: str, dtype, shape, index: int) -> int:
    """Elements from row to row of a [rows, cols] CUDA tensor whose rows are
    contiguous (a column slice of a wider tensor may be passed)."""
    if t.dtype is not dtype or t.shape != shape:
        raise ValueError(f"{name} must be a {dtype} {list(shape)} tensor")
    if t.get_device() != index:
        raise ValueError(f"{name} must be a CUDA tensor on the device of the others")
    stride, inner = t.stride()
    if inner != 1:
        raise ValueError(f"the rows of {name} must be contiguous")
    return stride if shape[0] > 1 else shape[1]


def _holds(t: torch.Tensor, dtype, count: int, index: int) -> bool:
    return t.dtype is dtype and t.numel() == count and t.get_device() == index and t.is_contiguous()


def _row_index(t: torch.Tensor, name: str, rows: int, index: int) -> int:
    if not _holds(t, torch.int32, rows, index):
        raise ValueError(f"{name} must hold one int32 per row, on the device of the others")
    return t.data_ptr()


def _cuda_index(t: torch.Tensor, name: str) -> int:
    index = t.get_device()
    if index < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    return index


@dataclass(slots=True)
class Norm:
    """A norm over the columns: kind "rms" or "layer", optional weight and bias."""
    kind: str = "rms"
    weight: torch.Tensor | None = None
    bias: torch.Tensor | None = None
    eps: float = 1e-6


_NORM_KINDS = {"rms": 1, "layer": 2}      # nvfp4_norm values
_DTYPES = {torch.bfloat16: 0, torch.float32: 1}  # nvfp4_dtype values


def _norm_kind(norm: Norm) -> int:
    kind = _NORM_KINDS.get(norm.kind)
    if kind is None:
        raise ValueError("a norm is 'rms' or 'layer'")
    return kind


def _vector(t: torch.Tensor, name: str, dtype, cols: int, index: int, groups: int) -> tuple[int, int, int]:
    """(pointer, elements from request to request, requests) of a weight or
    modulation vector; groups: the requests known so far, 0 where the vector
    cannot have any of its own."""
    if t.dtype is not dtype or dtype not in _DTYPES:
        raise ValueError("weights, biases, gate, scale and shift must all be bf16 or all fp32")
    size, strides = t.shape, t.stride()
    if t.get_device() != index or not size or size[-1] != cols or strides[-1] != 1:
        raise ValueError(f"{name} must hold {cols} contiguous values, on the device of the others")
    if len(size) == 1 or (groups and len(size) == 2 and size[0] == 1):
        return t.data_ptr(), 0, groups
    if not groups or len(size) != 2 or groups not in (1, size[0]) or not size[0]:
        raise ValueError(f"{name} must be [cols]" +
                         (" or [groups, cols], with the same groups for all" if groups else ""))
    return t.data_ptr(), strides[0], size[0]


class ResidualNorm(NamedTuple):
    """Results of residual_norm; what was not asked for is None."""
    h: torch.Tensor | None
    out: torch.Tensor | None
    quant: NVFP4Tensor | None


def residual_norm(residual: torch.Tensor, y: torch.Tensor | None = None, *,
                  post: Norm | None = None, gate: torch.Tensor | None = None,
                  pre: Norm | None = None, scale: torch.Tensor | None = None,
                  shift: torch.Tensor | None = None, row_group: torch.Tensor | None = None,
                  residual_scale: float = 1.0, branch_scale: float = 1.0,
                  h: torch.Tensor | None = None, want_h: bool = True,
                  out: torch.Tensor | None = None, want_out: bool = True,
                  quant: NVFP4Tensor | None = None, want_quant: bool = False,
                  amax_rows: torch.Tensor | None = None, stream=None) -> ResidualNorm:
    """The norms after one block and before the next, in one launch.  Per row,
    with g the row's request:

        h     = residual_scale * residual + branch_scale * gate[g] * post(y)
        out   = pre(h) * (1 + scale[g]) + shift[g]
        quant = quantize_rowwise(out)

    residual: [rows, cols] bf16 or fp32 (h has its type); y: [rows, cols] bf16,
    or None at the start of a model; cols a multiple of 16, at most 32768.
    gate, scale, shift: [cols], or [groups, cols] with any row stride that is a
    multiple of 8 (chunks of one modulation tensor); beside vectors of several
    groups [1, cols] is one for all.  Weights, biases, gate, scale and shift are
    all bf16 or all fp32.  row_group: int32 per row, its request; rows with a
    negative number, or one not below groups where a vector has groups, are
    padding, and their results are left as they were (in tensors that the call
    makes, whatever the memory held: give zeroed ones where a per-tensor quantize
    or the like will see those rows).  Without it each request has rows / groups
    consecutive rows.  h, out and quant may be given; h may be the residual itself.
    Without pre, only h is computed."""
    if residual.dim() != 2 or residual.dtype not in _DTYPES:
        raise ValueError("residual must be a bf16 or fp32 [rows, cols] tensor")
    stream_type, shape, bf16 = residual.dtype, residual.shape, torch.bfloat16
    rows, cols = shape
    dev = _cuda_index(residual, "residual")
    r_stride = _row_stride(residual, "residual", stream_type, shape, dev)
    y_ptr = y_stride = h_ptr = h_stride = out_ptr = out_stride = 0
    q_ptr = sf_ptr = s_dec_ptr = amax_ptr = 0
    if y is not None:
        y_stride = _row_stride(y, "y", bf16, shape, dev)
        y_ptr = y.data_ptr()
        if h is None and want_h:
            h = _empty(stream_type, residual.device, stream, rows, cols)
    elif post is not None or gate is not None or h is not None:
        raise ValueError("post, gate and h need y")
    if h is not None:
        h_stride = _row_stride(h, "h", stream_type, shape, dev)
        h_ptr = h.data_ptr()
    if pre is None:
        if scale is not None or shift is not None or out is not None or quant is not None or want_quant:
            raise ValueError("scale, shift, out and quant need pre")
    else:
        if out is None and want_out:
            out = _empty(bf16, residual.device, stream, rows, cols)
        if out is not None:
            out_stride = _row_stride(out, "out", bf16, shape, dev)
            out_ptr = out.data_ptr()
            if out_ptr == h_ptr and rows:
                raise ValueError("h and out must not be the same memory")
        if quant is None and want_quant:
            quant = empty_nvfp4(rows, cols, residual.device, True, stream)
        elif quant is not None:
            if not (quant.rows == rows and quant.cols == cols and
                    _holds(quant.q, torch.uint8, rows * cols // 2, dev) and
                    _holds(quant.sf, torch.uint8, sf_bytes(rows, cols), dev) and
                    _holds(quant.s_dec, torch.float32, rows, dev)):
                raise ValueError("quant must be a contiguous NVFP4Tensor of these rows and columns with "
                                 "row scales, on the device of the others")
        if quant is not None:
            q_ptr, sf_ptr, s_dec_ptr = quant.q.data_ptr(), quant.sf.data_ptr(), quant.s_dec.data_ptr()
    if amax_rows is not None:
        if quant is None or not _holds(amax_rows, torch.float32, rows, dev):
            raise ValueError("amax_rows must hold one fp32 per row, and needs quant")
        amax_ptr = amax_rows.data_ptr()

    vec_type, groups = None, 1
    post_kind = pre_kind = post_w = post_b = pre_w = pre_b = 0
    post_eps = pre_eps = 0.0
    gate_ptr = gate_stride = scale_ptr = scale_stride = shift_ptr = shift_stride = 0
    if post is not None:
        post_kind, post_eps = _norm_kind(post), post.eps
        if post.weight is not None:
            vec_type = post.weight.dtype
            post_w = _vector(post.weight, "post.weight", vec_type, cols, dev, 0)[0]
        if post.bias is not None:
            vec_type = vec_type or post.bias.dtype
            post_b = _vector(post.bias, "post.bias", vec_type, cols, dev, 0)[0]
    if pre is not None:
        pre_kind, pre_eps = _norm_kind(pre), pre.eps
        if pre.weight is not None:
            vec_type = vec_type or pre.weight.dtype
            pre_w = _vector(pre.weight, "pre.weight", vec_type, cols, dev, 0)[0]
        if pre.bias is not None:
            vec_type = vec_type or pre.bias.dtype
            pre_b = _vector(pre.bias, "pre.bias", vec_type, cols, dev, 0)[0]
    if gate is not None:
        vec_type = vec_type or gate.dtype
        gate_ptr, gate_stride, groups = _vector(gate, "gate", vec_type, cols, dev, groups)
    if scale is not None:
        vec_type = vec_type or scale.dtype
        scale_ptr, scale_stride, groups = _vector(scale, "scale", vec_type, cols, dev, groups)
    if shift is not None:
        vec_type = vec_type or shift.dtype
        shift_ptr, shift_stride, groups = _vector(shift, "shift", vec_type, cols, dev, groups)
    index = 0
    if row_group is not None:
        index = _row_index(row_group, "row_group", rows, dev)
        if groups == 1 and all(v is None or v.dim() == 1 for v in (gate, scale, shift)):
            groups = 1 << 31  # no vector of a request's own: every number from 0 on is one
    args = _pack_residual_norm(
        rows, cols, residual.data_ptr(), r_stride, y_ptr, y_stride, h_ptr, h_stride, out_ptr, out_stride,
        post_w, post_b, pre_w, pre_b, gate_ptr, gate_stride, scale_ptr, scale_stride, shift_ptr, shift_stride,
        index, groups, q_ptr, sf_ptr, s_dec_ptr, amax_ptr, residual_scale, branch_scale, post_eps, pre_eps,
        post_kind, pre_kind, _DTYPES[stream_type], 0 if vec_type is None else _DTYPES[vec_type])
    _launch("nvfp4_residual_norm", args, dev, stream)
    return ResidualNorm(h, out, quant)


@dataclass(slots=True)
class LoraAdapters:
    """Low-rank adapters of one projection, held side by side: slot s adds
    scale[s] * B[s] (A[s] x).  One rank for all, a multiple of 16 up to 128;
    pack_adapters pads smaller ones."""
    a: torch.Tensor      # bf16 [slots, rank, K]
    b: torch.Tensor      # bf16 [slots, N, rank]
    scale: torch.Tensor  # fp32 [slots]


def pack_adapters(adapters, device=None) -> LoraAdapters:
    """LoraAdapters from a list of (A [r, K], B [N, r], scale), whose ranks may
    differ: each is padded with zeros to the largest one's next multiple of 16
    (and an x that is not finite times those zeros makes its row NaN)."""
    if not adapters:
        raise ValueError("pack_adapters needs at least one adapter")
    k, n = adapters[0][0].shape[1], adapters[0][1].shape[0]
    for a, b, _ in adapters:
        if a.dim() != 2 or b.dim() != 2 or a.shape[1] != k or b.shape[0] != n or a.shape[0] != b.shape[1]:
            raise ValueError("each adapter is (A [r, K], B [N, r], scale), with the same K and N for all")
    rank = max(16, (max(a.shape[0] for a, _, _ in adapters) + 15) // 16 * 16)
    if rank > 128:
        raise ValueError("ranks up to 128 are supported")
    dev = adapters[0][0].device if device is None else device
    pa = torch.zeros(len(adapters), rank, k, dtype=torch.bfloat16, device=dev)
    pb = torch.zeros(len(adapters), n, rank, dtype=torch.bfloat16, device=dev)
    for i, (a, b, _) in enumerate(adapters):
        pa[i, :a.shape[0]] = a
        pb[i, :, :a.shape[0]] = b
    scale = torch.tensor([float(s) for _, _, s in adapters], dtype=torch.float32, device=dev)
    return LoraAdapters(pa, pb, scale)


def lora(x: torch.Tensor, y: torch.Tensor, adapters: LoraAdapters,
         row_slot: torch.Tensor | None = None, out: torch.Tensor | None = None,
         workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """out[m] = y[m] + scale[s] * B[s] (A[s] x[m]) with s = row_slot[m], the
    low-rank adapters of many requests beside a projection y they share.

    x: [rows, K] and y: [rows, N], bf16 (K % 16 == 0, N % 8 == 0; rows may be
    strided by a multiple of 8 elements).  row_slot: int32 per row, in any
    order; a number outside [0, slots) means no adapter (out = y).  None: slot 0
    for every row.  out may be y itself (but not share memory with x or, row on
    other rows, with y); a new tensor if not given.  workspace:
    nvfp4_lora_workspace_bytes of memory for calls that follow one another; the
    call's own if not given."""
    a, b, scale = adapters.a, adapters.b, adapters.scale
    bf16, dev = torch.bfloat16, _cuda_index(x, "x")
    if a.dim() != 3 or b.dim() != 3 or x.dim() != 2:
        raise ValueError("x is [rows, K], adapters.a [slots, rank, K], adapters.b [slots, N, rank]")
    slots, rank, k = a.shape
    rows, n = x.shape[0], b.shape[1]
    if (a.dtype is not bf16 or b.dtype is not bf16 or scale.dtype is not torch.float32 or
            b.shape != (slots, n, rank) or scale.shape != (slots,) or
            not (a.is_contiguous() and b.is_contiguous() and scale.is_contiguous()) or
            a.get_device() != dev or b.get_device() != dev or scale.get_device() != dev):
        raise ValueError("adapters must be contiguous bf16 a [slots, rank, K] and b [slots, N, rank] "
                         "and fp32 scale [slots], on the device of x")
    x_stride = _row_stride(x, "x", bf16, (rows, k), dev)
    y_stride = _row_stride(y, "y", bf16, (rows, n), dev)
    if out is None:
        out = _empty(bf16, x.device, stream, rows, n)
    out_stride = y_stride if out is y else _row_stride(out, "out", bf16, (rows, n), dev)
    index = 0 if row_slot is None else _row_index(row_slot, "row_slot", rows, dev)
    need = lib().nvfp4_lora_workspace_bytes(rows, k, n, rank)
    if need and workspace is None:
        # Of the stream it is used on, so that it is free again in that stream's order.
        with torch.cuda.stream(stream):
            workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    elif need and (workspace.get_device() != dev or not workspace.is_contiguous() or
                   workspace.numel() * workspace.element_size() < need):
        raise ValueError(f"workspace must hold {need} contiguous bytes on the device of x")
    args = _pack_lora(rows, k, n, rank, slots, x.data_ptr(), x_stride, y.data_ptr(), y_stride,
                      out.data_ptr(), out_stride, a.data_ptr(), b.data_ptr(), scale.data_ptr(), index,
                      workspace.data_ptr() if need else 0)
    _launch("nvfp4_lora", args, dev, stream)
    return out


def device_error() -> tuple[int, int]:
    """(code, detail) of the device error word, cleared on read (synchronises)."""
    c, d = ctypes.c_int(0), ctypes.c_int(0)
    _check("nvfp4_device_error", lib().nvfp4_device_error(ctypes.byref(c), ctypes.byref(d)))
    return c.value, d.value


def status_string(status: int) -> str:
    return lib().nvfp4_status_string(status).decode()
