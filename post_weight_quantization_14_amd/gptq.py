"""Python binding of the C ABI: the same entry points, taking torch tensors.

Argument marshalling only: tensors become device pointers, sizes and strides
become integers, the stream is torch's current HIP stream.  Every step of the
path runs in the HIP kernels of libgptq_mi355x.so; a non-OK status raises
GptqError carrying the library's message.
"""
from __future__ import annotations

import contextlib
import ctypes
from dataclasses import dataclass
from typing import Optional

import torch

from . import _lib
from ._lib import GptqConfig, lib


class GptqError(RuntimeError):
    def __init__(self, status: int, where: str):
        msg = lib().gptq_last_error().decode(errors="replace")
        super().__init__(f"{where}: {_lib.STATUS_NAMES.get(status, status)}: {msg}")
        self.status = status


@dataclass
class QuantConfig:
    """Quantizer settings (bits, group_size, sym, desc_act, damp_percent)."""
    bits: int = 4
    group_size: int = 128
    sym: bool = False
    desc_act: bool = True
    damp_percent: float = 0.01
    block_size: int = 128

    def c(self) -> GptqConfig:
        return GptqConfig(int(self.bits), int(self.group_size), int(bool(self.sym)),
                          int(bool(self.desc_act)), int(self.block_size), float(self.damp_percent))


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return _lib.GPTQ_BF16
    if t.dtype == torch.float32:
        return _lib.GPTQ_FP32
    raise TypeError(f"unsupported dtype {t.dtype}")


def _check(status: int, where: str) -> None:
    if status != _lib.GPTQ_OK:
        raise GptqError(status, where)


def _workspace(nbytes: int, device, workspace: Optional[torch.Tensor]) -> Optional[torch.Tensor]:
    if nbytes == 0:
        return workspace
    if workspace is not None and workspace.numel() * workspace.element_size() >= nbytes:
        return workspace
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


# ---------------------------------------------------------------- sizes
def gptq_hessian_workspace_bytes(n: int, tokens: int, x_dtype: int = _lib.GPTQ_BF16) -> int:
    return int(lib().gptq_hessian_workspace_bytes(n, tokens, x_dtype))


def gptq_prepare_workspace_bytes(n: int) -> int:
    return int(lib().gptq_prepare_workspace_bytes(n))


def gptq_quantize_workspace_bytes(m: int, n: int, cfg: QuantConfig) -> int:
    c = cfg.c()
    return int(lib().gptq_quantize_workspace_bytes(m, n, ctypes.byref(c)))


def gptq_qweight_words(n: int, bits: int) -> int:
    return int(lib().gptq_qweight_words(n, bits))


def gptq_num_groups(n: int, group_size: int) -> int:
    return int(lib().gptq_num_groups(n, group_size))


def gptq_last_error() -> str:
    return lib().gptq_last_error().decode(errors="replace")


# ---------------------------------------------------------------- stages
def gptq_hessian_accumulate(H: torch.Tensor, diag_key: Optional[torch.Tensor], X: torch.Tensor,
                            alpha: float = 2.0, workspace: Optional[torch.Tensor] = None,
                            stream=None) -> None:
    """H += alpha·XᵀX, diag_key += alpha·Σx² (fp64), for X [tokens, n] with unit column stride."""
    n = H.shape[0]
    if X.dim() != 2 or X.shape[1] != n or (X.shape[0] > 0 and X.stride(1) != 1):
        raise ValueError("X must be [tokens, n] with contiguous rows")
    code = _dtype_code(X)
    ws = _workspace(gptq_hessian_workspace_bytes(n, X.shape[0], code), H.device, workspace)
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    st = lib().gptq_hessian_accumulate(_ptr(H), _ptr(diag_key), n, _ptr(X), code, X.shape[0],
                                       X.stride(0) if X.shape[0] > 0 else n, float(alpha),
                                       _ptr(ws), nbytes, _stream(stream))
    _check(st, "gptq_hessian_accumulate")


def gptq_prepare_hinv(H: torch.Tensor, diag_key: Optional[torch.Tensor], damp_percent: float,
                      desc_act: bool, perm_out: torch.Tensor,
                      workspace: Optional[torch.Tensor] = None, stream=None) -> float:
    """H (in place) -> U; fills perm_out; returns the damping λ."""
    n = H.shape[0]
    ws = _workspace(gptq_prepare_workspace_bytes(n), H.device, workspace)
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    lam = ctypes.c_double(0.0)
    st = lib().gptq_prepare_hinv(_ptr(H), _ptr(diag_key), n, float(damp_percent), int(bool(desc_act)),
                                 _ptr(perm_out), _ptr(ws), nbytes, ctypes.byref(lam), _stream(stream))
    _check(st, "gptq_prepare_hinv")
    return lam.value


def gptq_quantize_layer(W: torch.Tensor, U: torch.Tensor, perm: torch.Tensor, cfg: QuantConfig,
                        qweight: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor,
                        g_idx: torch.Tensor, loss: torch.Tensor, status: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """Enqueue the quantization; never synchronises.  `status` (int32 [1] on
    the device, optional) receives 0 or GPTQ_ERR_NONFINITE in stream order:
    read it with check_status()."""
    if not W.is_contiguous():
        raise ValueError("W must be contiguous [m, n]")
    m, n = W.shape
    c = cfg.c()
    ws = _workspace(gptq_quantize_workspace_bytes(m, n, cfg), W.device, workspace)
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    st = lib().gptq_quantize_layer(_ptr(W), _dtype_code(W), m, n, _ptr(U), _ptr(perm), ctypes.byref(c),
                                   _ptr(qweight), _ptr(scales), _ptr(zeros), _ptr(g_idx), _ptr(loss),
                                   _ptr(status), _ptr(ws), nbytes, _stream(stream))
    _check(st, "gptq_quantize_layer")


def check_status(*outs) -> None:
    """Read the device status words of earlier quantizations (one host
    synchronisation for all of them) and raise GptqError for the first that
    is not GPTQ_OK.  Each argument is an output dict of quantize_layer /
    quantize_shared_input, or a list of them."""
    flat = []
    for o in outs:
        if isinstance(o, dict):
            flat.append(o)
        else:
            for x in o:
                flat.extend(x if isinstance(x, list) else [x])
    if not flat:
        return
    words = torch.cat([o["status"] for o in flat]).cpu().tolist()
    for w in words:
        if w != _lib.GPTQ_OK:
            lib().gptq_last_error()   # keeps the message API uniform
            raise GptqError(int(w), "gptq_quantize_layer (status word)")


# ---------------------------------------------------------------- linear (RTN) quantizer
@dataclass
class RtnConfig:
    """Settings of gptq_rtn_quantize: bits 2/3/4/8; group_size -1 (one group
    per output row) or >= 1; sym; clip_ratio in (0, 1]."""
    bits: int = 8
    group_size: int = -1
    sym: bool = True
    clip_ratio: float = 0.99

    def c(self) -> "_lib.GptqRtnConfig":
        return _lib.GptqRtnConfig(self.bits, self.group_size, int(self.sym), self.clip_ratio)


def gptq_rtn_workspace_bytes(m: int, n: int, cfg: RtnConfig) -> int:
    c = cfg.c()
    return int(lib().gptq_rtn_workspace_bytes(m, n, ctypes.byref(c)))


def _status_word(status: Optional[torch.Tensor], check: bool, device) -> Optional[torch.Tensor]:
    if status is None and check:
        status = torch.zeros(1, dtype=torch.int32, device=device)
    return status


def _read_status(status: torch.Tensor, where: str) -> None:
    """Synchronise on the device status word and raise on a non-OK status."""
    w = int(status.item())
    if w != _lib.GPTQ_OK:
        raise GptqError(w, f"{where} (status word: the input holds a NaN or Inf)")


def gptq_rtn_quantize(W: torch.Tensor, cfg: RtnConfig, qweight: torch.Tensor, scales: torch.Tensor,
                      zeros: torch.Tensor, err: torch.Tensor, workspace: Optional[torch.Tensor] = None,
                      stream=None, status: Optional[torch.Tensor] = None, check: bool = True) -> None:
    """Enqueue the quantizer (the call itself never synchronises).  check=True
    reads the device status word afterwards and raises on a NaN/Inf in W;
    check=False leaves it in `status` (int32 [1]) for the caller."""
    if not W.is_contiguous():
        raise ValueError("W must be contiguous [m, n]")
    m, n = W.shape
    c = cfg.c()
    ws = _workspace(gptq_rtn_workspace_bytes(m, n, cfg), W.device, workspace)
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    status = _status_word(status, check, W.device)
    st = lib().gptq_rtn_quantize(_ptr(W), _dtype_code(W), m, n, ctypes.byref(c), _ptr(qweight),
                                 _ptr(scales), _ptr(zeros), _ptr(err), _ptr(status), _ptr(ws), nbytes,
                                 _stream(stream))
    _check(st, "gptq_rtn_quantize")
    if check and m > 0 and n > 0:
        _read_status(status, "gptq_rtn_quantize")


def rtn_quantize(W: torch.Tensor, cfg: RtnConfig) -> dict:
    """Allocate the outputs and run gptq_rtn_quantize on W [m, n]."""
    m, n = W.shape
    dev = W.device
    # sizes of an invalid config come back negative: allocate nothing and let
    # the library report the config
    words = max(gptq_qweight_words(n, cfg.bits), 0)
    groups = max(gptq_num_groups(n, cfg.group_size), 0)
    out = dict(
        qweight=torch.empty(m, words, dtype=torch.int32, device=dev),
        scales=torch.empty(m, groups, dtype=torch.float32, device=dev),
        zeros=torch.empty(m, groups, dtype=torch.int32, device=dev),
        err=torch.zeros(2, dtype=torch.float64, device=dev),
    )
    gptq_rtn_quantize(W, cfg, out["qweight"], out["scales"], out["zeros"], out["err"])
    return out


# ---------------------------------------------------------------- AWQ channel scaling
def gptq_awq_stats_workspace_bytes(n: int, tokens: int) -> int:
    return int(lib().gptq_awq_stats_workspace_bytes(n, tokens))


def gptq_awq_channel_stats(X: torch.Tensor, abs_sum: torch.Tensor, workspace: Optional[torch.Tensor] = None,
                           stream=None) -> None:
    """abs_sum [n] fp64 += Σ_t |X[t]| for X [tokens, n] (bf16 or fp32) with contiguous rows."""
    if X.dim() != 2 or (X.shape[0] > 0 and X.stride(1) != 1):
        raise ValueError("X must be [tokens, n] with contiguous rows")
    tokens, n = X.shape
    ws = _workspace(gptq_awq_stats_workspace_bytes(n, tokens), X.device, workspace)
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    st = lib().gptq_awq_channel_stats(_ptr(X), _dtype_code(X), tokens, X.stride(0) if tokens > 0 else n, n,
                                      _ptr(abs_sum), _ptr(ws), nbytes, _stream(stream))
    _check(st, "gptq_awq_channel_stats")


def gptq_awq_workspace_bytes(m: int, n: int, cfg: RtnConfig) -> int:
    c = cfg.c()
    return int(lib().gptq_awq_workspace_bytes(m, n, ctypes.byref(c)))


def gptq_awq_quantize(W: torch.Tensor, abs_sum: torch.Tensor, tokens: int, protect: float, cfg: RtnConfig,
                      qweight: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor,
                      channel_scale: torch.Tensor, err: torch.Tensor, workspace: Optional[torch.Tensor] = None,
                      stream=None, status: Optional[torch.Tensor] = None, check: bool = True) -> None:
    """Enqueue the AWQ-scaled quantizer (never synchronises by itself);
    check as in gptq_rtn_quantize (NaN/Inf in W or in abs_sum)."""
    if not W.is_contiguous():
        raise ValueError("W must be contiguous [m, n]")
    m, n = W.shape
    c = cfg.c()
    ws = _workspace(gptq_awq_workspace_bytes(m, n, cfg), W.device, workspace)
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    status = _status_word(status, check, W.device)
    st = lib().gptq_awq_quantize(_ptr(W), _dtype_code(W), m, n, _ptr(abs_sum), tokens, float(protect),
                                 ctypes.byref(c), _ptr(qweight), _ptr(scales), _ptr(zeros), _ptr(channel_scale),
                                 _ptr(err), _ptr(status), _ptr(ws), nbytes, _stream(stream))
    _check(st, "gptq_awq_quantize")
    if check and m > 0 and n > 0:
        _read_status(status, "gptq_awq_quantize")


def awq_quantize(W: torch.Tensor, x_tiles, cfg: RtnConfig, protect: float = 2.0) -> dict:
    """Channel statistics over every X tile, then gptq_awq_quantize on W [m, n]."""
    m, n = W.shape
    dev = W.device
    abs_sum = torch.zeros(n, dtype=torch.float64, device=dev)
    tokens = 0
    for X in x_tiles:
        gptq_awq_channel_stats(X, abs_sum)
        tokens += X.shape[0]
    words = max(gptq_qweight_words(n, cfg.bits), 0)
    groups = max(gptq_num_groups(n, cfg.group_size), 0)
    out = dict(
        qweight=torch.empty(m, words, dtype=torch.int32, device=dev),
        scales=torch.empty(m, groups, dtype=torch.float32, device=dev),
        zeros=torch.empty(m, groups, dtype=torch.int32, device=dev),
        channel_scale=torch.empty(n, dtype=torch.float32, device=dev),
        err=torch.zeros(2, dtype=torch.float64, device=dev),
        abs_sum=abs_sum,
        tokens=tokens,
    )
    gptq_awq_quantize(W, abs_sum, tokens, protect, cfg, out["qweight"], out["scales"], out["zeros"],
                      out["channel_scale"], out["err"])
    return out


# ---------------------------------------------------------------- W4A16 product
def _torch_stream(stream, device) -> torch.cuda.Stream:
    """torch's object of a stream that is given as one or as its handle."""
    if isinstance(stream, torch.cuda.Stream):
        return stream
    handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    # ExternalStream(0) is not the default stream but a new one of torch's
    return torch.cuda.ExternalStream(handle, device=device) if handle else torch.cuda.default_stream(device)


def _new_packed(nbytes: int, like: torch.Tensor, stream) -> torch.Tensor:
    """Memory for a packed weight.  It outlives the call, so it is the current
    stream's; a pack on another stream waits until the current one is done with
    what was there before."""
    packed = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=like.device)
    if stream is not None and like.is_cuda:
        _torch_stream(stream, like.device).wait_stream(torch.cuda.current_stream(like.device))
    return packed


def gptq_w4a16_packed_bytes(m: int, n: int, group_size: int) -> int:
    return int(lib().gptq_w4a16_packed_bytes(m, n, group_size))


def gptq_w4a16_pack(qweight: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor,
                    g_idx: torch.Tensor, n: int, bits: int, group_size: int,
                    packed: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The quantizer's output of an m x n weight -> the product's layout (uint8 tensor)."""
    m = qweight.shape[0]
    nbytes = gptq_w4a16_packed_bytes(m, n, group_size)
    if packed is None:
        packed = _new_packed(nbytes, qweight, stream)
    st = lib().gptq_w4a16_pack(_ptr(qweight), _ptr(scales), _ptr(zeros), _ptr(g_idx), m, n, bits,
                               group_size, _ptr(packed), packed.numel() * packed.element_size(),
                               _stream(stream))
    _check(st, "gptq_w4a16_pack")
    return packed


def gptq_checkpoint_qweight_rows(n: int, bits: int) -> int:
    return int(lib().gptq_checkpoint_qweight_rows(n, bits))


def gptq_checkpoint_qzeros_words(m: int, bits: int) -> int:
    return int(lib().gptq_checkpoint_qzeros_words(m, bits))


def gptq_export_checkpoint(qweight: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor, n: int,
                           bits: int, group_size: int, zero_offset: int = 0, stream=None) -> dict:
    """The quantizer's output of an m x n weight -> the checkpoint tensors
    {"qweight": int32 [ceil(n·bits/32), m], "qzeros": int32 [G, ceil(m·bits/32)],
    "scales": float16 [G, m]} (g_idx is the quantizer's own)."""
    m = qweight.shape[0]
    G = gptq_num_groups(n, group_size)
    rows = gptq_checkpoint_qweight_rows(n, bits)
    zw = gptq_checkpoint_qzeros_words(m, bits)
    if G < 0 or rows < 0 or zw < 0:
        raise ValueError(f"bits={bits} group_size={group_size} n={n}")
    dev = qweight.device
    out = {"qweight": torch.empty(rows, m, dtype=torch.int32, device=dev),
           "qzeros": torch.empty(G, zw, dtype=torch.int32, device=dev),
           "scales": torch.empty(G, m, dtype=torch.float16, device=dev)}
    st = lib().gptq_export_checkpoint(_ptr(qweight), _ptr(scales), _ptr(zeros), m, n, bits, group_size,
                                      zero_offset, _ptr(out["qweight"]), _ptr(out["qzeros"]),
                                      _ptr(out["scales"]), _stream(stream))
    _check(st, "gptq_export_checkpoint")
    return out


def gptq_w4a16_workspace_bytes(tokens: int, m: int, n: int) -> int:
    return int(lib().gptq_w4a16_workspace_bytes(tokens, m, n))


def gptq_w4a16_matmul(X: torch.Tensor, packed: torch.Tensor, m: int, n: int, group_size: int,
                      Y: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                      stream=None) -> torch.Tensor:
    """Y [tokens, m] fp32 = X [tokens, n] bf16 · Ŵᵀ from a packed weight."""
    if X.dim() != 2 or X.shape[1] != n or (X.shape[0] > 0 and X.stride(1) != 1):
        raise ValueError("X must be [tokens, n] with contiguous rows")
    tokens = X.shape[0]
    if Y is None:
        Y = torch.empty(tokens, m, dtype=torch.float32, device=X.device)
    ws = _workspace(gptq_w4a16_workspace_bytes(tokens, m, n), X.device, workspace)
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    st = lib().gptq_w4a16_matmul(_ptr(X), tokens, X.stride(0) if tokens > 0 else n, _ptr(packed), m, n,
                                 group_size, _ptr(Y), Y.stride(0) if tokens > 0 else m, _ptr(ws), nbytes,
                                 _stream(stream))
    _check(st, "gptq_w4a16_matmul")
    return Y


def gptq_w4a16_matmul_noalloc(X: torch.Tensor, packed: torch.Tensor, m: int, n: int, group_size: int,
                              Y: torch.Tensor, stream=None) -> torch.Tensor:
    """gptq_w4a16_matmul on the library's own device scratch (no workspace;
    the C call allocates nothing).  Y [tokens, m] fp32 must be given."""
    if X.dim() != 2 or X.shape[1] != n or (X.shape[0] > 0 and X.stride(1) != 1):
        raise ValueError("X must be [tokens, n] with contiguous rows")
    tokens = X.shape[0]
    st = lib().gptq_w4a16_matmul_noalloc(_ptr(X), tokens, X.stride(0) if tokens > 0 else n, _ptr(packed), m, n,
                                         group_size, _ptr(Y), Y.stride(0) if tokens > 0 else m, _stream(stream))
    _check(st, "gptq_w4a16_matmul_noalloc")
    return Y


# ---------------------------------------------------------------- layers on packed weights
def _activation_code(name: str) -> int:
    try:
        return _lib.ACTIVATIONS[name]
    except KeyError:
        raise ValueError(f"activation {name!r}: one of {', '.join(_lib.ACTIVATIONS)}") from None


def _on(X: torch.Tensor, **tensors: Optional[torch.Tensor]) -> None:
    """Every tensor of a call lives on X's GPU (a pointer of another device,
    or of the host, would be read by the kernels as it is)."""
    if not X.is_cuda:
        raise ValueError("X must be on the GPU")
    dev = X.get_device()
    for name, t in tensors.items():
        if t is not None and t.get_device() != dev:
            raise ValueError(f"{name} is on {t.device}, X on {X.device}")


def _rows(name: str, t: torch.Tensor, rows: int, cols: int) -> int:
    """The row stride of a [rows, cols] tensor with contiguous rows."""
    if t.dim() != 2 or t.shape[0] != rows or t.shape[1] != cols or (cols > 1 and rows > 0 and t.stride(1) != 1):
        raise ValueError(f"{name} must be [{rows}, {cols}] with contiguous rows")
    return t.stride(0) if rows > 1 else cols


def _vector(name: str, t: Optional[torch.Tensor], m: int) -> Optional[int]:
    if t is None:
        return None
    if t.dim() != 1 or t.shape[0] != m or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous [{m}]")
    return t.data_ptr()


# the handle of a device's current stream, without building a Stream object
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_on(X: torch.Tensor, stream) -> Optional[int]:
    """The given stream, or the current stream of X's device."""
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(X.device.index)
        stream = torch.cuda.current_stream(X.device)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _bf16_rows(X: torch.Tensor, n: int) -> int:
    if X.dim() != 2 or X.shape[1] != n or (X.shape[0] > 0 and n > 1 and X.stride(1) != 1):
        raise ValueError(f"X must be [tokens, {n}] with contiguous rows")
    if X.dtype != torch.bfloat16:
        raise TypeError(f"X must be bfloat16, not {X.dtype}")
    return X.stride(0) if X.shape[0] > 1 else n


def _uint8(name: str, t: torch.Tensor) -> int:
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.nbytes


def _empty(shape, dtype: torch.dtype, X: torch.Tensor, stream) -> torch.Tensor:
    """A new tensor whose memory the stream of the call may write at once: torch
    hands out memory that is free in the order of the stream it is asked on."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=X.device)
    with torch.cuda.stream(_torch_stream(stream, X.device)):
        return torch.empty(shape, dtype=dtype, device=X.device)


def _with_workspace(call, nbytes, X: torch.Tensor, workspace: Optional[torch.Tensor], stream, where: str) -> None:
    """call(pointer, bytes) -> status on the caller's workspace (it then belongs
    to this call until its work is done), or on a new one of nbytes() bytes if
    there is none or the library finds it too small or misaligned."""
    if workspace is not None:
        st = call(workspace.data_ptr(), _uint8("workspace", workspace))
        if st != _lib.GPTQ_ERR_WORKSPACE:
            return _check(st, where)
    ws = _empty(nbytes(), torch.uint8, X, stream)
    _check(call(ws.data_ptr(), ws.nbytes), where)


class _Device:
    """The tensors' GPU is the current device during a call."""

    __slots__ = ("index", "was")

    def __init__(self, X: torch.Tensor):
        self.index = X.device.index

    def __enter__(self):
        self.was = torch.cuda.current_device()
        torch.cuda.set_device(self.index)

    def __exit__(self, *exc):
        torch.cuda.set_device(self.was)


_SAME_DEVICE = contextlib.nullcontext()


def _device(X: torch.Tensor):
    """X's GPU as the current device (nothing to do where it already is)."""
    return _SAME_DEVICE if X.device.index == torch.cuda.current_device() else _Device(X)


def _int32(**tensors: torch.Tensor) -> None:
    for name, t in tensors.items():
        if t.dtype != torch.int32 or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous int32")


def _quantized(name: str, qweight: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor, m: int, n: int,
               group_size: int) -> None:
    """The quantizer's tensors of an m x n weight (codes of 4-bit fields)."""
    G = gptq_num_groups(n, group_size)
    words = gptq_qweight_words(n, 4)
    _int32(**{f"{name} qweight": qweight, f"{name} zeros": zeros})
    if scales.dtype != torch.float32 or not scales.is_contiguous():
        raise ValueError(f"{name} scales must be contiguous float32")
    if tuple(qweight.shape) != (m, words) or (G >= 0 and not tuple(scales.shape) == tuple(zeros.shape) == (m, G)):
        raise ValueError(f"{name}: qweight must be [{m}, {words}], scales and zeros [{m}, {G}]")


def gptq_w4a16_linear_workspace_bytes(tokens: int, m: int, n: int, group_size: int) -> int:
    return int(lib().gptq_w4a16_linear_workspace_bytes(tokens, m, n, group_size))


def gptq_w4a16_linear(X: torch.Tensor, packed: torch.Tensor, m: int, n: int, group_size: int,
                      bias: Optional[torch.Tensor] = None, activation: str = "none",
                      residual: Optional[torch.Tensor] = None, Y: Optional[torch.Tensor] = None,
                      out_dtype: torch.dtype = torch.bfloat16, workspace: Optional[torch.Tensor] = None,
                      stream=None) -> torch.Tensor:
    """Y [tokens, m] = act(X·Ŵᵀ + bias) + residual for X [tokens, n] bf16 and
    gptq_w4a16_pack's packed weight.  bias [m] and residual [tokens, m] are
    bf16 or fp32; activation is none, relu, silu, gelu or gelu_tanh.  Y (bf16
    or fp32; out_dtype if it is allocated here) may be the residual itself.
    A workspace made for some number of tokens serves every smaller batch;
    without one, or with one that is too small, the call allocates its own."""
    ldx = _bf16_rows(X, n)
    tokens = X.shape[0]
    _on(X, packed=packed, bias=bias, residual=residual, Y=Y, workspace=workspace)
    if Y is None:
        Y = _empty((tokens, m), out_dtype, X, stream)
    e = _lib.GptqEpilogue(activation=_activation_code(activation))
    if bias is not None:
        e.bias, e.bias_dtype = _vector("bias", bias, m), _dtype_code(bias)
    if residual is not None:
        e.ldr = _rows("residual", residual, tokens, m)
        e.residual, e.residual_dtype = residual.data_ptr(), _dtype_code(residual)
    fn = lib().gptq_w4a16_linear
    args = (X.data_ptr(), tokens, ldx, packed.data_ptr(), _uint8("packed", packed), m, n, group_size, ctypes.byref(e),
            Y.data_ptr(), _dtype_code(Y), _rows("Y", Y, tokens, m))
    s = _stream_on(X, stream)
    with _device(X):
        _with_workspace(lambda ws, nbytes: fn(*args, ws, nbytes, s),
                        lambda: gptq_w4a16_linear_workspace_bytes(tokens, m, n, group_size), X, workspace, stream,
                        "gptq_w4a16_linear")
    return Y


def gptq_w4a16_glu_packed_bytes(m: int, n: int, group_size: int) -> int:
    return int(lib().gptq_w4a16_glu_packed_bytes(m, n, group_size))


def gptq_w4a16_glu_pack(gate_qweight: torch.Tensor, gate_scales: torch.Tensor, gate_zeros: torch.Tensor,
                        up_qweight: torch.Tensor, up_scales: torch.Tensor, up_zeros: torch.Tensor,
                        g_idx: torch.Tensor, n: int, bits: int, group_size: int,
                        packed: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The quantizer's output of gate and up (both m x n, one g_idx: they read
    one input) -> the glu's layout (uint8 tensor)."""
    m = gate_qweight.shape[0]
    if bits in (2, 3, 4):
        _quantized("gate", gate_qweight, gate_scales, gate_zeros, m, n, group_size)
        _quantized("up", up_qweight, up_scales, up_zeros, m, n, group_size)
    _int32(g_idx=g_idx)
    if g_idx.numel() != n:
        raise ValueError(f"g_idx must be [{n}]")
    _on(gate_qweight, gate_scales=gate_scales, gate_zeros=gate_zeros, up_qweight=up_qweight, up_scales=up_scales,
        up_zeros=up_zeros, g_idx=g_idx, packed=packed)
    if packed is None:
        packed = _new_packed(gptq_w4a16_glu_packed_bytes(m, n, group_size), gate_qweight, stream)
    with _device(gate_qweight):
        st = lib().gptq_w4a16_glu_pack(_ptr(gate_qweight), _ptr(gate_scales), _ptr(gate_zeros), _ptr(up_qweight),
                                       _ptr(up_scales), _ptr(up_zeros), _ptr(g_idx), m, n, bits, group_size,
                                       _ptr(packed), _uint8("packed", packed), _stream_on(gate_qweight, stream))
    _check(st, "gptq_w4a16_glu_pack")
    return packed


def gptq_w4a16_glu_workspace_bytes(tokens: int, m: int, n: int, group_size: int) -> int:
    return int(lib().gptq_w4a16_glu_workspace_bytes(tokens, m, n, group_size))


def gptq_w4a16_glu(X: torch.Tensor, packed: torch.Tensor, m: int, n: int, group_size: int, activation: str = "silu",
                   gate_bias: Optional[torch.Tensor] = None, up_bias: Optional[torch.Tensor] = None,
                   Y: Optional[torch.Tensor] = None, out_dtype: torch.dtype = torch.bfloat16,
                   workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Y [tokens, m] = act(X·Ŵgᵀ + gate_bias) ⊙ (X·Ŵuᵀ + up_bias) for X
    [tokens, n] bf16 and gptq_w4a16_glu_pack's packed weight."""
    ldx = _bf16_rows(X, n)
    tokens = X.shape[0]
    _on(X, packed=packed, gate_bias=gate_bias, up_bias=up_bias, Y=Y, workspace=workspace)
    if Y is None:
        Y = _empty((tokens, m), out_dtype, X, stream)
    some = gate_bias if gate_bias is not None else up_bias
    if gate_bias is not None and up_bias is not None and gate_bias.dtype != up_bias.dtype:
        raise TypeError("gate_bias and up_bias must have one dtype")
    fn = lib().gptq_w4a16_glu
    args = (X.data_ptr(), tokens, ldx, packed.data_ptr(), _uint8("packed", packed), m, n, group_size,
            _activation_code(activation), _vector("gate_bias", gate_bias, m), _vector("up_bias", up_bias, m),
            0 if some is None else _dtype_code(some), Y.data_ptr(), _dtype_code(Y), _rows("Y", Y, tokens, m))
    s = _stream_on(X, stream)
    with _device(X):
        _with_workspace(lambda ws, nbytes: fn(*args, ws, nbytes, s),
                        lambda: gptq_w4a16_glu_workspace_bytes(tokens, m, n, group_size), X, workspace, stream,
                        "gptq_w4a16_glu")
    return Y


# ---------------------------------------------------------------- mixture of experts
@dataclass
class MoeConfig:
    """Sizes and settings of gptq_w4a16_moe: hidden (the layer's width), inter
    (an expert's), experts, top_k, the experts' bits and group_size, the
    gate's activation, and whether the top_k router weights are divided by
    their sum."""
    hidden: int
    inter: int
    experts: int
    top_k: int
    bits: int = 4
    group_size: int = 64
    activation: str = "silu"
    renormalize: bool = True

    def c(self) -> "_lib.GptqMoeConfig":
        return _lib.GptqMoeConfig(self.hidden, self.inter, self.experts, self.top_k, self.bits, self.group_size,
                                  _activation_code(self.activation), int(bool(self.renormalize)))


def gptq_w4a16_moe_packed_bytes(cfg: MoeConfig) -> int:
    c = cfg.c()
    return int(lib().gptq_w4a16_moe_packed_bytes(ctypes.byref(c)))


def gptq_w4a16_moe_workspace_bytes(cfg: MoeConfig, tokens: int) -> int:
    c = cfg.c()
    return int(lib().gptq_w4a16_moe_workspace_bytes(ctypes.byref(c), tokens))


def gptq_w4a16_moe_pack(cfg: MoeConfig, expert: int, gate_qweight: torch.Tensor, gate_scales: torch.Tensor,
                        gate_zeros: torch.Tensor, up_qweight: torch.Tensor, up_scales: torch.Tensor,
                        up_zeros: torch.Tensor, g_idx: torch.Tensor, down_qweight: torch.Tensor,
                        down_scales: torch.Tensor, down_zeros: torch.Tensor, down_g_idx: torch.Tensor,
                        packed: torch.Tensor, stream=None) -> torch.Tensor:
    """One expert's quantized weights into its place in `packed`
    (gptq_w4a16_moe_packed_bytes(cfg) bytes for all experts): gate and up
    [inter x hidden] share g_idx, down [hidden x inter] has its own."""
    if cfg.bits in (2, 3, 4):
        _quantized("gate", gate_qweight, gate_scales, gate_zeros, cfg.inter, cfg.hidden, cfg.group_size)
        _quantized("up", up_qweight, up_scales, up_zeros, cfg.inter, cfg.hidden, cfg.group_size)
        _quantized("down", down_qweight, down_scales, down_zeros, cfg.hidden, cfg.inter, cfg.group_size)
    _int32(g_idx=g_idx, down_g_idx=down_g_idx)
    if g_idx.numel() != cfg.hidden or down_g_idx.numel() != cfg.inter:
        raise ValueError(f"g_idx must be [{cfg.hidden}] and down_g_idx [{cfg.inter}]")
    _on(gate_qweight, gate_scales=gate_scales, gate_zeros=gate_zeros, up_qweight=up_qweight, up_scales=up_scales,
        up_zeros=up_zeros, g_idx=g_idx, down_qweight=down_qweight, down_scales=down_scales, down_zeros=down_zeros,
        down_g_idx=down_g_idx, packed=packed)
    c = cfg.c()
    with _device(gate_qweight):
        st = lib().gptq_w4a16_moe_pack(ctypes.byref(c), expert, _ptr(gate_qweight), _ptr(gate_scales),
                                       _ptr(gate_zeros), _ptr(up_qweight), _ptr(up_scales), _ptr(up_zeros),
                                       _ptr(g_idx), _ptr(down_qweight), _ptr(down_scales), _ptr(down_zeros),
                                       _ptr(down_g_idx), _ptr(packed), _uint8("packed", packed), _stream_on(gate_qweight, stream))
    _check(st, "gptq_w4a16_moe_pack")
    return packed


def moe_pack_experts(cfg: MoeConfig, experts) -> torch.Tensor:
    """Allocate the packed buffer and pack every expert: `experts` yields
    (gate, up, down) output dicts of quantize_layer, quantize_shared_input
    (gate and up of one expert in one call) or rtn_quantize (which has no
    g_idx: groups of consecutive columns)."""
    packed = None
    count = 0

    def g_idx(o, n):
        if "g_idx" in o:
            return o["g_idx"]
        g = n if cfg.group_size == -1 else cfg.group_size
        return (torch.arange(n, device=o["qweight"].device) // g).to(torch.int32)

    for expert, (gate, up, down) in enumerate(experts):
        gi = g_idx(gate, cfg.hidden)
        if not torch.equal(gi, g_idx(up, cfg.hidden)):
            raise ValueError(f"expert {expert}: gate and up have different g_idx (quantize them on one input)")
        if packed is None:
            packed = torch.empty(max(gptq_w4a16_moe_packed_bytes(cfg), 1), dtype=torch.uint8,
                                 device=gate["qweight"].device)
        gptq_w4a16_moe_pack(cfg, expert, gate["qweight"], gate["scales"], gate["zeros"], up["qweight"], up["scales"],
                            up["zeros"], gi, down["qweight"], down["scales"], down["zeros"],
                            g_idx(down, cfg.inter), packed)
        count += 1
    if count != cfg.experts:
        raise ValueError(f"{count} experts given, the config has {cfg.experts}")
    return packed


def gptq_w4a16_moe(X: torch.Tensor, router: torch.Tensor, packed: torch.Tensor, cfg: MoeConfig,
                   residual: Optional[torch.Tensor] = None, Y: Optional[torch.Tensor] = None,
                   out_dtype: torch.dtype = torch.bfloat16, topk_ids: Optional[torch.Tensor] = None,
                   topk_weights: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                   stream=None) -> tuple:
    """The whole layer for X [tokens, hidden] bf16: softmax router (weights
    [experts, hidden], bf16 or fp32), the top_k experts' gated MLPs, their
    weighted sum plus the residual.  Returns (Y [tokens, hidden], topk_ids
    int32 [tokens, top_k], topk_weights fp32 [tokens, top_k])."""
    ldx = _bf16_rows(X, cfg.hidden)
    tokens = X.shape[0]
    _on(X, router=router, packed=packed, residual=residual, Y=Y, topk_ids=topk_ids, topk_weights=topk_weights,
        workspace=workspace)
    if tuple(router.shape) != (cfg.experts, cfg.hidden) or not router.is_contiguous():
        raise ValueError(f"router must be a contiguous [{cfg.experts}, {cfg.hidden}]")
    if Y is None:
        Y = _empty((tokens, cfg.hidden), out_dtype, X, stream)
    if topk_ids is None:
        topk_ids = _empty((tokens, cfg.top_k), torch.int32, X, stream)
    if topk_weights is None:
        topk_weights = _empty((tokens, cfg.top_k), torch.float32, X, stream)
    _int32(topk_ids=topk_ids)
    if topk_weights.dtype != torch.float32 or not topk_weights.is_contiguous():
        raise ValueError("topk_weights must be contiguous float32")
    if not tuple(topk_ids.shape) == tuple(topk_weights.shape) == (tokens, cfg.top_k):
        raise ValueError(f"topk_ids and topk_weights must be [{tokens}, {cfg.top_k}]")
    ldr = cfg.hidden if residual is None else _rows("residual", residual, tokens, cfg.hidden)
    c = cfg.c()
    fn = lib().gptq_w4a16_moe
    args = (X.data_ptr(), tokens, ldx, router.data_ptr(), _dtype_code(router), ctypes.byref(c), packed.data_ptr(),
            _uint8("packed", packed), _ptr(residual), 0 if residual is None else _dtype_code(residual), ldr,
            Y.data_ptr(), _dtype_code(Y), _rows("Y", Y, tokens, cfg.hidden), topk_ids.data_ptr(),
            topk_weights.data_ptr())
    s = _stream_on(X, stream)
    with _device(X):
        _with_workspace(lambda ws, nbytes: fn(*args, ws, nbytes, s),
                        lambda: int(lib().gptq_w4a16_moe_workspace_bytes(ctypes.byref(c), tokens)), X, workspace, stream,
                        "gptq_w4a16_moe")
    return Y, topk_ids, topk_weights


# ---------------------------------------------------------------- attention and its 4-bit cache
# These calls are made for every layer of every token: a call's checks read each
# attribute once.
@dataclass(frozen=True)
class KvConfig:
    """A key/value cache held in 4 bits: heads and channels of its keys, the
    channels that share a scale (-1: all of a head), positions of a page."""
    kv_heads: int
    head_dim: int = 128
    group_size: int = 128
    page_size: int = 64

    def __post_init__(self):
        c = _lib.GptqKvConfig(self.kv_heads, self.head_dim, self.group_size, self.page_size)
        object.__setattr__(self, "_c", c)
        object.__setattr__(self, "_ref", ctypes.byref(c))
        object.__setattr__(self, "_page_bytes", None)

    def __reduce__(self):   # copies and pickles are made from the fields: the C struct's address is of one process
        return type(self), (self.kv_heads, self.head_dim, self.group_size, self.page_size)

    def c(self) -> "_lib.GptqKvConfig":
        return self._c


def gptq_kv_page_bytes(cfg: KvConfig) -> int:
    if cfg._page_bytes is None:
        object.__setattr__(cfg, "_page_bytes", int(lib().gptq_kv_page_bytes(cfg._ref)))
    return cfg._page_bytes


_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _heads(name: str, t: torch.Tensor, tokens: int, heads: int, dim: int) -> tuple:
    """(token stride, head stride) of a [tokens, heads, dim] tensor."""
    if t.shape != (tokens, heads, dim):
        raise ValueError(f"{name} must be [{tokens}, {heads}, {dim}]")
    ld, hs, one = t.stride()
    if one != 1 and tokens > 0:
        raise ValueError(f"{name} must have unit stride in its last dimension")
    return ld, hs


def _new_heads(tokens: int, heads: int, dim: int, dtype: torch.dtype, X: torch.Tensor, stream) -> torch.Tensor:
    """_empty's [tokens, heads, dim], by the cheapest of torch's ways where the stream is the current one."""
    if stream is None:
        return torch.empty_strided((tokens, heads, dim), (heads * dim, dim, 1), dtype=dtype, device=X.device)
    return _empty((tokens, heads, dim), dtype, X, stream)


def _sequences(cfg: KvConfig, X: torch.Tensor, other: Optional[torch.Tensor], pages: torch.Tensor,
               page_table: torch.Tensor, kv_lens: torch.Tensor, cu_seqlens: Optional[torch.Tensor],
               status: Optional[torch.Tensor]) -> tuple:
    """The sequences of a call as the C entry points take them: cu_seqlens,
    kv_lens, page_table, batch, its width and row stride, pages, their number;
    and status."""
    dev = X.get_device()
    if not (0 <= dev == pages.get_device() == page_table.get_device() == kv_lens.get_device()
            and (cu_seqlens is None or cu_seqlens.get_device() == dev) and (other is None or other.get_device() == dev)
            and (status is None or status.get_device() == dev)):
        _on(X, pages=pages, page_table=page_table, kv_lens=kv_lens, cu_seqlens=cu_seqlens, output=other, status=status)
    page_bytes = cfg._page_bytes or gptq_kv_page_bytes(cfg)
    if page_bytes <= 0:
        raise ValueError("the cache's config is not supported (gptq_kv_page_bytes is 0)")
    shape = page_table.shape
    if page_table.dtype is not torch.int32 or len(shape) != 2:
        raise ValueError("page_table must be int32 [batch, pages of a sequence]")
    batch, width = shape
    if kv_lens.dtype is not torch.int32 or kv_lens.shape != (batch,) or not kv_lens.is_contiguous():
        raise ValueError(f"kv_lens must be a contiguous int32 [{batch}], as page_table has rows")
    ld = width
    if not page_table.is_contiguous():
        ld, one = page_table.stride()
        if batch == 1:
            ld = width
        if width > 1 and one != 1:
            raise ValueError("page_table must have contiguous rows")
    cu = None
    if cu_seqlens is not None:
        if cu_seqlens.dtype is not torch.int32 or cu_seqlens.shape != (batch + 1,) or not cu_seqlens.is_contiguous():
            raise ValueError(f"cu_seqlens must be a contiguous int32 [{batch + 1}]")
        cu = cu_seqlens.data_ptr()
    st = None
    if status is not None:
        if status.dtype is not torch.int32 or status.numel() != 1:
            raise ValueError("status must be one int32")
        st = status.data_ptr()
    if pages.dtype is not torch.uint8 or not pages.is_contiguous():
        raise ValueError("pages must be contiguous uint8")
    return (cu, kv_lens.data_ptr(), page_table.data_ptr(), batch, width, ld, pages.data_ptr(),
            pages.nbytes // page_bytes), st


def _run_on(X: torch.Tensor, stream, fn, *args) -> int:
    """fn(*args, stream) with X's GPU as the current device."""
    dev = X.get_device()
    s = _raw_stream(dev) if stream is None and _raw_stream is not None else _stream_on(X, stream)
    if dev == _current_device():
        return fn(*args, s)
    with _Device(X):
        return fn(*args, s)


def gptq_kv_append(cfg: KvConfig, K: torch.Tensor, V: torch.Tensor, pages: torch.Tensor, page_table: torch.Tensor,
                   kv_lens: torch.Tensor, cu_seqlens: Optional[torch.Tensor] = None,
                   status: Optional[torch.Tensor] = None, stream=None) -> None:
    """Quantize K and V [tokens, kv_heads, head_dim] (bf16 or fp32) into the
    pages (uint8, gptq_kv_page_bytes(cfg) bytes each).  kv_lens [batch]: each
    sequence's positions with these tokens, which are its last.  cu_seqlens
    [batch + 1]: its rows of K and V (None: one each)."""
    tokens = K.shape[0]
    kld, khs = _heads("K", K, tokens, cfg.kv_heads, cfg.head_dim)
    vld, vhs = _heads("V", V, tokens, cfg.kv_heads, cfg.head_dim)
    if K.dtype is not V.dtype:
        raise TypeError("K and V must have one dtype")
    seqs, status = _sequences(cfg, K, V, pages, page_table, kv_lens, cu_seqlens, status)
    st = _run_on(K, stream, lib().gptq_kv_append, cfg._ref, K.data_ptr(), V.data_ptr(), _dtype_code(K), tokens, kld, khs,
                 vld, vhs, *seqs, status)
    if st:
        _check(st, "gptq_kv_append")


def gptq_kv_read(cfg: KvConfig, pages: torch.Tensor, page_table: torch.Tensor, kv_lens: torch.Tensor, tokens: int,
                 cu_seqlens: Optional[torch.Tensor] = None, K: Optional[torch.Tensor] = None,
                 V: Optional[torch.Tensor] = None, out_dtype: torch.dtype = torch.bfloat16,
                 status: Optional[torch.Tensor] = None, stream=None) -> tuple:
    """(K, V) [tokens, kv_heads, head_dim], bf16 or fp32: the last
    cu_seqlens[b + 1] - cu_seqlens[b] positions of each sequence (None: the last
    one), as the cache keeps them."""
    heads, dim = cfg.kv_heads, cfg.head_dim
    kld = vld = heads * dim
    khs = vhs = dim
    own = K is None
    if own:
        K = _new_heads(tokens, heads, dim, out_dtype if V is None else V.dtype, pages, stream)
    else:
        kld, khs = _heads("K", K, tokens, heads, dim)
    if V is None:
        V = torch.empty_like(K) if own and stream is None else _new_heads(tokens, heads, dim, K.dtype, pages, stream)
    else:
        vld, vhs = _heads("V", V, tokens, heads, dim)
        if K.dtype is not V.dtype:
            raise TypeError("K and V must have one dtype")
    seqs, status = _sequences(cfg, K, V, pages, page_table, kv_lens, cu_seqlens, status)
    st = _run_on(K, stream, lib().gptq_kv_read, cfg._ref, K.data_ptr(), V.data_ptr(), _dtype_code(K), tokens, kld, khs,
                 vld, vhs, *seqs, status)
    if st:
        _check(st, "gptq_kv_read")
    return K, V


def gptq_kv_attention_workspace_bytes(cfg: KvConfig, heads: int, batch: int, tokens: int, max_queries: int = 1) -> int:
    return int(lib().gptq_kv_attention_workspace_bytes(cfg._ref, heads, batch, tokens, max_queries))


def gptq_kv_attention(cfg: KvConfig, Q: torch.Tensor, pages: torch.Tensor, page_table: torch.Tensor,
                      kv_lens: torch.Tensor, cu_seqlens: Optional[torch.Tensor] = None,
                      max_queries: Optional[int] = None, scale: Optional[float] = None,
                      Y: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                      status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Y [tokens, heads, head_dim] bf16: attention of each sequence's last
    tokens over its cache (those tokens' keys and values appended before).
    cu_seqlens as in gptq_kv_append; max_queries: the most tokens of a sequence
    in this call as far as it is known (None: a sequence's equal share of them).
    It chooses between kernels, and above 16 weights are rounded to bf16, which
    otherwise have two bf16 parts.  scale: 1/sqrt(head_dim) if None.  Without a
    workspace, or with one that is too small, the call allocates its own."""
    dim = cfg.head_dim
    if Q.dim() != 3:
        raise ValueError(f"Q must be [tokens, heads, {dim}]")
    tokens, heads, _ = Q.shape
    qld, qhs = _heads("Q", Q, tokens, heads, dim)
    if Q.dtype is not torch.bfloat16:
        raise TypeError(f"Q must be bfloat16, not {Q.dtype}")
    seqs, status = _sequences(cfg, Q, Y, pages, page_table, kv_lens, cu_seqlens, status)
    if Y is None:
        Y = _new_heads(tokens, heads, dim, torch.bfloat16, Q, stream)
        yld, yhs = heads * dim, dim
    else:
        yld, yhs = _heads("Y", Y, tokens, heads, dim)
        if Y.dtype is not torch.bfloat16:
            raise TypeError(f"Y must be bfloat16, not {Y.dtype}")
    if max_queries is None:
        max_queries = -(-tokens // max(seqs[3], 1))
    fn = lib().gptq_kv_attention
    args = (cfg._ref, Q.data_ptr(), tokens, heads, qld, qhs, seqs[0], max_queries, *seqs[1:],
            dim ** -0.5 if scale is None else scale, Y.data_ptr(), yld, yhs, status)
    st = _lib.GPTQ_ERR_WORKSPACE
    if workspace is not None:
        if workspace.get_device() != Q.get_device() or not workspace.is_contiguous():
            raise ValueError(f"workspace must be contiguous and on {Q.device}")
        st = _run_on(Q, stream, fn, *args, workspace.data_ptr(), workspace.nbytes)
    if st == _lib.GPTQ_ERR_WORKSPACE:
        nbytes = max(gptq_kv_attention_workspace_bytes(cfg, heads, seqs[3], tokens, max_queries), 1)
        ws = _empty(nbytes, torch.uint8, Q, stream)
        st = _run_on(Q, stream, fn, *args, ws.data_ptr(), nbytes)
    if st:
        _check(st, "gptq_kv_attention")
    return Y


def gptq_prompt_attention(Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, cu_seqlens: torch.Tensor,
                          scale: Optional[float] = None, Y: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Y [tokens, heads, head_dim] bf16: causal attention within each sequence
    (rows cu_seqlens[b] .. cu_seqlens[b + 1]) of Q [tokens, heads, head_dim] and
    K, V [tokens, kv_heads, head_dim], all bf16; heads / kv_heads query heads
    read one key head.  scale: 1/sqrt(head_dim) if None."""
    if Q.dim() != 3 or K.dim() != 3:
        raise ValueError("Q and K must be [tokens, heads, head_dim]")
    tokens, heads, dim = Q.shape
    kv_heads = K.shape[1]
    qld, qhs = _heads("Q", Q, tokens, heads, dim)
    kld, khs = _heads("K", K, tokens, kv_heads, dim)
    vld, vhs = _heads("V", V, tokens, kv_heads, dim)
    dev = Q.get_device()
    if not (0 <= dev == K.get_device() == V.get_device() == cu_seqlens.get_device() and (Y is None or Y.get_device() == dev)):
        _on(Q, K=K, V=V, cu_seqlens=cu_seqlens, Y=Y)
    if Y is None:
        Y = _new_heads(tokens, heads, dim, torch.bfloat16, Q, stream)
        yld, yhs = heads * dim, dim
    else:
        yld, yhs = _heads("Y", Y, tokens, heads, dim)
    if not Q.dtype is K.dtype is V.dtype is Y.dtype is torch.bfloat16:
        raise TypeError("Q, K, V and Y must be bfloat16")
    sequences = cu_seqlens.numel() - 1
    if cu_seqlens.dtype is not torch.int32 or cu_seqlens.dim() != 1 or sequences < 0 or not cu_seqlens.is_contiguous():
        raise ValueError("cu_seqlens must be a contiguous int32 [sequences + 1]")
    st = _run_on(Q, stream, lib().gptq_prompt_attention, Q.data_ptr(), K.data_ptr(), V.data_ptr(), tokens, heads, kv_heads,
                 dim, qld, qhs, kld, khs, vld, vhs, cu_seqlens.data_ptr(), sequences, dim ** -0.5 if scale is None else scale,
                 Y.data_ptr(), yld, yhs)
    if st:
        _check(st, "gptq_prompt_attention")
    return Y


# ---------------------------------------------------------------- whole layer
def alloc_outputs(m: int, n: int, cfg: QuantConfig, device) -> dict:
    words = gptq_qweight_words(n, cfg.bits)
    groups = gptq_num_groups(n, cfg.group_size)
    return dict(
        qweight=torch.empty(m, words, dtype=torch.int32, device=device),
        scales=torch.empty(m, groups, dtype=torch.float32, device=device),
        zeros=torch.empty(m, groups, dtype=torch.int32, device=device),
        g_idx=torch.empty(n, dtype=torch.int32, device=device),
        loss=torch.zeros(2, dtype=torch.float64, device=device),
        perm=torch.empty(n, dtype=torch.int32, device=device),
        status=torch.zeros(1, dtype=torch.int32, device=device),
    )


def quantize_layer(W: torch.Tensor, x_tiles, cfg: QuantConfig, alpha: float = 2.0,
                   keep_hessian: bool = False, check: bool = True) -> dict:
    """The three calls in order on one layer: accumulate every X tile into H,
    prepare U, quantize W.  Returns the outputs (and H/key if keep_hessian).
    check=False leaves the quantizer's status word unread (check_status()
    reads many at once), so the quantization adds no host synchronisation."""
    m, n = W.shape
    dev = W.device
    H = torch.zeros(n, n, dtype=torch.float32, device=dev)
    key = torch.zeros(n, dtype=torch.float64, device=dev)
    for X in x_tiles:
        gptq_hessian_accumulate(H, key, X, alpha)
    out = alloc_outputs(m, n, cfg, dev)
    if keep_hessian:
        out["H"] = H.clone()
        out["key"] = key.clone()
    lam = gptq_prepare_hinv(H, key, cfg.damp_percent, cfg.desc_act, out["perm"])
    out["U"] = H
    out["lam"] = lam
    gptq_quantize_layer(W, H, out["perm"], cfg, out["qweight"], out["scales"], out["zeros"],
                        out["g_idx"], out["loss"], out["status"])
    if check:
        check_status(out)
    return out


def quantize_shared_input(Ws, x_tiles, cfgs, alpha: float = 2.0, check: bool = True) -> list:
    """Linears that read the same input (q/k/v of one attention block, gate/up
    of one MLP) have one Hessian H = 2·XᵀX, and the inverse factor U and the
    column order depend only on H, the damping and act-order: accumulate H and
    prepare U once, then quantize every W under every config (for instance
    two bit widths).  All configs must share damp_percent and desc_act.
    The quantizations issue no host synchronisation; with check=True their
    status words are read once, after the last of them.

    Returns out[i][j] for W i under config j (the alloc_outputs dict), each
    identical to what quantize_layer gives for that W, X and config."""
    cfgs = list(cfgs)
    Ws = list(Ws)
    if not Ws or not cfgs:
        raise ValueError("need at least one weight and one config")
    n = Ws[0].shape[1]
    if any(W.dim() != 2 or W.shape[1] != n for W in Ws):
        raise ValueError("every W must be [m_i, n] with the same n")
    if any(c.damp_percent != cfgs[0].damp_percent or bool(c.desc_act) != bool(cfgs[0].desc_act)
           for c in cfgs):
        raise ValueError("configs sharing one U must agree on damp_percent and desc_act")
    dev = Ws[0].device
    H = torch.zeros(n, n, dtype=torch.float32, device=dev)
    key = torch.zeros(n, dtype=torch.float64, device=dev)
    for X in x_tiles:
        gptq_hessian_accumulate(H, key, X, alpha)
    perm = torch.empty(n, dtype=torch.int32, device=dev)
    lam = gptq_prepare_hinv(H, key, cfgs[0].damp_percent, cfgs[0].desc_act, perm)
    res = []
    for W in Ws:
        row = []
        for cfg in cfgs:
            o = alloc_outputs(W.shape[0], n, cfg, dev)
            o["perm"].copy_(perm)
            gptq_quantize_layer(W, H, perm, cfg, o["qweight"], o["scales"], o["zeros"], o["g_idx"],
                                o["loss"], o["status"])
            o["lam"] = lam
            row.append(o)
        res.append(row)
    if check:
        check_status(res)
    return res
