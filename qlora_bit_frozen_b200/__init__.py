"""QLoRA linear layer on NVIDIA B200: Python binding of libqlora.

Thin marshalling over the C ABI declared in include/qlora.h: each function
here has the name of the C entry point it calls, takes torch tensors, and
passes their device pointers and the current CUDA stream.  Every step of the
computation runs in the library's CUDA kernels; torch only allocates device
memory (outputs and workspaces) and provides the stream.  There is no CPU
fallback: without the built library or a CUDA device the calls raise.
"""
from __future__ import annotations

import contextlib
import ctypes
from dataclasses import dataclass
from typing import List, Optional, Sequence, Tuple

import torch

from . import _ffi
from ._ffi import (COMPUTE_BF16, COMPUTE_FP32, DTYPE_BF16, DTYPE_FP32, FMT_AFFINE, FMT_INT8,
                   FMT_NF4_DQ, FMT_NF4_FP32SCALE, OP_BWD, OP_FWD, STATE_BLOCK, qlora_tensor, qlora_weight)

__all__ = [
    "QLoraError", "QuantizedWeight", "qlora_status_string", "qlora_nf4_codebook",
    "qlora_nf4_payload_bytes", "qlora_quantize_nf4", "qlora_quantize_nf4_noalloc", "qlora_quantize_affine",
    "qlora_nf4_fp32scale_payload_bytes", "qlora_quantize_nf4_fp32scale",
    "qlora_int8_pitch", "qlora_quantize_int8",
    "qlora_dequantize", "qlora_merge", "qlora_adam_step",
    "OptimTensors", "step_control", "qlora_grad_norm_workspace_bytes", "qlora_grad_norm", "qlora_adamw_step",
    "qlora_linear_workspace_bytes", "qlora_linear_fwd", "qlora_linear_bwd",
    "qlora_workspace_status", "qlora_selftest_wait_timeout", "qlora_kernel_launch_count",
    "qlora_kernel_timing_enable", "qlora_kernel_timing_collect",
    "COMPUTE_FP32", "COMPUTE_BF16", "FMT_NF4_DQ", "FMT_NF4_FP32SCALE", "FMT_AFFINE", "FMT_INT8",
    "STATE_BLOCK", "workspace",
]


class QLoraError(RuntimeError):
    def __init__(self, status: int, where: str = ""):
        self.status = int(status)
        msg = _ffi.load().qlora_status_string(self.status).decode()
        super().__init__(f"{where}: {msg} (status {self.status})" if where else msg)


def _check(status: int, where: str):
    if status != _ffi.OK:
        raise QLoraError(status, where)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _stream(stream, dev) -> int:
    """The given stream, or the current one of the call's device."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev.index)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


_HERE = contextlib.nullcontext()


def _on(dev):
    """Makes the tensors' device the current one for a call."""
    return _HERE if dev.index == torch._C._cuda_getDevice() else torch.cuda.device(dev)


def _need(where: str, name: str, t: Optional[torch.Tensor], dev, shape=None, dtype=None):
    """Reject (before any launch) a tensor the kernels would misread: not on
    the weight's CUDA device, not dense, or of the wrong shape or dtype."""
    if t is None or (t.is_cuda and t.device == dev and (dtype is None or t.dtype is dtype)
                     and (shape is None or t.shape == shape) and t.is_contiguous()):
        return
    if not t.is_cuda or t.device != dev:
        raise ValueError(f"{where}: {name} must be a CUDA tensor on {dev}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{where}: {name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{where}: {name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{where}: {name} must be contiguous")


def workspace(nbytes: int, device="cuda") -> torch.Tensor:
    """A 256-byte aligned device workspace of at least nbytes (torch allocates)."""
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def _on_stream(stream, dev, *given):
    """Allocations and copies of a call are made on the stream that it runs on:
    memory of another stream's pool may still be in use there or be handed out
    again there too early, and a copy made there is not ordered before the call.
    (Nothing to do where all buffers are given: the switch takes microseconds.)"""
    if stream is None or (given and all(t is not None for t in given)):
        return _HERE
    if not isinstance(stream, torch.cuda.Stream):
        raw = _stream(stream, dev)
        stream = torch.cuda.ExternalStream(raw, device=dev) if raw else torch.cuda.default_stream(dev)
    return torch.cuda.stream(stream)


@dataclass
class QuantizedWeight:
    """Device buffers of a frozen quantized weight (immutable by convention)."""
    fmt: int
    O: int
    I: int
    block: int
    group: int
    bits: int
    codes: torch.Tensor
    scale_codes: Optional[torch.Tensor] = None
    group_absmax: Optional[torch.Tensor] = None
    mean: Optional[torch.Tensor] = None
    scale: Optional[torch.Tensor] = None
    bias: Optional[torch.Tensor] = None

    def c_struct(self) -> qlora_weight:
        return qlora_weight(self.fmt, self.O, self.I, self.block, self.group, self.bits, _ptr(self.codes),
                            _ptr(self.scale_codes), _ptr(self.group_absmax), _ptr(self.mean),
                            _ptr(self.scale), _ptr(self.bias))

    _BUFFERS = ("codes", "scale_codes", "group_absmax", "mean", "scale", "bias")

    def expected_sizes(self) -> dict:
        """Element count and dtype of every buffer the format defines."""
        N = self.O * self.I
        if self.fmt == FMT_NF4_DQ:
            M = -(-N // self.block)
            S = -(-M // self.group)
            return {"codes": ((N + 1) // 2, torch.uint8), "scale_codes": (M, torch.uint8),
                    "group_absmax": (S, torch.float32), "mean": (1, torch.float32)}
        if self.fmt == FMT_NF4_FP32SCALE:
            return {"codes": ((N + 1) // 2, torch.uint8), "scale": (-(-N // self.block), torch.float32)}
        if self.fmt == FMT_INT8:
            return {"codes": (self.O * qlora_int8_pitch(self.I), torch.int8), "scale": (self.O, torch.float32)}
        ng = -(-N // self.block)
        return {"codes": (N if self.bits == 8 else (N + 1) // 2, torch.uint8),
                "scale": (ng, torch.float32), "bias": (ng, torch.float32)}

    def state_dict(self) -> dict:
        """Host copy of the format fields and the packed buffers, byte for
        byte (the canonical serialization for checkpoints)."""
        d = {"fmt": self.fmt, "O": self.O, "I": self.I, "block": self.block, "group": self.group,
             "bits": self.bits}
        for k in self._BUFFERS:
            t = getattr(self, k)
            if t is not None:
                d[k] = t.detach().cpu().contiguous().numpy().copy()
        return d

    @classmethod
    def from_state_dict(cls, d: dict, device="cuda") -> "QuantizedWeight":
        """Inverse of state_dict(); every buffer is checked against the size
        and dtype its format fields imply before it reaches the device."""
        import numpy as np
        w = cls(int(d["fmt"]), int(d["O"]), int(d["I"]), int(d["block"]), int(d["group"]), int(d["bits"]),
                codes=torch.empty(0, dtype=torch.uint8))
        if w.fmt not in (FMT_NF4_DQ, FMT_NF4_FP32SCALE, FMT_AFFINE, FMT_INT8) or w.O < 0 or w.I < 0 or w.block < 1 \
                or (w.fmt == FMT_NF4_DQ and (w.group < 1 or w.bits != 4)) \
                or (w.fmt == FMT_NF4_FP32SCALE and w.bits != 4) or (w.fmt == FMT_AFFINE and w.bits not in (4, 8)) \
                or (w.fmt == FMT_INT8 and w.bits != 8):
            raise ValueError("inconsistent format fields")
        for k, (n, dt) in w.expected_sizes().items():
            if k not in d or d[k] is None:
                raise ValueError(f"missing buffer {k}")
            a = np.ascontiguousarray(d[k])
            t = torch.from_numpy(a)
            if t.dtype != dt or t.numel() != n:
                raise ValueError(f"buffer {k}: expected {n} x {dt}, got {t.numel()} x {t.dtype}")
            setattr(w, k, t.reshape(-1).to(device))
        return w

    def payload_bytes(self) -> int:
        ts = [self.codes, self.scale_codes, self.group_absmax, self.mean, self.scale, self.bias]
        return sum(t.numel() * t.element_size() for t in ts if t is not None)


def qlora_status_string(status: int) -> str:
    return _ffi.load().qlora_status_string(int(status)).decode()


def qlora_nf4_codebook():
    out = (ctypes.c_float * 16)()
    _check(_ffi.load().qlora_nf4_codebook(out), "qlora_nf4_codebook")
    return [float(v) for v in out]


def qlora_nf4_payload_bytes(N: int, B: int = 64, C: int = 256) -> int:
    return int(_ffi.load().qlora_nf4_payload_bytes(N, B, C))


def qlora_quantize_nf4(W: torch.Tensor, B: int = 64, C: int = 256, stream=None) -> QuantizedWeight:
    """NF4 + double-quantized scales of a CUDA fp32 [O x I] matrix (synchronizes the stream)."""
    lib = _ffi.load()
    if W.dim() != 2 or W.dtype != torch.float32 or not W.is_cuda:
        raise ValueError("W must be a CUDA float32 matrix")
    O, I = W.shape
    N = O * I
    M = -(-N // B)
    S = -(-M // C)
    dev = W.device
    with _on_stream(stream, dev):
        W = W.contiguous()
        codes = torch.empty((N + 1) // 2, dtype=torch.uint8, device=dev)
        q = torch.empty(M, dtype=torch.uint8, device=dev)
        t = torch.empty(S, dtype=torch.float32, device=dev)
        mu = torch.empty(1, dtype=torch.float32, device=dev)
        ws = workspace(lib.qlora_quantize_nf4_workspace_bytes(N, B, C), dev)
    with _on(dev):
        st = lib.qlora_quantize_nf4(_ptr(W), O, I, B, C, _ptr(codes), _ptr(q), _ptr(t), _ptr(mu), _ptr(ws),
                                    ws.numel(), _stream(stream, dev))
    _check(st, "qlora_quantize_nf4")
    return QuantizedWeight(FMT_NF4_DQ, O, I, B, C, 4, codes, q, t, mu)


def qlora_quantize_nf4_noalloc(W: torch.Tensor, B: int = 64, C: int = 256, stream=None) -> QuantizedWeight:
    """As qlora_quantize_nf4, for callers that cannot supply a workspace: the
    library's fixed device scratch is used (see include/qlora.h).  The output
    buffers are still the caller's; calls sharing the scratch must not overlap."""
    lib = _ffi.load()
    if W.dim() != 2 or W.dtype != torch.float32 or not W.is_cuda:
        raise ValueError("W must be a CUDA float32 matrix")
    O, I = W.shape
    N = O * I
    M = -(-N // B)
    S = -(-M // C)
    dev = W.device
    with _on_stream(stream, dev):
        W = W.contiguous()
        codes = torch.empty((N + 1) // 2, dtype=torch.uint8, device=dev)
        q = torch.empty(M, dtype=torch.uint8, device=dev)
        t = torch.empty(S, dtype=torch.float32, device=dev)
        mu = torch.empty(1, dtype=torch.float32, device=dev)
    with _on(dev):
        st = lib.qlora_quantize_nf4_noalloc(_ptr(W), O, I, B, C, _ptr(codes), _ptr(q), _ptr(t), _ptr(mu),
                                            _stream(stream, dev))
    _check(st, "qlora_quantize_nf4_noalloc")
    return QuantizedWeight(FMT_NF4_DQ, O, I, B, C, 4, codes, q, t, mu)


def qlora_nf4_fp32scale_payload_bytes(N: int, B: int = 64) -> int:
    return int(_ffi.load().qlora_nf4_fp32scale_payload_bytes(N, B))


def qlora_quantize_nf4_fp32scale(W: torch.Tensor, B: int = 64, stream=None) -> QuantizedWeight:
    """NF4 codes with the legacy scale storage (one fp32 absmax per block) of
    a CUDA fp32 [O x I] matrix (synchronizes the stream)."""
    lib = _ffi.load()
    if W.dim() != 2 or W.dtype != torch.float32 or not W.is_cuda:
        raise ValueError("W must be a CUDA float32 matrix")
    O, I = W.shape
    N = O * I
    M = -(-N // B)
    dev = W.device
    with _on_stream(stream, dev):
        W = W.contiguous()
        codes = torch.empty((N + 1) // 2, dtype=torch.uint8, device=dev)
        scale = torch.empty(M, dtype=torch.float32, device=dev)
        ws = workspace(lib.qlora_quantize_nf4_fp32scale_workspace_bytes(N, B), dev)
    with _on(dev):
        st = lib.qlora_quantize_nf4_fp32scale(_ptr(W), O, I, B, _ptr(codes), _ptr(scale), _ptr(ws), ws.numel(),
                                              _stream(stream, dev))
    _check(st, "qlora_quantize_nf4_fp32scale")
    return QuantizedWeight(FMT_NF4_FP32SCALE, O, I, B, 0, 4, codes, scale=scale)


def qlora_quantize_affine(W: torch.Tensor, bits: int = 4, G: int = 64, stream=None) -> QuantizedWeight:
    """Affine group-wise 4/8-bit codes with fp32 scale and bias (synchronizes the stream)."""
    lib = _ffi.load()
    if W.dim() != 2 or W.dtype != torch.float32 or not W.is_cuda:
        raise ValueError("W must be a CUDA float32 matrix")
    O, I = W.shape
    N = O * I
    ng = -(-N // G)
    dev = W.device
    with _on_stream(stream, dev):
        W = W.contiguous()
        codes = torch.empty(N if bits == 8 else (N + 1) // 2, dtype=torch.uint8, device=dev)
        scale = torch.empty(ng, dtype=torch.float32, device=dev)
        bias = torch.empty(ng, dtype=torch.float32, device=dev)
        ws = workspace(lib.qlora_quantize_affine_workspace_bytes(N, bits, G), dev)
    with _on(dev):
        st = lib.qlora_quantize_affine(_ptr(W), O, I, bits, G, _ptr(codes), _ptr(scale), _ptr(bias), _ptr(ws),
                                       ws.numel(), _stream(stream, dev))
    _check(st, "qlora_quantize_affine")
    return QuantizedWeight(FMT_AFFINE, O, I, G, 0, bits, codes, scale=scale, bias=bias)


def qlora_int8_pitch(I: int) -> int:
    """Bytes of one row of INT8 codes (I rounded up to a multiple of 16)."""
    return (int(I) + 15) // 16 * 16


def qlora_quantize_int8(W: torch.Tensor, stream=None) -> QuantizedWeight:
    """Symmetric 8-bit codes with one fp32 scale per row (output channel) of a
    CUDA fp32 [O x I] matrix (synchronizes the stream).  The linear layer
    multiplies such a weight in 8-bit integers."""
    lib = _ffi.load()
    if W.dim() != 2 or W.dtype != torch.float32 or not W.is_cuda:
        raise ValueError("W must be a CUDA float32 matrix")
    O, I = W.shape
    dev = W.device
    with _on_stream(stream, dev):
        W = W.contiguous()
        codes = torch.empty((O, qlora_int8_pitch(I)), dtype=torch.int8, device=dev)
        scale = torch.empty(O, dtype=torch.float32, device=dev)
        ws = workspace(lib.qlora_quantize_int8_workspace_bytes(O, I), dev)
    with _on(dev):
        st = lib.qlora_quantize_int8(_ptr(W), O, I, _ptr(codes), _ptr(scale), _ptr(ws), ws.numel(),
                                     _stream(stream, dev))
    _check(st, "qlora_quantize_int8")
    return QuantizedWeight(FMT_INT8, O, I, max(I, 1), 0, 8, codes, scale=scale)


def qlora_dequantize(w: QuantizedWeight, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Diagnostic fp32 reconstruction of the whole weight (never used by fwd/bwd)."""
    lib = _ffi.load()
    if out is None:
        with _on_stream(stream, w.codes.device):
            out = torch.empty((w.O, w.I), dtype=torch.float32, device=w.codes.device)
    _need("qlora_dequantize", "out", out, w.codes.device, (w.O, w.I), torch.float32)
    cw = w.c_struct()
    with _on(w.codes.device):
        st = lib.qlora_dequantize(ctypes.byref(cw), _ptr(out), _stream(stream, w.codes.device))
    _check(st, "qlora_dequantize")
    return out


def qlora_merge(w: QuantizedWeight, A: torch.Tensor, B: torch.Tensor, alpha: float,
                out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Export: W_hat + (alpha/r) B A as an fp32 [O x I] matrix (A [r x I], B [O x r] fp32)."""
    lib = _ffi.load()
    r = A.shape[0]
    if A.dtype != torch.float32 or B.dtype != torch.float32 or tuple(A.shape) != (r, w.I) \
            or tuple(B.shape) != (w.O, r) or not A.is_contiguous() or not B.is_contiguous():
        raise ValueError("A must be contiguous fp32 [r x I] and B contiguous fp32 [O x r]")
    if out is None:
        with _on_stream(stream, w.codes.device):
            out = torch.empty((w.O, w.I), dtype=torch.float32, device=w.codes.device)
    dev = w.codes.device
    _need("qlora_merge", "A", A, dev)
    _need("qlora_merge", "B", B, dev)
    _need("qlora_merge", "out", out, dev, (w.O, w.I), torch.float32)
    cw = w.c_struct()
    with _on(dev):
        st = lib.qlora_merge(ctypes.byref(cw), _ptr(A), _ptr(B), r, float(alpha), _ptr(out), _stream(stream, dev))
    _check(st, "qlora_merge")
    return out


def qlora_adam_step(params: torch.Tensor, grads: torch.Tensor, m: torch.Tensor, v: torch.Tensor, t: int,
                    lr: float, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
                    page_elems: int = 0, stream=None) -> None:
    """One in-place Adam step over flat contiguous fp32 tensors (step count t >= 1)."""
    n = params.numel()
    for x in (params, grads, m, v):
        if x.dtype != torch.float32 or not x.is_contiguous() or x.numel() != n:
            raise ValueError("params, grads, m and v must be contiguous fp32 tensors of one size")
        _need("qlora_adam_step", "params/grads/m/v", x, params.device)
    with _on(params.device):
        st = _ffi.load().qlora_adam_step(_ptr(params), _ptr(grads), _ptr(m), _ptr(v), n, int(t), float(lr),
                                         float(beta1), float(beta2), float(eps), int(page_elems),
                                         _stream(stream, params.device))
    _check(st, "qlora_adam_step")


_DTYPES = {torch.float32: DTYPE_FP32, torch.bfloat16: DTYPE_BF16}


class OptimTensors:
    """The tensors of an optimizer step, checked once: gradients and, for
    qlora_adamw_step, parameters and their AdamW states.  grads and params are
    fp32 or bf16, each pair of one size.  States in 32 bits: m and v are fp32
    of the parameter's size.  States in 8 bits: m is int8 and v uint8 of that
    size, with fp32 scales m_scale and v_scale for each STATE_BLOCK values
    (zeros stand for zero states).  with_states() allocates zero states.

    The tensors are kept and used in place: keep writing gradients into the
    same storage (or build a new object for new tensors).  Their storage is
    held, so that it stays valid where a listed tensor is given another one
    (`p.data = ...`, `module.to(...)`).  For moved parameters and gradients the
    calls then refuse: each looks at one of each, in turn, so that they notice at
    once where all have moved, and where one has after at most as many calls as
    there are tensors.  (States that move are not noticed: the listed storage is
    stepped on.)
    No two parameters or states may overlap, nor a gradient with one of them."""

    def __init__(self, grads: Sequence[torch.Tensor], params: Optional[Sequence[torch.Tensor]] = None,
                 m: Optional[Sequence[torch.Tensor]] = None, v: Optional[Sequence[torch.Tensor]] = None,
                 m_scale: Optional[Sequence[torch.Tensor]] = None,
                 v_scale: Optional[Sequence[torch.Tensor]] = None):
        self.grads = list(grads)
        self.params = None if params is None else list(params)
        self.m, self.v = (None if x is None else list(x) for x in (m, v))
        self.m_scale, self.v_scale = (None if x is None else list(x) for x in (m_scale, v_scale))
        self.device = self.grads[0].device if self.grads else None
        n = len(self.grads)
        for name in ("params", "m", "v", "m_scale", "v_scale"):
            x = getattr(self, name)
            if x is not None and len(x) != n:
                raise ValueError(f"OptimTensors: {name} must list {n} tensors, one for each gradient")
        if self.params is not None and (self.m is None or self.v is None):
            raise ValueError("OptimTensors: params need the states m and v")
        if (self.m_scale is None) != (self.v_scale is None):
            raise ValueError("OptimTensors: 8-bit states need both m_scale and v_scale")
        self.state_bits = 8 if self.m_scale is not None else 32
        self._c = (qlora_tensor * max(n, 1))()
        self._at = []  # of each index, where its gradient and its parameter are
        self._turn = [0, 0]  # of the norm, of the step
        self._held = []
        f = "OptimTensors"
        bits8 = self.state_bits == 8
        states = [(name, x, dt, per) for name, x, dt, per in (
            ("m", self.m, torch.int8 if bits8 else torch.float32, 1),
            ("v", self.v, torch.uint8 if bits8 else torch.float32, 1),
            ("m_scale", self.m_scale, torch.float32, STATE_BLOCK),
            ("v_scale", self.v_scale, torch.float32, STATE_BLOCK)) if x is not None]
        for i, g in enumerate(self.grads):
            if g.dtype not in _DTYPES:
                raise ValueError(f"{f}: grads must be float32 or bfloat16, got {g.dtype}")
            _need(f, f"grads[{i}]", g, self.device)
            c = self._c[i]
            grad, values = g.data_ptr(), g.numel()
            c.grad, c.n, c.grad_type = grad, values, _DTYPES[g.dtype]
            self._held.append(g.untyped_storage())
            if self.params is None:
                self._at.append(((g.data_ptr, grad),))
                continue
            p = self.params[i]
            if p.dtype not in _DTYPES:
                raise ValueError(f"{f}: params must be float32 or bfloat16, got {p.dtype}")
            _need(f, f"params[{i}]", p, self.device, g.shape)
            for name, x, dt, per in states:
                x, size = x[i], -(-values // per)
                _need(f, f"{name}[{i}]", x, self.device, dtype=dt)
                if x.numel() != size:
                    raise ValueError(f"{f}: {name}[{i}] must have {size} values, got {x.numel()}")
                setattr(c, name, x.data_ptr())
                self._held.append(x.untyped_storage())
            param = p.data_ptr()
            c.param, c.param_type = param, _DTYPES[p.dtype]
            self._held.append(p.untyped_storage())
            self._at.append(((g.data_ptr, grad), (p.data_ptr, param)))
        if self.params is not None:
            self._refuse_overlap()
        self._norm_ws = None  # workspace bytes of qlora_grad_norm

    def _in_place(self, where: str, step: bool):
        """One gradient and, for a step, one parameter, in turn, is where it was."""
        i = self._turn[step]
        now = self._at[i]
        for k in range(1 + step):
            data_ptr, was = now[k]
            if data_ptr() != was:
                raise ValueError(f"{where}: {('grads', 'params')[k]}[{i}] has other storage than when it was listed: "
                                 "build a new OptimTensors")
        self._turn[step] = i + 1 if i + 1 < len(self._at) else 0

    def _refuse_overlap(self):
        spans = []
        for name in ("params", "m", "v", "m_scale", "v_scale", "grads"):
            for x in getattr(self, name) or ():
                if x.numel() > 0:
                    spans.append((x.data_ptr(), x.data_ptr() + x.numel() * x.element_size(), name != "grads"))
        spans.sort()
        written = read = 0  # where what came before ends
        for start, end, writes in spans:
            if start < written or (writes and start < read):
                raise ValueError("OptimTensors: parameters or states overlap (a tensor listed twice?)")
            if writes:
                written = max(written, end)
            else:
                read = max(read, end)

    @classmethod
    def with_states(cls, params: Sequence[torch.Tensor], grads: Sequence[torch.Tensor],
                    state_bits: int = 32) -> "OptimTensors":
        """The parameters and gradients with new zero states of 32 or 8 bits."""
        params = list(params)
        if state_bits == 32:
            z = lambda: [torch.zeros(p.shape, dtype=torch.float32, device=p.device) for p in params]  # noqa: E731
            return cls(grads, params, z(), z())
        if state_bits != 8:
            raise ValueError("state_bits must be 8 or 32")
        z = lambda dt: [torch.zeros(p.shape, dtype=dt, device=p.device) for p in params]  # noqa: E731
        s = lambda: [torch.zeros(-(-p.numel() // STATE_BLOCK), dtype=torch.float32, device=p.device)  # noqa: E731
                     for p in params]
        return cls(grads, params, z(torch.int8), z(torch.uint8), s(), s())


def step_control(device="cuda") -> torch.Tensor:
    """A zeroed qlora_step_control: int32[4] holding norm (fp32 bits), scale
    (fp32 bits), skip and step."""
    return torch.zeros(4, dtype=torch.int32, device=device)


def qlora_grad_norm_workspace_bytes(tensors: OptimTensors) -> int:
    if tensors._norm_ws is None:
        tensors._norm_ws = int(_ffi.load().qlora_grad_norm_workspace_bytes(tensors._c, len(tensors.grads)))
    return tensors._norm_ws


def qlora_grad_norm(tensors: OptimTensors, max_norm: float, control: torch.Tensor,
                    ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Global L2 norm of the gradients into control (see step_control), with
    the clip factor, the skip flag and the advanced step count; nothing is
    read back to the host.  max_norm <= 0: no clipping."""
    dev = tensors.device if tensors.device is not None else control.device
    f = "qlora_grad_norm"
    _need(f, "control", control, dev, (4,), torch.int32)
    if tensors._at:
        tensors._in_place(f, step=False)
    with _on(dev):
        if ws is None:
            with _on_stream(stream, dev):
                ws = workspace(qlora_grad_norm_workspace_bytes(tensors), dev)
        _need(f, "ws", ws, dev)
        st = _ffi.load().qlora_grad_norm(tensors._c, len(tensors.grads), float(max_norm), _ptr(control),
                                         _ptr(ws), ws.numel() * ws.element_size(), _stream(stream, dev))
    _check(st, f)
    return control


def qlora_adamw_step(tensors: OptimTensors, t: int = 0, lr: float = 1e-3, beta1: float = 0.9,
                     beta2: float = 0.999, eps: float = 1e-8, weight_decay: float = 0.0,
                     control: Optional[torch.Tensor] = None, stream=None) -> None:
    """One in-place AdamW step over every tensor at once.  The step count, the
    gradient factor and the skip flag come from control where it is given
    (written by qlora_grad_norm), else the step count is t >= 1."""
    f = "qlora_adamw_step"
    if tensors.params is None:
        raise ValueError(f"{f}: the OptimTensors hold gradients only")
    dev = tensors.device
    if dev is None:
        return
    _need(f, "control", control, dev, (4,), torch.int32)
    tensors._in_place(f, step=True)
    with _on(dev):
        st = _ffi.load().qlora_adamw_step(tensors._c, len(tensors.grads), tensors.state_bits, int(t), float(lr),
                                          float(beta1), float(beta2), float(eps), float(weight_decay),
                                          _ptr(control), _stream(stream, dev))
    _check(st, f)


def qlora_linear_workspace_bytes(w: QuantizedWeight, R: int, r: int, op: int, compute: int) -> int:
    cw = w.c_struct()
    return int(_ffi.load().qlora_linear_workspace_bytes(ctypes.byref(cw), R, r, op, compute))


def _compute_of(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return COMPUTE_BF16
    if t.dtype == torch.float32:
        return COMPUTE_FP32
    raise ValueError("activations must be bfloat16 or float32")


def qlora_linear_fwd(w: QuantizedWeight, X: torch.Tensor, A: torch.Tensor, B: torch.Tensor, alpha: float,
                     Y: Optional[torch.Tensor] = None, U_out: Optional[torch.Tensor] = None,
                     ws: Optional[torch.Tensor] = None, stream=None,
                     want_u: bool = True) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Y = X W_hat^T + (alpha/r)(X A^T) B^T; returns (Y, U = X A^T)."""
    lib = _ffi.load()
    R = X.shape[0]
    r = A.shape[0]
    compute = _compute_of(X)
    cw = ctypes.byref(w.c_struct())
    with _on_stream(stream, X.device, Y, U_out if want_u else Y, ws):
        if Y is None:
            Y = X.new_empty((R, w.O))
        if U_out is None and want_u:
            U_out = A.new_empty((R, r))
        if ws is None:
            ws = workspace(lib.qlora_linear_workspace_bytes(cw, R, r, OP_FWD, compute), X.device)
    dev, f = w.codes.device, "qlora_linear_fwd"
    _need(f, "X", X, dev, (R, w.I))
    _need(f, "A", A, dev, (r, w.I), torch.float32)
    _need(f, "B", B, dev, (w.O, r), torch.float32)
    _need(f, "Y", Y, dev, (R, w.O), X.dtype)
    _need(f, "U_out", U_out, dev, (R, r), torch.float32)
    _need(f, "ws", ws, dev)
    with _on(dev):
        st = lib.qlora_linear_fwd(cw, _ptr(X), R, _ptr(A), _ptr(B), r, float(alpha), compute,
                                  _ptr(Y), _ptr(U_out), _ptr(ws), ws.numel(), _stream(stream, dev))
    _check(st, "qlora_linear_fwd")
    return Y, U_out


def qlora_linear_bwd(w: QuantizedWeight, X: Optional[torch.Tensor], dY: torch.Tensor, A: torch.Tensor,
                     B: torch.Tensor, alpha: float, U: Optional[torch.Tensor] = None,
                     want_dx: bool = True, want_da: bool = True, want_db: bool = True,
                     dX: Optional[torch.Tensor] = None, dA: Optional[torch.Tensor] = None,
                     dB: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None, stream=None):
    """(dX, dA, dB) of the QLoRA linear layer (no weight gradient)."""
    lib = _ffi.load()
    R = dY.shape[0]
    r = A.shape[0]
    compute = _compute_of(dY)
    dev = dY.device
    cw = ctypes.byref(w.c_struct())
    with _on_stream(stream, dev, dX if want_dx else dY, dA if want_da else dY, dB if want_db else dY, ws):
        if want_dx and dX is None:
            dX = torch.empty((R, w.I), dtype=dY.dtype, device=dev)
        if want_da and dA is None:
            dA = torch.empty((r, w.I), dtype=torch.float32, device=dev)
        if want_db and dB is None:
            dB = torch.empty((w.O, r), dtype=torch.float32, device=dev)
        if ws is None:
            ws = workspace(lib.qlora_linear_workspace_bytes(cw, R, r, OP_BWD, compute), dev)
    wd, f = w.codes.device, "qlora_linear_bwd"
    _need(f, "dY", dY, wd, (R, w.O))
    _need(f, "X", X, wd, (R, w.I), dY.dtype)
    _need(f, "A", A, wd, (r, w.I), torch.float32)
    _need(f, "B", B, wd, (w.O, r), torch.float32)
    _need(f, "U", U, wd, (R, r), torch.float32)
    _need(f, "dX", dX if want_dx else None, wd, (R, w.I), dY.dtype)
    _need(f, "dA", dA if want_da else None, wd, (r, w.I), torch.float32)
    _need(f, "dB", dB if want_db else None, wd, (w.O, r), torch.float32)
    _need(f, "ws", ws, wd)
    with _on(wd):
        st = lib.qlora_linear_bwd(cw, _ptr(X), _ptr(dY), R, _ptr(A), _ptr(B), r, float(alpha),
                                  _ptr(U), compute, _ptr(dX if want_dx else None), _ptr(dA if want_da else None),
                                  _ptr(dB if want_db else None), _ptr(ws), ws.numel(), _stream(stream, wd))
    _check(st, "qlora_linear_bwd")
    return (dX if want_dx else None), (dA if want_da else None), (dB if want_db else None)


def qlora_workspace_status(ws: torch.Tensor, stream=None) -> int:
    """Device error word of the last call that used ws (synchronizes)."""
    with _on(ws.device):
        return int(_ffi.load().qlora_workspace_status(_ptr(ws), _stream(stream, ws.device)))


def qlora_selftest_wait_timeout(limit_us: int = 1000, stream=None, device="cuda") -> int:
    ws = workspace(256, device)
    with _on(ws.device):
        return int(_ffi.load().qlora_selftest_wait_timeout(_ptr(ws), ws.numel(), int(limit_us),
                                                           _stream(stream, ws.device)))


def qlora_kernel_launch_count() -> int:
    return int(_ffi.load().qlora_kernel_launch_count())


def qlora_kernel_timing_enable(max_records: int) -> None:
    _check(_ffi.load().qlora_kernel_timing_enable(int(max_records)), "qlora_kernel_timing_enable")


def qlora_kernel_timing_collect(max_records: int = 4096):
    """[(kind, ms, flops)] of the tensor-core GEMM launches recorded since enable."""
    ms = (ctypes.c_float * max_records)()
    kind = (ctypes.c_int32 * max_records)()
    fl = (ctypes.c_double * max_records)()
    n = _ffi.load().qlora_kernel_timing_collect(ms, kind, fl, max_records)
    if n < 0:
        raise QLoraError(_ffi.ERR_CUDA, "qlora_kernel_timing_collect")
    return [(int(kind[i]), float(ms[i]), float(fl[i])) for i in range(n)]
