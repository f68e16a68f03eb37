"""Decode-layer operators of libgdn.so: what a quantised Gated DeltaNet layer runs
around the recurrence when it serves.

    hidden -> add_rms_norm_int8 -> int8_matmul (q, k, v, gate, ...)
           -> recurrent_fwd -> gated_rms_norm_int8 -> int8_matmul -> hidden

Argument marshalling only, as in gdn.py.  Every call is asynchronous on the
device's current stream (or ``stream``), takes tensors whose last dimension is
contiguous, and serves inference: an input that requires a gradient is refused
while gradients are recorded.
"""
from __future__ import annotations

import ctypes
import struct
from typing import Optional, Tuple

import torch

from .gdn import GDN_BF16, GDN_F32, GDN_OK, GDNError, last_error, lib

ROWS_PLAIN, ROWS_NORM, ROWS_GATED = 0, 1, 2

_I, _F, _P, _Q, _U = ctypes.c_int32, ctypes.c_float, ctypes.c_void_p, ctypes.c_int64, ctypes.c_uint64


class RecurrentArgs(ctypes.Structure):
    """Mirror of ``gdn_recurrent_args``."""
    _fields_ = [(n, _I) for n in ("rows", "seqs", "H", "Hk", "dk", "dv", "pool", "io_dtype", "o_dtype", "qk_norm")]
    _fields_ += [("qk_eps", _F), ("q", _P), ("k", _P), ("v", _P)]
    _fields_ += [(n, _Q) for n in ("q_row", "q_head", "k_row", "k_head", "v_row", "v_head")]
    _fields_ += [("alpha", _P), ("beta", _P), ("alpha_row", _Q), ("beta_row", _Q)]
    _fields_ += [(n, _P) for n in ("cu_seqlens", "slots", "state", "o")]


class RowsArgs(ctypes.Structure):
    """Mirror of ``gdn_rows_args``."""
    _fields_ = [(n, _I) for n in ("op", "rows", "width", "head", "x_dtype", "residual_dtype", "weight_dtype")]
    _fields_ += [("eps", _F), ("x", _P), ("residual", _P), ("gate", _P), ("weight", _P)]
    _fields_ += [(n, _Q) for n in ("x_row", "residual_row", "gate_row", "residual_out_row", "q_row")]
    _fields_ += [("residual_out", _P), ("q", _P), ("scale", _P)]


class Int8MatmulArgs(ctypes.Structure):
    """Mirror of ``gdn_int8_matmul_args``."""
    _fields_ = [("M", _I), ("N", _I), ("K", _I), ("out_dtype", _I), ("x", _P), ("w", _P), ("x_row", _Q),
                ("w_row", _Q), ("out_row", _Q), ("x_scale", _P), ("w_scale", _P), ("bias", _P), ("out", _P),
                ("workspace", _P), ("workspace_bytes", _U)]


def _packer(mirror):
    """``pack(*fields)`` -> the struct's bytes: several times quicker than filling a ctypes
    struct field by field, which is most of a small call's time."""
    codes = {_I: "i", _F: "f", _P: "P", _Q: "q", _U: "Q"}
    s = struct.Struct("@" + "".join(codes[t] for _, t in mirror._fields_))
    assert s.size == ctypes.sizeof(mirror), mirror
    return s.pack


_pack_recurrent, _pack_rows, _pack_matmul = (_packer(m) for m in (RecurrentArgs, RowsArgs, Int8MatmulArgs))
_DTYPES = {torch.float32: GDN_F32, torch.bfloat16: GDN_BF16}
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _check(t, name, shape, dtypes, device):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device:
        raise ValueError(f"{name} must be a CUDA tensor on {device} (got {t.device})")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected " + " or ".join(map(str, dtypes)))
    if t.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{name} requires a gradient: the decode-layer operators have none")
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")


def _first(t, name, dims, dtypes):
    """Checks the tensor whose shape and device the others follow."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor (got {t.device})")
    if t.dim() < dims:
        raise ValueError(f"{name} must have {dims} dimensions or more (got {t.dim()})")
    _check(t, name, t.shape, dtypes, t.device)


_IO = (torch.bfloat16, torch.float32)
_F32, _I32, _I8 = (torch.float32,), (torch.int32,), (torch.int8,)


def _rows(t, name):
    """(rows, stride) of t seen as rows of its last dimension."""
    if t.dim() == 2:
        return t.shape[0], t.stride(0)
    try:
        t = t.view(-1, t.shape[-1])
    except RuntimeError:
        raise ValueError(f"{name}: the leading dimensions must be one run of rows with one stride") from None
    return t.shape[0], t.stride(0)


def _other_stream(stream, device, tensors, call):
    """``call()`` on ``stream``: what it allocates belongs to that stream, and what it
    reads or writes stays allocated until the stream is past it."""
    if stream.device != device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
    with torch.cuda.stream(stream):
        r = call()
    for t in tensors:
        if t is not None:
            t.record_stream(stream)
    return r


def _launch(fn, packed, device):
    """Raw call on the device's current stream; raises GDNError on a non-OK status."""
    i = device.index
    if torch.cuda.current_device() == i:
        s = fn(packed, _raw_stream(i))
    else:
        with torch.cuda.device(i):
            s = fn(packed, _raw_stream(i))
    if s != GDN_OK:
        raise GDNError(s, last_error())


def call_recurrent(args: RecurrentArgs, stream: Optional[int] = None) -> None:
    """Raw gdn_recurrent_fwd call; raises GDNError on a non-OK status."""
    s = lib().gdn_recurrent_fwd(ctypes.string_at(ctypes.byref(args), ctypes.sizeof(args)), stream or 0)
    if s != GDN_OK:
        raise GDNError(s, last_error())


def call_rows(args: RowsArgs, stream: Optional[int] = None) -> None:
    """Raw gdn_rows_int8 call; raises GDNError on a non-OK status."""
    s = lib().gdn_rows_int8(ctypes.string_at(ctypes.byref(args), ctypes.sizeof(args)), stream or 0)
    if s != GDN_OK:
        raise GDNError(s, last_error())


def call_int8_matmul(args: Int8MatmulArgs, stream: Optional[int] = None) -> None:
    """Raw gdn_int8_matmul call; raises GDNError on a non-OK status."""
    s = lib().gdn_int8_matmul(ctypes.string_at(ctypes.byref(args), ctypes.sizeof(args)), stream or 0)
    if s != GDN_OK:
        raise GDNError(s, last_error())


def int8_matmul_workspace_bytes(args: Int8MatmulArgs) -> int:
    """Device workspace gdn_int8_matmul needs for ``args`` (0 if invalid; host only)."""
    return int(lib().gdn_int8_matmul_workspace_bytes(ctypes.string_at(ctypes.byref(args), ctypes.sizeof(args))))


def recurrent_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, alpha: Optional[torch.Tensor],
                  beta: Optional[torch.Tensor], state: torch.Tensor, slots: Optional[torch.Tensor] = None,
                  cu_seqlens: Optional[torch.Tensor] = None, *, qk_norm_eps: Optional[float] = None,
                  o_dtype: Optional[torch.dtype] = None, out: Optional[torch.Tensor] = None,
                  stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Gated delta rule, token by token, on a pool of states that it updates in place.

    q, k: [N, Hk, dk], v: [N, H, dv] (bf16 or fp32, same dtype; any row and head
    strides, e.g. parts of one projection's rows): the sequences' tokens one after
    another.  Value head h reads key head h // (H // Hk).  alpha, beta: [N, H] fp32
    (None = 1).  state: [P, H, dk, dv] fp32, contiguous, the layout of ``chunk_fwd``'s
    ``S_T`` (which may be written into a pool's row).  slots: [S] int32, the state of
    each sequence, -1 for an entry that holds none (None: sequence s owns state s).
    cu_seqlens: [S + 1] int32, sequence s owns rows cu_seqlens[s] up to cu_seqlens[s + 1]
    (None: one token a sequence, S = N).  dk 16, 32, 64 or 128; dv 32, 64, 96 or 128.

    Returns o [N, H, dv] in ``o_dtype`` (default: q's): 0 for entries of slot -1; rows of
    no sequence are left as they were in ``out``, and are 0 where ``out`` is made here.
    ``qk_norm_eps``: q and k are divided by sqrt(sum of squares + qk_norm_eps) first.

    slots and cu_seqlens are read on the device: an entry out of bounds touches nothing
    and is reported by ``device_check``.  A slot may be named once in a call.  Prompts
    of hundreds of tokens run quicker through ``chunk_fwd``.
    """
    if stream is not None:
        return _other_stream(stream, q.device, (q, k, v, alpha, beta, state, slots, cu_seqlens, out), lambda: recurrent_fwd(
            q, k, v, alpha, beta, state, slots, cu_seqlens, qk_norm_eps=qk_norm_eps, o_dtype=o_dtype, out=out))
    _first(q, "q", 3, _IO)
    dev, io = q.device, (q.dtype,)
    if q.dim() != 3 or not isinstance(v, torch.Tensor) or v.dim() != 3:
        raise ValueError("q must be [N, Hk, dk] and v [N, H, dv]")
    N, Hk, dk = q.shape
    H, dv = v.shape[1:]
    _check(k, "k", q.shape, io, dev)
    _check(v, "v", (N, H, dv), io, dev)
    if alpha is not None:
        _check(alpha, "alpha", (N, H), _F32, dev)
    if beta is not None:
        _check(beta, "beta", (N, H), _F32, dev)
    if not isinstance(state, torch.Tensor) or state.dim() != 4:
        raise ValueError("state must be [P, H, dk, dv]")
    _check(state, "state", (state.shape[0], H, dk, dv), _F32, dev)
    if not state.is_contiguous():
        raise ValueError("state must be contiguous")
    S = N
    if cu_seqlens is not None:
        if not isinstance(cu_seqlens, torch.Tensor) or cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1:
            raise ValueError("cu_seqlens must be [S + 1]")
        S = cu_seqlens.shape[0] - 1
        _check(cu_seqlens, "cu_seqlens", (S + 1,), _I32, dev)
    if slots is not None:
        _check(slots, "slots", (S,), _I32, dev)
    if out is None:
        make = torch.empty if cu_seqlens is None else torch.zeros
        out = make((N, H, dv), device=dev, dtype=o_dtype or q.dtype)
    _check(out, "out", (N, H, dv), _IO if o_dtype is None else (o_dtype,), dev)
    if not out.is_contiguous():
        raise ValueError("out must be contiguous")
    opt = lambda t: 0 if t is None else t.data_ptr()  # noqa: E731
    (qr, qh, _), (kr, kh, _), (vr, vh, _) = q.stride(), k.stride(), v.stride()
    _launch(lib().gdn_recurrent_fwd, _pack_recurrent(
        N, S, H, Hk, dk, dv, state.shape[0], _DTYPES[q.dtype], _code(out.dtype), int(qk_norm_eps is not None),
        qk_norm_eps or 0.0, q.data_ptr(), k.data_ptr(), v.data_ptr(), qr, qh, kr, kh, vr, vh, opt(alpha), opt(beta),
        0 if alpha is None else alpha.stride(0), 0 if beta is None else beta.stride(0), opt(cu_seqlens), opt(slots),
        state.data_ptr(), out.data_ptr()), dev)
    return out


def _code(dt):
    if dt not in _DTYPES:
        raise TypeError(f"unsupported dtype {dt}; use torch.bfloat16 or torch.float32")
    return _DTYPES[dt]


def _steps(lead, rows, width, dev):
    """A tensor [*lead, width] of int8 whose rows start on 16 bytes, and its row stride."""
    pitch = (width + 15) // 16 * 16
    if pitch == width:
        return torch.empty((*lead, width), device=dev, dtype=torch.int8), pitch
    return torch.empty((*lead, pitch), device=dev, dtype=torch.int8)[..., :width], pitch


def add_rms_norm_int8(x: torch.Tensor, weight: Optional[torch.Tensor] = None, residual: Optional[torch.Tensor] = None, *,
                      eps: float = 1e-6, residual_out: Optional[torch.Tensor] = None,
                      stream: Optional[torch.cuda.Stream] = None
                      ) -> Tuple[torch.Tensor, torch.Tensor, Optional[torch.Tensor]]:
    """``(q, scale, h)`` of h = x + residual and the rows y = h / sqrt(mean(h^2) + eps) * weight
    in 8 bits: y is about q * scale[..., None].

    x, residual: [..., D] (bf16 or fp32 each; residual None = 0), D up to 32768; weight: [D]
    (bf16 or fp32; None = 1).  q: [..., D] int8, its rows on 16-byte boundaries; scale: [...]
    fp32, max|y| / 127; h: rounded to the residual's dtype, into ``residual_out`` if given
    (which may be ``residual``), None without a residual.  The norm takes h before that
    rounding.  Rows of zeros have scale 0, rows with an infinity or a NaN scale NaN."""
    if stream is not None:
        return _other_stream(stream, x.device, (x, weight, residual, residual_out), lambda: add_rms_norm_int8(
            x, weight, residual, eps=eps, residual_out=residual_out))
    _first(x, "x", 1, _IO)
    dev, D = x.device, x.shape[-1]
    rows, xr = _rows(x, "x")
    rr = ror = rdt = wdt = rp = wp = rop = 0
    if weight is not None:
        _check(weight, "weight", (D,), _IO, dev)
        wdt, wp = _DTYPES[weight.dtype], weight.data_ptr()
    if residual is not None:
        _check(residual, "residual", x.shape, _IO, dev)
        rdt, rp = _DTYPES[residual.dtype], residual.data_ptr()
        rr = _rows(residual, "residual")[1]
        if residual_out is None:
            residual_out = torch.empty(x.shape, device=dev, dtype=residual.dtype)
        _check(residual_out, "residual_out", x.shape, (residual.dtype,), dev)
        rop, ror = residual_out.data_ptr(), _rows(residual_out, "residual_out")[1]
    elif residual_out is not None:
        raise ValueError("residual_out needs a residual")
    lead = x.shape[:-1]
    q, qr = _steps(lead, rows, D, dev)
    scale = torch.empty(lead, device=dev, dtype=torch.float32)
    _launch(lib().gdn_rows_int8, _pack_rows(ROWS_NORM, rows, D, 0, _DTYPES[x.dtype], rdt, wdt, eps, x.data_ptr(), rp, 0, wp,
                                            xr, rr, 0, ror, qr, rop, q.data_ptr(), scale.data_ptr()), dev)
    return q, scale, residual_out


def _head_rows(t, name):
    """(rows, stride) of t [..., H, d] seen as rows of H * d."""
    if t.dim() == 3 and (t.stride(1) == t.shape[2] or t.shape[1] == 1):
        return t.shape[0], t.stride(0)
    try:
        t = t.view(-1, t.shape[-2] * t.shape[-1])
    except RuntimeError:
        raise ValueError(f"{name}: a row's heads must be adjacent, and the rows one run with one stride") from None
    return t.shape[0], t.stride(0)


def gated_rms_norm_int8(x: torch.Tensor, gate: torch.Tensor, weight: Optional[torch.Tensor] = None, *, eps: float = 1e-6,
                        stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """``(q, scale)``: for each head y = x / sqrt(mean(x^2) + eps) * weight * gate * sigmoid(gate),
    and the rows of all heads in 8 bits.

    x, gate: [..., H, d] (bf16 or fp32, same dtype; the heads of a row adjacent, any row
    stride), d a multiple of 8 up to 256; weight: [d] (bf16 or fp32; None = 1).  q: [..., H * d]
    int8, its rows on 16-byte boundaries; scale: [...] fp32, one for all heads of a row."""
    if stream is not None:
        return _other_stream(stream, x.device, (x, gate, weight), lambda: gated_rms_norm_int8(x, gate, weight, eps=eps))
    _first(x, "x", 2, _IO)
    dev = x.device
    *lead, H, d = x.shape
    _check(gate, "gate", x.shape, (x.dtype,), dev)
    wdt = wp = 0
    if weight is not None:
        _check(weight, "weight", (d,), _IO, dev)
        wdt, wp = _DTYPES[weight.dtype], weight.data_ptr()
    rows, xr = _head_rows(x, "x")
    gr = _head_rows(gate, "gate")[1]
    q, qr = _steps(lead, rows, H * d, dev)
    scale = torch.empty(lead, device=dev, dtype=torch.float32)
    _launch(lib().gdn_rows_int8, _pack_rows(ROWS_GATED, rows, H * d, d, _DTYPES[x.dtype], 0, wdt, eps, x.data_ptr(), 0,
                                            gate.data_ptr(), wp, xr, 0, gr, 0, qr, 0, q.data_ptr(), scale.data_ptr()), dev)
    return q, scale


def quantize_int8(x: torch.Tensor, *, stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """``(q, scale)``: the rows of x [..., D] (bf16 or fp32, D up to 32768) in 8 bits, e.g. a
    weight [N, K] for ``int8_matmul``.  q: [..., D] int8, its rows on 16-byte boundaries
    whatever D is; scale: [...] fp32, the row's largest absolute value / 127."""
    if stream is not None:
        return _other_stream(stream, x.device, (x,), lambda: quantize_int8(x))
    _first(x, "x", 1, _IO)
    dev, D = x.device, x.shape[-1]
    rows, xr = _rows(x, "x")
    lead = x.shape[:-1]
    q, qr = _steps(lead, rows, D, dev)
    scale = torch.empty(lead, device=dev, dtype=torch.float32)
    _launch(lib().gdn_rows_int8, _pack_rows(ROWS_PLAIN, rows, D, 0, _DTYPES[x.dtype], 0, 0, 0.0, x.data_ptr(), 0, 0, 0,
                                            xr, 0, 0, 0, qr, 0, q.data_ptr(), scale.data_ptr()), dev)
    return q, scale


def int8_matmul(x: torch.Tensor, x_scale: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor,
                bias: Optional[torch.Tensor] = None, *, out_dtype: torch.dtype = torch.bfloat16,
                out: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """out[..., n] = x_scale * w_scale[n] * (x . w[n]) + bias[n], with the sum over K exact.

    x: [..., K] int8, x_scale: [...] fp32; w: [N, K] int8, w_scale: [N] fp32; bias: [N] fp32
    or None; K up to 131071.  Rows that start on 16 bytes (as ``quantize_int8`` and the norms
    lay them out) are read where they are; others are copied to such rows first, in every
    call.  ``out``: [..., N] in ``out_dtype`` (bf16 or fp32), or None to allocate it."""
    if stream is not None:
        return _other_stream(stream, x.device, (x, x_scale, w, w_scale, bias, out), lambda: int8_matmul(
            x, x_scale, w, w_scale, bias, out_dtype=out_dtype, out=out))
    _first(x, "x", 1, _I8)
    dev, K = x.device, x.shape[-1]
    if not isinstance(w, torch.Tensor) or w.dim() != 2:
        raise ValueError("w must be [N, K]")
    N, lead = w.shape[0], x.shape[:-1]
    _check(w, "w", (N, K), _I8, dev)
    _check(w_scale, "w_scale", (N,), _F32, dev)
    _check_scale(x_scale, lead, dev)
    if bias is not None:
        _check(bias, "bias", (N,), _F32, dev)
    M, xr = _rows(x, "x")
    if out is None:
        out = torch.empty((*lead, N), device=dev, dtype=out_dtype)
    _check(out, "out", (*lead, N), (out_dtype,), dev)
    wr, xp, wp = w.stride(0), x.data_ptr(), w.data_ptr()
    fields = (M, N, K, _code(out_dtype), xp, wp, xr, wr, _rows(out, "out")[1], x_scale.data_ptr(), w_scale.data_ptr(),
              0 if bias is None else bias.data_ptr(), out.data_ptr())
    ws, need = None, 0
    if (xp | wp | xr | wr) & 15 or not xr or not wr:
        # from torch's allocator and not kept: a call's copies belong to its stream, or its graph
        need = int8_matmul_workspace_bytes(Int8MatmulArgs(*fields))
        ws = torch.empty(need, device=dev, dtype=torch.uint8) if need else None
    _launch(lib().gdn_int8_matmul, _pack_matmul(*fields, 0 if ws is None else ws.data_ptr(), need), dev)
    return out


def _check_scale(t, lead, dev):
    if not isinstance(t, torch.Tensor):
        raise TypeError("x_scale must be a torch.Tensor")
    if not t.is_contiguous():
        raise ValueError("x_scale must be contiguous")
    if t.dim() == 0:
        if len(lead):
            raise ValueError(f"x_scale has shape (), expected {tuple(lead)}")
        t = t.view(1)
        lead = (1,)
    _check(t, "x_scale", lead, _F32, dev)
