"""Decode-layer operators of libgdn.so: what a quantised Gated DeltaNet layer runs
around the recurrence when it serves.

    hidden -> add_rms_norm_int8 -> int8_matmul (q, k, v, gate, ...)
           -> recurrent_fwd -> gated_rms_norm_int8 -> int8_matmul -> hidden

Argument marshalling only, as in gdn.py.  Every call is asynchronous on the
device's current stream (or ``stream``), takes tensors whose last dimension is
contiguous, and serves inference: an input that requires a gradient is refused
while gradients are recorded, and one that carries a tangent (forward mode).
"""
from __future__ import annotations

import ctypes
import struct
from typing import Optional, Tuple

import torch
from torch.autograd import forward_ad

from .build import binding_for
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
    """``pack(*fields)`` -> the struct's bytes, from fields in order."""
    codes = {_I: "i", _F: "f", _P: "P", _Q: "q", _U: "Q"}
    s = struct.Struct("@" + "".join(codes[t] for _, t in mirror._fields_))
    assert s.size == ctypes.sizeof(mirror), mirror
    return s.pack


_pack_recurrent, _pack_rows, _pack_matmul = (_packer(m) for m in (RecurrentArgs, RowsArgs, Int8MatmulArgs))
_DTYPES = {torch.float32: GDN_F32, torch.bfloat16: GDN_BF16}


class _NoQuick:
    """In place of the quick binding where it was not built for this torch: every call goes the long way."""
    recurrent_fwd = add_rms_norm_int8 = gated_rms_norm_int8 = quantize_int8 = int8_matmul = staticmethod(lambda *a: None)


_quick = None


def _bind_quick():
    """_layer.so (csrc/layer_binding.cpp): the operators' calls on plain tensors at a quarter of the
    host's time.  What it does not take comes back as None and goes the long way below."""
    global _quick
    L = lib()
    try:
        from . import _layer
    except ImportError:
        _layer = None
    if getattr(_layer, "built_for", None) != binding_for():      # torch's C++ tensors change between releases
        _quick = _NoQuick
    else:
        _layer.bind(*(ctypes.cast(f, ctypes.c_void_p).value for f in (
            L.gdn_recurrent_fwd, L.gdn_rows_int8, L.gdn_int8_matmul, L.gdn_int8_matmul_workspace_bytes)), L.gdn_abi_version())
        _quick = _layer
    return _quick


def _failed(status):
    raise GDNError(status, last_error())


_IO = (torch.bfloat16, torch.float32)
_F32, _I32, _I8 = (torch.float32,), (torch.int32,), (torch.int8,)


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
    if forward_ad._current_level >= 0 and forward_ad.unpack_dual(t).tangent is not None:
        raise ValueError(f"{name} carries a tangent: the decode-layer operators have no derivatives")
    if t.dim() and t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")
    if any(n > 2 ** 31 - 1 for n in t.shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}: sizes up to 2^31 - 1 are taken")


def _first(t, name, dims, dtypes):
    """Checks the tensor whose shape and device the others follow."""
    _tensors(**{name: t})
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor (got {t.device})")
    if t.dim() < dims:
        raise ValueError(f"{name} must have {dims} dimensions or more (got {t.dim()})")
    _check(t, name, t.shape, dtypes, t.device)


def _tensors(**named):
    for name in named:
        if not isinstance(named[name], torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")


def _code(dt):
    if dt not in _DTYPES:
        raise TypeError(f"unsupported dtype {dt}; use torch.bfloat16 or torch.float32")
    return _DTYPES[dt]


def _eps(x):
    """x as the struct's 32 bits hold it."""
    return ctypes.c_float(x).value


def _ptr(t):
    return 0 if t is None else t.data_ptr()


def _rows(t, name):
    """(rows, stride) of t seen as rows of its last dimension."""
    if t.dim() != 2:
        try:
            t = t.view(-1, t.shape[-1])
        except RuntimeError:
            raise ValueError(f"{name}: the leading dimensions must be one run of rows with one stride") from None
    if t.shape[0] > 2 ** 31 - 1:
        raise ValueError(f"{name} has {t.shape[0]} rows: up to 2^31 - 1 are taken")
    return t.shape[0], t.stride(0)


def _other_stream(stream, first, tensors, call):
    """``call()`` on ``stream``: what it allocates belongs to that stream, and what it
    reads or writes stays allocated until the stream is past it."""
    _first(first, "the first tensor", 0, (first.dtype,) if isinstance(first, torch.Tensor) else ())
    device = first.device
    if stream.device != device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
    with torch.cuda.stream(stream):
        r = call()
    for t in tensors:
        if t is not None:
            t.record_stream(stream)
    return r


def _launch(name, packed, i):
    """Raw call on device i's current stream; raises GDNError on a non-OK status."""
    with torch.cuda.device(i):
        s = getattr(lib(), name)(packed, torch.cuda.current_stream(i).cuda_stream)
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
    ``qk_norm_eps`` (> 0): q and k are divided by sqrt(sum of squares + qk_norm_eps) first.

    slots and cu_seqlens are read on the device: an entry out of bounds touches nothing
    and is reported by ``device_check``.  A slot may be named once in a call.  A sequence's
    results do not depend on the others of the call, to the last bit.  Prompts of hundreds
    of tokens run quicker through ``chunk_fwd``.
    """
    if stream is not None:
        return _other_stream(stream, q, (q, k, v, alpha, beta, state, slots, cu_seqlens, out), lambda: recurrent_fwd(
            q, k, v, alpha, beta, state, slots, cu_seqlens, qk_norm_eps=qk_norm_eps, o_dtype=o_dtype, out=out))
    r = (_quick or _bind_quick()).recurrent_fwd(q, k, v, alpha, beta, state, slots, cu_seqlens, qk_norm_eps, o_dtype, out)
    if r is not None:
        return r if type(r) is not int else _failed(r)
    _tensors(q=q, k=k, v=v, state=state)
    if q.dim() != 3 or v.dim() != 3 or state.dim() != 4:
        raise ValueError("q must be [N, Hk, dk], v [N, H, dv] and state [P, H, dk, dv]")
    _first(q, "q", 3, _IO)
    dev, io, (N, Hk, dk), (_, H, dv), P, S = q.device, q.dtype, q.shape, v.shape, state.shape[0], q.shape[0]
    _check(k, "k", q.shape, (io,), dev)
    _check(v, "v", (N, H, dv), (io,), dev)
    _check(state, "state", (P, H, dk, dv), _F32, dev)
    if not state.is_contiguous():
        raise ValueError("state must be contiguous")
    for t, name in ((alpha, "alpha"), (beta, "beta")):
        if t is not None:
            _check(t, name, (N, H), _F32, dev)
    if cu_seqlens is not None:
        _tensors(cu_seqlens=cu_seqlens)
        if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1:
            raise ValueError("cu_seqlens must be [S + 1]")
        S = cu_seqlens.shape[0] - 1
        _check(cu_seqlens, "cu_seqlens", (S + 1,), _I32, dev)
    if slots is not None:
        _check(slots, "slots", (S,), _I32, dev)
    if out is not None:
        _tensors(out=out)
        _check(out, "out", (N, H, dv), (o_dtype or out.dtype,), dev)
        if not out.is_contiguous():
            raise ValueError("out must be contiguous")
    od = out.dtype if out is not None else o_dtype or io
    code = _code(od)
    if out is None:
        out = (torch.empty if cu_seqlens is None else torch.zeros)((N, H, dv), device=dev, dtype=od)
    row = lambda t: 0 if t is None else t.stride(0)  # noqa: E731
    _launch("gdn_recurrent_fwd", _pack_recurrent(
        N, S, H, Hk, dk, dv, P, _DTYPES[io], code, 0 if qk_norm_eps is None else 1, 0.0 if qk_norm_eps is None else _eps(qk_norm_eps),
        _ptr(q), _ptr(k), _ptr(v), *q.stride()[:2], *k.stride()[:2], *v.stride()[:2], _ptr(alpha), _ptr(beta), row(alpha), row(beta),
        _ptr(cu_seqlens), _ptr(slots), _ptr(state), _ptr(out)), dev.index)
    return out


def _steps(lead, width, dev):
    """Rows of int8 [*lead, width] that start on 16 bytes, their stride, and their scales [*lead]."""
    pitch = (width + 15) // 16 * 16
    q = torch.empty((*lead, pitch), device=dev, dtype=torch.int8)
    return q if pitch == width else q[..., :width], pitch, torch.empty(lead, device=dev, dtype=torch.float32)


def _weight(weight, shape, dev):
    """(dtype code, address) of a norm's weight."""
    if weight is None:
        return 0, 0
    _check(weight, "weight", shape, _IO, dev)
    return _DTYPES[weight.dtype], weight.data_ptr()


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
    rounding.  Rows of zeros have scale 0, rows with an infinity or a NaN scale NaN and
    steps 0 (h * weight and y past fp32 are infinities)."""
    if stream is not None:
        return _other_stream(stream, x, (x, weight, residual, residual_out), lambda: add_rms_norm_int8(
            x, weight, residual, eps=eps, residual_out=residual_out))
    r = (_quick or _bind_quick()).add_rms_norm_int8(x, weight, residual, eps, residual_out)
    if r is not None:
        return r if type(r) is not int else _failed(r)
    _first(x, "x", 1, _IO)
    shape, dev, D = x.shape, x.device, x.shape[-1]
    rows, xr = _rows(x, "x")
    wdt, wp = _weight(weight, (D,), dev)
    rr = ror = rdt = 0
    if residual is not None:
        _check(residual, "residual", shape, _IO, dev)
        rdt, rr = _DTYPES[residual.dtype], _rows(residual, "residual")[1]
        if residual_out is None:
            residual_out = torch.empty(shape, device=dev, dtype=residual.dtype)
        _check(residual_out, "residual_out", shape, (residual.dtype,), dev)
        ror = _rows(residual_out, "residual_out")[1]
    elif residual_out is not None:
        raise ValueError("residual_out needs a residual")
    q, qr, scale = _steps(shape[:-1], D, dev)
    _launch("gdn_rows_int8", _pack_rows(ROWS_NORM, rows, D, 0, _DTYPES[x.dtype], rdt, wdt, _eps(eps), _ptr(x), _ptr(residual), 0, wp, xr, rr, 0,
                                        ror, qr, _ptr(residual_out), _ptr(q), _ptr(scale)), dev.index)
    return q, scale, residual_out


def _head_rows(t, name):
    """(rows, stride) of t [..., H, d] seen as rows of H * d."""
    if t.dim() == 3:
        rows, H, d = t.shape
        row, head, _ = t.stride()
        if head == d or H == 1:
            return rows, row
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
    stride), d a multiple of 8 up to 256, H * d up to 32768 (H * (d / 8, rounded up to a power of
    two) up to 4096); weight: [d] (bf16 or fp32; None = 1).  q: [..., H * d] int8, its rows on
    16-byte boundaries; scale: [...] fp32, one for all heads of a row."""
    if stream is not None:
        return _other_stream(stream, x, (x, gate, weight), lambda: gated_rms_norm_int8(x, gate, weight, eps=eps))
    r = (_quick or _bind_quick()).gated_rms_norm_int8(x, gate, weight, eps)
    if r is not None:
        return r if type(r) is not int else _failed(r)
    _first(x, "x", 2, _IO)
    dev, (*lead, H, d) = x.device, x.shape
    _check(gate, "gate", x.shape, (x.dtype,), dev)
    wdt, wp = _weight(weight, (d,), dev)
    rows, xr = _head_rows(x, "x")
    gr = _head_rows(gate, "gate")[1]
    q, qr, scale = _steps(lead, H * d, dev)
    _launch("gdn_rows_int8", _pack_rows(ROWS_GATED, rows, H * d, d, _DTYPES[x.dtype], 0, wdt, _eps(eps), _ptr(x), 0, _ptr(gate), wp, xr,
                                        0, gr, 0, qr, 0, _ptr(q), _ptr(scale)), dev.index)
    return q, scale


def quantize_int8(x: torch.Tensor, *, stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """``(q, scale)``: the rows of x [..., D] (bf16 or fp32, D up to 32768) in 8 bits, e.g. a
    weight [N, K] for ``int8_matmul``.  q: [..., D] int8, its rows on 16-byte boundaries
    whatever D is; scale: [...] fp32, the row's largest absolute value / 127."""
    if stream is not None:
        return _other_stream(stream, x, (x,), lambda: quantize_int8(x))
    r = (_quick or _bind_quick()).quantize_int8(x)
    if r is not None:
        return r if type(r) is not int else _failed(r)
    _first(x, "x", 1, _IO)
    D, (rows, xr) = x.shape[-1], _rows(x, "x")
    q, qr, scale = _steps(x.shape[:-1], D, x.device)
    _launch("gdn_rows_int8", _pack_rows(ROWS_PLAIN, rows, D, 0, _DTYPES[x.dtype], 0, 0, 0.0, _ptr(x), 0, 0, 0, xr, 0, 0, 0, qr, 0,
                                        _ptr(q), _ptr(scale)), x.device.index)
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
        return _other_stream(stream, x, (x, x_scale, w, w_scale, bias, out), lambda: int8_matmul(
            x, x_scale, w, w_scale, bias, out_dtype=out_dtype, out=out))
    r = (_quick or _bind_quick()).int8_matmul(x, x_scale, w, w_scale, bias, out_dtype, out)
    if r is not None:
        return r if type(r) is not int else _failed(r)
    _tensors(x=x, x_scale=x_scale, w=w, w_scale=w_scale)
    if w.dim() != 2:
        raise ValueError("w must be [N, K]")
    _first(x, "x", 1, _I8)
    dev, (*lead, K), N = x.device, x.shape, w.shape[0]
    _check(w, "w", (N, K), _I8, dev)
    _check(w_scale, "w_scale", (N,), _F32, dev)
    if not x_scale.is_contiguous():
        raise ValueError("x_scale must be contiguous")
    _check(x_scale, "x_scale", tuple(lead), _F32, dev)
    if bias is not None:
        _check(bias, "bias", (N,), _F32, dev)
    od = _code(out_dtype)
    if out is None:
        out = torch.empty((*lead, N), device=dev, dtype=out_dtype)
    _check(out, "out", (*lead, N), (out_dtype,), dev)
    M, xr = _rows(x, "x")
    outr = _rows(out, "out")[1]
    fields = (M, N, K, od, _ptr(x), _ptr(w), xr, w.stride(0), outr, _ptr(x_scale), _ptr(w_scale), _ptr(bias), _ptr(out))
    need = lib().gdn_int8_matmul_workspace_bytes(_pack_matmul(*fields, 0, 0))
    # from torch's allocator and not kept: a call's copies belong to its stream, or its graph
    workspace = torch.empty(need, device=dev, dtype=torch.uint8) if need else None
    _launch("gdn_int8_matmul", _pack_matmul(*fields, _ptr(workspace), need), dev.index)
    return out
