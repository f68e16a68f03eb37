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
    """``pack(*fields)`` -> the struct's bytes: several times quicker than filling a ctypes
    struct field by field."""
    codes = {_I: "i", _F: "f", _P: "P", _Q: "q", _U: "Q"}
    s = struct.Struct("@" + "".join(codes[t] for _, t in mirror._fields_))
    assert s.size == ctypes.sizeof(mirror), mirror
    return s.pack


_pack_recurrent, _pack_rows, _pack_matmul = (_packer(m) for m in (RecurrentArgs, RowsArgs, Int8MatmulArgs))
_DTYPES = {torch.float32: GDN_F32, torch.bfloat16: GDN_BF16}
_functions = {}
# torch.cuda.current_stream(i).cuda_stream and current_device(), without their objects (2 us a call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda i: torch.cuda.current_stream(i).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_empty = torch.empty_strided          # a third quicker than torch.empty


class _NoQuick:
    """In place of the quick binding where it was not built for this torch: every call goes the long way."""
    recurrent_fwd = add_rms_norm_int8 = gated_rms_norm_int8 = quantize_int8 = int8_matmul = staticmethod(lambda *a: None)


_quick = None


def _bind_quick():
    """_layer.so (csrc/layer_binding.cpp): the operators' calls of the usual form at a third of
    the host's time.  What it does not take comes back as None and goes the long way below."""
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
    if t.dim() and t.stride(-1) != 1 and t.shape[-1] > 1:
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
        return t.shape[0], t.stride()[0]
    try:
        t = t.view(-1, t.shape[-1])
    except RuntimeError:
        raise ValueError(f"{name}: the leading dimensions must be one run of rows with one stride") from None
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
    fn = _functions.get(name) or _functions.setdefault(name, getattr(lib(), name))
    if _current_device() == i:
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
    # What a correct call looks like, tested in place; _recurrent_refuse says what is wrong with another.
    try:
        N, Hk, dk = shape = q.shape
        _, H, dv = v.shape
        io, i, S = q.dtype, q.get_device(), N
        P, gates = state.shape[0], (N, H)
        qr, qh, q1 = q.stride()
        kr, kh, k1 = k.stride()
        vr, vh, v1 = v.stride()
        ap = bp = ar = br = cp = sp = 0
        fits = (i >= 0 and k.shape == shape and v.shape == (N, H, dv) and k.dtype is io and v.dtype is io and q1 == k1 == v1 == 1
                and k.get_device() == i and v.get_device() == i and state.dtype is torch.float32 and state.get_device() == i
                and state.shape == (P, H, dk, dv) and state.is_contiguous())
        if alpha is not None:
            ar, a1 = alpha.stride()
            ap = alpha.data_ptr()
            fits = fits and a1 == 1 and alpha.shape == gates and alpha.dtype is torch.float32 and alpha.get_device() == i
        if beta is not None:
            br, b1 = beta.stride()
            bp = beta.data_ptr()
            fits = fits and b1 == 1 and beta.shape == gates and beta.dtype is torch.float32 and beta.get_device() == i
        if cu_seqlens is not None:
            S = cu_seqlens.shape[0] - 1
            cp = cu_seqlens.data_ptr()
            fits = fits and S >= 0 and cu_seqlens.dtype is torch.int32 and cu_seqlens.stride() == (1,) and cu_seqlens.get_device() == i
        if slots is not None:
            sp = slots.data_ptr()
            fits = fits and slots.shape == (S,) and slots.dtype is torch.int32 and slots.stride() == (1,) and slots.get_device() == i
        if out is not None:
            od = out.dtype
            fits = fits and out.shape == (N, H, dv) and (o_dtype is None or od is o_dtype) and out.get_device() == i and out.is_contiguous()
        else:
            od = o_dtype or io
        if torch.is_grad_enabled():
            fits = fits and not any(t is not None and t.requires_grad for t in (q, k, v, alpha, beta, state, out))
        fits = fits and io in _DTYPES and od in _DTYPES
    except (AttributeError, TypeError, ValueError, IndexError):
        fits = False
    if not fits:
        _recurrent_refuse(q, k, v, alpha, beta, state, slots, cu_seqlens, o_dtype, out)
    if out is None:
        dev = q.device
        out = _empty((N, H, dv), (H * dv, dv, 1), device=dev, dtype=od) if cu_seqlens is None else torch.zeros((N, H, dv), device=dev, dtype=od)
    _launch("gdn_recurrent_fwd", _pack_recurrent(
        N, S, H, Hk, dk, dv, P, _DTYPES[io], _DTYPES[od], 0 if qk_norm_eps is None else 1, qk_norm_eps or 0.0,
        q.data_ptr(), k.data_ptr(), v.data_ptr(), qr, qh, kr, kh, vr, vh, ap, bp, ar, br, cp, sp, state.data_ptr(),
        out.data_ptr()), i)
    return out


def _recurrent_refuse(q, k, v, alpha, beta, state, slots, cu_seqlens, o_dtype, out):
    """Raises for what recurrent_fwd does not take; returns where only its quick test was too
    strict (a dimension of one element with some other stride)."""
    _tensors(q=q, k=k, v=v, state=state)
    if q.dim() != 3 or v.dim() != 3 or state.dim() != 4:
        raise ValueError("q must be [N, Hk, dk], v [N, H, dv] and state [P, H, dk, dv]")
    _first(q, "q", 3, _IO)
    dev, (N, _, dk), (_, H, dv), S = q.device, q.shape, v.shape, q.shape[0]
    _check(k, "k", q.shape, (q.dtype,), dev)
    _check(v, "v", (N, H, dv), (q.dtype,), dev)
    _check(state, "state", (state.shape[0], H, dk, dv), _F32, dev)
    if alpha is not None:
        _check(alpha, "alpha", (N, H), _F32, dev)
    if beta is not None:
        _check(beta, "beta", (N, H), _F32, dev)
    if cu_seqlens is not None:
        _tensors(cu_seqlens=cu_seqlens)
        if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1:
            raise ValueError("cu_seqlens must be [S + 1]")
        S = cu_seqlens.shape[0] - 1
        _check(cu_seqlens, "cu_seqlens", (S + 1,), _I32, dev)
    if slots is not None:
        _check(slots, "slots", (S,), _I32, dev)
    if not state.is_contiguous():
        raise ValueError("state must be contiguous")
    _code(q.dtype), _code(o_dtype or q.dtype)
    if out is not None:
        _tensors(out=out)
        _check(out, "out", (N, H, dv), (o_dtype or out.dtype,), dev)
        _code(out.dtype)
        if not out.is_contiguous():
            raise ValueError("out must be contiguous")


def _tensors(**named):
    for name in named:
        if not isinstance(named[name], torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")


def _code(dt):
    if dt not in _DTYPES:
        raise TypeError(f"unsupported dtype {dt}; use torch.bfloat16 or torch.float32")
    return _DTYPES[dt]


def _steps(lead, rows, width, dev):
    """Rows of int8 [*lead, width] that start on 16 bytes, their stride, and their scales [*lead]."""
    pitch = (width + 15) // 16 * 16
    if len(lead) == 1:
        return (_empty((rows, width), (pitch, 1), device=dev, dtype=torch.int8), pitch,
                _empty((rows,), (1,), device=dev, dtype=torch.float32))
    q = torch.empty((*lead, pitch), device=dev, dtype=torch.int8)
    return q if pitch == width else q[..., :width], pitch, torch.empty(lead, device=dev, dtype=torch.float32)


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
        return _other_stream(stream, x, (x, weight, residual, residual_out), lambda: add_rms_norm_int8(
            x, weight, residual, eps=eps, residual_out=residual_out))
    r = (_quick or _bind_quick()).add_rms_norm_int8(x, weight, residual, eps, residual_out)
    if r is not None:
        return r if type(r) is not int else _failed(r)
    i, grad, xd = _row_input(x, 1)
    shape, dev = x.shape, x.device
    flat = len(shape) == 2
    rows, xr = (shape[0], x.stride()[0]) if flat else _rows(x, "x")
    D = shape[-1]
    rr = ror = rdt = wdt = wp = rp = rop = 0
    if weight is not None:
        wdt, wp = _row_weight(weight, (D,), i, grad, dev)
    if residual is not None:
        try:
            rd, (rr, r1) = residual.dtype, residual.stride()
            fits = flat and r1 == 1 and residual.shape == shape and rd in _DTYPES and residual.get_device() == i and not (grad and residual.requires_grad)
        except (AttributeError, ValueError):
            fits = False
        if not fits:
            _tensors(residual=residual)
            _check(residual, "residual", shape, _IO, dev)
            rd, rr = residual.dtype, _rows(residual, "residual")[1]
        rdt, rp = _DTYPES[rd], residual.data_ptr()
        if residual_out is None:
            residual_out = _empty(shape, (D, 1), device=dev, dtype=rd) if flat else torch.empty(shape, device=dev, dtype=rd)
            ror = D
        else:
            _tensors(residual_out=residual_out)
            _check(residual_out, "residual_out", shape, (rd,), dev)
            ror = _rows(residual_out, "residual_out")[1]
        rop = residual_out.data_ptr()
    elif residual_out is not None:
        raise ValueError("residual_out needs a residual")
    q, qr, scale = _steps(shape[:-1], rows, D, dev)
    _launch("gdn_rows_int8", _pack_rows(ROWS_NORM, rows, D, 0, xd, rdt, wdt, eps, x.data_ptr(), rp, 0, wp, xr, rr, 0, ror, qr,
                                        rop, q.data_ptr(), scale.data_ptr()), i)
    return q, scale, residual_out


def _row_input(x, dims):
    """(device index, whether gradients are recorded, dtype code) of a checked x."""
    grad = torch.is_grad_enabled()
    try:
        i, xd, stride = x.get_device(), _DTYPES.get(x.dtype), x.stride()
        fits = xd is not None and i >= 0 and len(stride) >= dims and stride[-1] == 1 and not (grad and x.requires_grad)
    except AttributeError:
        fits = False
    if not fits:
        _first(x, "x", dims, _IO)
    return i, grad, xd


def _row_weight(weight, shape, i, grad, dev):
    try:
        wd = weight.dtype
        fits = (wd in _DTYPES and weight.shape == shape and weight.stride() == (1,) and weight.get_device() == i
                and not (grad and weight.requires_grad))
    except AttributeError:
        fits = False
    if not fits:
        _tensors(weight=weight)
        _check(weight, "weight", shape, _IO, dev)
    return _DTYPES[weight.dtype], weight.data_ptr()


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
    stride), d a multiple of 8 up to 256; weight: [d] (bf16 or fp32; None = 1).  q: [..., H * d]
    int8, its rows on 16-byte boundaries; scale: [...] fp32, one for all heads of a row."""
    if stream is not None:
        return _other_stream(stream, x, (x, gate, weight), lambda: gated_rms_norm_int8(x, gate, weight, eps=eps))
    r = (_quick or _bind_quick()).gated_rms_norm_int8(x, gate, weight, eps)
    if r is not None:
        return r if type(r) is not int else _failed(r)
    i, grad, xd = _row_input(x, 2)
    dev = x.device
    shape = x.shape
    *lead, H, d = shape
    try:
        fits = (gate.shape == shape and gate.dtype is x.dtype and gate.get_device() == i and gate.stride()[-1] == 1
                and not (grad and gate.requires_grad))
    except AttributeError:
        fits = False
    if not fits:
        _tensors(gate=gate)
        _check(gate, "gate", shape, (x.dtype,), dev)
    wdt = wp = 0
    if weight is not None:
        wdt, wp = _row_weight(weight, (d,), i, grad, dev)
    rows, xr = _head_rows(x, "x")
    gr = _head_rows(gate, "gate")[1]
    q, qr, scale = _steps(lead, rows, H * d, dev)
    _launch("gdn_rows_int8", _pack_rows(ROWS_GATED, rows, H * d, d, xd, 0, wdt, eps, x.data_ptr(), 0, gate.data_ptr(), wp, xr,
                                        0, gr, 0, qr, 0, q.data_ptr(), scale.data_ptr()), i)
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
    i, _, xd = _row_input(x, 1)
    D = x.shape[-1]
    rows, xr = _rows(x, "x")
    q, qr, scale = _steps(x.shape[:-1], rows, D, x.device)
    _launch("gdn_rows_int8", _pack_rows(ROWS_PLAIN, rows, D, 0, xd, 0, 0, 0.0, x.data_ptr(), 0, 0, 0, xr, 0, 0, 0, qr, 0,
                                        q.data_ptr(), scale.data_ptr()), i)
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
    grad = torch.is_grad_enabled()
    try:
        shape, i = x.shape, x.get_device()
        lead, K = shape[:-1], shape[-1]
        N, wk = w.shape
        wr, w1 = w.stride()
        fits = (i >= 0 and x.dtype is torch.int8 and x.stride()[-1] == 1 and wk == K and w1 == 1 and w.dtype is torch.int8
                and w.get_device() == i and w_scale.shape == (N,) and w_scale.dtype is torch.float32 and w_scale.stride() == (1,)
                and w_scale.get_device() == i and x_scale.shape == lead and x_scale.dtype is torch.float32
                and x_scale.get_device() == i and x_scale.is_contiguous() and not (grad and (x_scale.requires_grad or w_scale.requires_grad)))
    except (AttributeError, TypeError, ValueError, IndexError):
        fits = False
    dev = x.device if fits else _product_refuse(x, x_scale, w, w_scale)
    bp = 0
    if bias is not None:
        _tensors(bias=bias)
        if not (bias.shape == (N,) and bias.dtype is torch.float32 and bias.stride() == (1,) and bias.get_device() == i and not (grad and bias.requires_grad)):
            _check(bias, "bias", (N,), _F32, dev)
        bp = bias.data_ptr()
    M, xr = _rows(x, "x")
    od = _code(out_dtype)
    if out is None:
        out = _empty((M, N), (N, 1), device=dev, dtype=out_dtype) if len(lead) == 1 else torch.empty((*lead, N), device=dev, dtype=out_dtype)
        outr = N
    else:
        _tensors(out=out)
        _check(out, "out", (*lead, N), (out_dtype,), dev)
        outr = _rows(out, "out")[1]
    xp, wp = x.data_ptr(), w.data_ptr()
    fields = (M, N, K, od, xp, wp, xr, wr, outr, x_scale.data_ptr(), w_scale.data_ptr(), bp, out.data_ptr())
    ws = need = 0
    if (xp | wp | xr | wr) & 15 or not xr or not wr:
        # from torch's allocator and not kept: a call's copies belong to its stream, or its graph
        need = lib().gdn_int8_matmul_workspace_bytes(_pack_matmul(*fields, 0, 0))
        if need:
            buffer = _empty((need,), (1,), device=dev, dtype=torch.uint8)
            ws = buffer.data_ptr()
    _launch("gdn_int8_matmul", _pack_matmul(*fields, ws, need), i)
    return out


def _product_refuse(x, x_scale, w, w_scale):
    """Raises for what int8_matmul does not take; the device where only its quick test was too
    strict."""
    _tensors(x=x, x_scale=x_scale, w=w, w_scale=w_scale)
    if w.dim() != 2:
        raise ValueError("w must be [N, K]")
    _first(x, "x", 1, _I8)
    _check(w, "w", (w.shape[0], x.shape[-1]), _I8, x.device)
    _check(w_scale, "w_scale", (w.shape[0],), _F32, x.device)
    _check_scale(x_scale, x.shape[:-1], x.device)
    return x.device


def _check_scale(t, lead, dev):
    if not t.is_contiguous():
        raise ValueError("x_scale must be contiguous")
    if t.dim() == 0:
        if len(lead):
            raise ValueError(f"x_scale has shape (), expected {tuple(lead)}")
        t, lead = t.view(1), (1,)
    _check(t, "x_scale", lead, _F32, dev)
