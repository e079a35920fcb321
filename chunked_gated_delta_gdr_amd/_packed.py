"""ctypes binding of the packed forms and the RMS norm of libgdr.so (see include/gdr.h).

Same names as the C ABI.  The functions check their tensors, fill the structs and launch on the
current stream (or ``stream``) of the tensors' device; they never synchronise.
"""
from __future__ import annotations

import ctypes
import functools
import inspect
from typing import Optional, Tuple

import torch

from . import _binding as B

GDR_F16 = 2
GDR_OUT_IO, GDR_OUT_INT8, GDR_OUT_FP8 = 0, 1, 2
_IO = {torch.float32: B.GDR_F32, torch.bfloat16: B.GDR_BF16, torch.float16: GDR_F16}
_OUT = {None: GDR_OUT_IO, torch.int8: GDR_OUT_INT8, torch.float8_e4m3fn: GDR_OUT_FP8}


class gdr_packed_desc_t(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_uint32)] + [
        (n, ctypes.c_int32) for n in ("n_tokens", "n_seqs", "Hk", "Hv", "Dk", "Dv", "n_slots", "io_dtype",
                                      "decay", "qk_norm", "impl")] + [
        (n, ctypes.c_float) for n in ("scale", "qk_eps", "norm_eps")] + [
        (n, ctypes.c_int64) for n in ("q_stride", "k_stride", "v_stride", "out_stride", "gate_stride")]


class gdr_packed_inputs_t(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("q", "k", "v", "beta", "log_alpha", "cu_seqlens", "state_index",
                                               "has_state", "norm_weight", "norm_gate")]


class gdr_norm_desc_t(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_uint32)] + [
        (n, ctypes.c_int32) for n in ("rows", "D", "io_dtype", "out_kind")] + [("eps", ctypes.c_float)] + [
        (n, ctypes.c_int64) for n in ("x_stride", "residual_stride", "gate_stride", "dy_stride")]


_vp, _u64, _P = ctypes.c_void_p, ctypes.c_uint64, ctypes.POINTER


@functools.lru_cache(maxsize=None)
def _lib() -> ctypes.CDLL:
    L = B.lib()
    pd, pi, nd = _P(gdr_packed_desc_t), _P(gdr_packed_inputs_t), _P(gdr_norm_desc_t)
    for name, args, res in (
            ("gdr_packed_fwd", [pd, pi, _vp, _vp, _vp, _u64, _vp], ctypes.c_int),
            ("gdr_packed_step", [pd, pi, _vp, _vp, _vp], ctypes.c_int),
            ("gdr_packed_fwd_workspace_size", [pd], _u64),
            ("gdr_packed_fwd_impl", [pd], ctypes.c_int),
            ("gdr_validate_packed", [pd, pi, _vp, _vp, _vp, _u64, ctypes.c_int], ctypes.c_int),
            ("gdr_rms_norm", [nd] + [_vp] * 8, ctypes.c_int),
            ("gdr_rms_norm_bwd", [nd] + [_vp] * 9 + [_u64, _vp], ctypes.c_int),
            ("gdr_rms_norm_bwd_workspace_size", [nd], _u64),
            ("gdr_validate_norm", [nd] + [_vp] * 7, ctypes.c_int),
            ("gdr_validate_norm_bwd", [nd] + [_vp] * 9 + [_u64], ctypes.c_int)):
        f = getattr(L, name)
        f.argtypes, f.restype = args, res
    return L


# ------------------------------------------------------------------------------------
# descriptors: by value, so that calls of one shape share them (fields are plain numbers: a tensor
# would be found again by its identity, whatever it holds by then)
# ------------------------------------------------------------------------------------

@functools.lru_cache(maxsize=1024)
def _packed_desc(*fields) -> gdr_packed_desc_t:
    return gdr_packed_desc_t(ctypes.sizeof(gdr_packed_desc_t), *fields)


@functools.lru_cache(maxsize=1024)
def _norm_desc(*fields) -> gdr_norm_desc_t:
    return gdr_norm_desc_t(ctypes.sizeof(gdr_norm_desc_t), *fields)


@functools.lru_cache(maxsize=1024)
def _packed_ws(*fields) -> int:
    return int(_lib().gdr_packed_fwd_workspace_size(_packed_desc(*fields)))


def make_packed_desc(*, n_tokens, n_seqs, Hk, Hv, Dk, Dv, n_slots=0, io_dtype=B.GDR_BF16, decay=B.GDR_DECAY_NONE,
                     qk_norm=0, impl=B.GDR_IMPL_AUTO, scale=1.0, qk_eps=1e-6, norm_eps=1e-6, q_stride=0, k_stride=0,
                     v_stride=0, out_stride=0, gate_stride=0) -> gdr_packed_desc_t:
    return gdr_packed_desc_t(ctypes.sizeof(gdr_packed_desc_t), n_tokens, n_seqs, Hk, Hv, Dk, Dv, n_slots, io_dtype,
                             decay, qk_norm, impl, scale, qk_eps, norm_eps, q_stride, k_stride, v_stride,
                             out_stride, gate_stride)


def make_norm_desc(*, rows, D, io_dtype=B.GDR_BF16, out_kind=GDR_OUT_IO, eps=1e-6, x_stride=0, residual_stride=0,
                   gate_stride=0, dy_stride=0) -> gdr_norm_desc_t:
    return gdr_norm_desc_t(ctypes.sizeof(gdr_norm_desc_t), rows, D, io_dtype, out_kind, eps, x_stride,
                           residual_stride, gate_stride, dy_stride)


def gdr_validate_packed(desc, inputs, pool=None, out=None, workspace=None, workspace_bytes=0, for_step=False) -> int:
    """Host-side argument check of gdr_packed_fwd and gdr_packed_step (no HIP call).  Pointers are ints or None."""
    return _lib().gdr_validate_packed(ctypes.byref(desc), ctypes.byref(inputs), pool, out, workspace, workspace_bytes,
                                      int(for_step))


def gdr_validate_norm(desc, x=None, residual=None, weight=None, gate=None, y=None, scales=None, residual_out=None) -> int:
    """gdr_rms_norm's host-side argument check (no HIP call).  Pointers are ints or None."""
    return _lib().gdr_validate_norm(ctypes.byref(desc), x, residual, weight, gate, y, scales, residual_out)


def gdr_validate_norm_bwd(desc, x=None, dy=None, weight=None, gate=None, d_residual=None, dx=None, dweight=None,
                          dgate=None, workspace=None, workspace_bytes=0) -> int:
    """gdr_rms_norm_bwd's host-side argument check (no HIP call).  Pointers are ints or None."""
    return _lib().gdr_validate_norm_bwd(ctypes.byref(desc), x, dy, weight, gate, d_residual, dx, dweight, dgate,
                                        workspace, workspace_bytes)


def gdr_packed_fwd_impl(desc) -> int:
    """Which kernel gdr_packed_fwd runs for a descriptor (GDR_IMPL_*; -1: none)."""
    return _lib().gdr_packed_fwd_impl(ctypes.byref(desc))


def gdr_packed_fwd_workspace_size(desc) -> int:
    return int(_lib().gdr_packed_fwd_workspace_size(ctypes.byref(desc)))


def gdr_rms_norm_bwd_workspace_size(desc) -> int:
    return int(_lib().gdr_rms_norm_bwd_workspace_size(ctypes.byref(desc)))


# ------------------------------------------------------------------------------------
# torch marshalling
# ------------------------------------------------------------------------------------

_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


class _On:
    """The device and stream that a call's allocations and launch go to, where they are not the
    current ones."""

    def __init__(self, device, stream):
        self.ctx = [torch.cuda.device(device)]
        if stream is not None:
            if not hasattr(stream, "cuda_stream"):
                stream = torch.cuda.ExternalStream(int(stream), device=device)
            if stream.device != device:
                raise ValueError(f"stream of {stream.device}, tensors on {device}")
            self.ctx.append(torch.cuda.stream(stream))

    def __enter__(self):
        for c in self.ctx:
            c.__enter__()

    def __exit__(self, *exc):
        for c in reversed(self.ctx):
            c.__exit__(*exc)


def _placed(call):
    """Adds ``stream`` to ``call``'s keyword arguments: it runs with its first argument's device
    current, on ``stream`` where one is given."""
    sig = inspect.signature(call)
    first = next(iter(sig.parameters))

    @functools.wraps(call)
    def placed(*args, stream=None, **kw):
        x = args[0] if args else kw.get(first)
        if x is None:
            return call(*args, **kw)   # (names what is missing)
        index = x.get_device()
        if index < 0:
            raise ValueError(f"tensors must be on a GPU, not on {x.device}")
        if stream is None and torch.cuda.current_device() == index:
            return call(*args, **kw)
        with _On(x.device, stream):
            return call(*args, **kw)
    placed.__signature__ = sig.replace(parameters=[
        *sig.parameters.values(), inspect.Parameter("stream", inspect.Parameter.KEYWORD_ONLY, default=None)])
    return placed


def _rows(name, t, shape, width, dtype, index) -> int:
    """Checks rows of contiguous trailing dimensions (``width`` elements) and returns the elements
    between them."""
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name}: device {t.device}, expected GPU {index}")
    if t.is_contiguous():
        return width
    strides, w = t.stride(), 1
    for n, st in zip(reversed(shape[1:]), reversed(strides[1:])):
        if st != w and n > 1:
            raise ValueError(f"{name}: the dimensions within a row must be contiguous")
        w *= n
    if shape[0] <= 1:
        return width
    if strides[0] < width:
        raise ValueError(f"{name}: rows {strides[0]} elements apart overlap (a row has {width})")
    return strides[0]


def _flat(name, t, shape, dtypes, index):
    if t is None:
        return None
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtypes[0]}")
    if t.get_device() != index:
        raise ValueError(f"{name}: device {t.device}, expected GPU {index}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _new_rows(like, dtype):
    """A contiguous tensor of ``like``'s shape (cheaper than from a shape and a device)."""
    return torch.empty_like(like, dtype=dtype, memory_format=torch.contiguous_format)


def _scratch(workspace, need, index, device):
    """(tensor, pointer, bytes) of the caller's workspace or of one of ``need`` bytes."""
    if workspace is None:
        if not need:
            return None, None, 0
        workspace = torch.empty(need, dtype=torch.uint8, device=device)   # (an allocation is 512-byte aligned)
    elif workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the inputs' device")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


_F32, _I32, _FLAG = (torch.float32,), (torch.int32,), (torch.bool, torch.uint8)


def _packed(q, k, v, n_seqs, cu_seqlens, beta, log_alpha, state, state_index, has_state, qk_norm, qk_eps, norm_weight,
            norm_gate, norm_eps, out, scale, impl):
    """(descriptor fields, inputs, pool pointer) of a packed call."""
    N, Hk, Dk = q.shape
    _, Hv, Dv = v.shape
    index, io = q.get_device(), q.dtype
    code = _IO.get(io)
    if code is None:
        raise TypeError(f"unsupported io dtype {io} (float32, bfloat16 or float16)")
    kw, vw, heads, values = Hk * Dk, Hv * Dv, (N, Hv), (N, Hv, Dv)
    qs = _rows("q", q, (N, Hk, Dk), kw, io, index)
    ks = _rows("k", k, (N, Hk, Dk), kw, io, index)
    vs = _rows("v", v, values, vw, io, index)
    os_ = _rows("out", out, values, vw, io, index)
    zs = 0 if norm_gate is None else _rows("norm_gate", norm_gate, values, vw, io, index)
    slots, pool = 0, None
    if state is not None:
        slots = state.shape[0]
        if slots == 0 and n_seqs > 0:   # (its pointer is null, which means no pool at all)
            raise ValueError("state has no slots")
        pool = _flat("state", state, (slots, Hv, Dv, Dk), _F32, index)
    if beta is None:
        raise ValueError("beta is required")
    ins = gdr_packed_inputs_t(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), _flat("beta", beta, heads, _F32, index),
        _flat("log_alpha", log_alpha, heads, _F32, index),
        _flat("cu_seqlens", cu_seqlens, (n_seqs + 1,), _I32, index),
        _flat("state_index", state_index, (n_seqs,), _I32, index),
        _flat("has_state", has_state, (n_seqs,), _FLAG, index),
        _flat("norm_weight", norm_weight, (Dv,), (io,), index),
        None if norm_gate is None else norm_gate.data_ptr())
    fields = (N, n_seqs, Hk, Hv, Dk, Dv, slots, code, B.GDR_DECAY_NONE if log_alpha is None else B.GDR_DECAY_SCALAR,
              int(qk_norm), impl, float(scale), float(qk_eps), float(norm_eps), qs, ks, vs, os_, zs)
    return fields, ins, pool


@_placed
def gdr_packed_fwd(q, k, v, cu_seqlens, *, beta, log_alpha=None, state=None, state_index=None, has_state=None,
                   qk_norm: bool = False, qk_eps: float = 1e-6, norm_weight=None, norm_gate=None,
                   norm_eps: float = 1e-6, out=None, scale: float = 1.0, impl: str = "auto", workspace=None):
    """The gated delta rule over sequences packed on one token axis.  Returns ``out`` [N, Hv, Dv].

    ``q``, ``k`` [N, Hk, Dk] and ``v`` [N, Hv, Dv] may be parts of wider rows; ``beta``,
    ``log_alpha`` [N, Hv] fp32; ``cu_seqlens`` [n + 1] int32 on the GPU.  ``state`` is the pool
    [slots, Hv, Dv, Dk] fp32, read and written in place at ``state_index`` [n] int32 (None:
    sequence s has slot s; negative: the sequence is skipped); ``has_state`` [n] bool, False
    starts from zeros.  ``qk_norm`` divides q and k by their L2 norms.  ``norm_weight`` [Dv] and
    ``norm_gate`` [N, Hv, Dv] apply the output norm.  ``impl``: "auto", "generic" (token by
    token) or "mfma" (chunked).  Rows of ``out`` in no sequence, and of skipped ones, are not
    written (undefined in an ``out`` made here).  ``workspace``: a uint8 tensor of
    ``gdr_packed_fwd_workspace_size`` bytes, allocated when not given.  ``stream``: the stream to
    launch on (the current one by default).
    """
    n_seqs = cu_seqlens.numel() - 1
    if out is None:
        out = _new_rows(v, q.dtype)
    fields, ins, pool = _packed(q, k, v, n_seqs, cu_seqlens, beta, log_alpha, state, state_index, has_state, qk_norm,
                                qk_eps, norm_weight, norm_gate, norm_eps, out, scale, B._IMPL[impl])
    index = q.get_device()
    workspace, ws, nbytes = _scratch(workspace, _packed_ws(*fields), index, q.device)
    st = _lib().gdr_packed_fwd(_packed_desc(*fields), ins, pool, out.data_ptr(), ws, nbytes, _raw_stream(index))
    if st:
        B._raise(st)
    return out


@_placed
def gdr_packed_step(q, k, v, state, *, beta, log_alpha=None, cu_seqlens=None, state_index=None, has_state=None,
                    qk_norm: bool = False, qk_eps: float = 1e-6, norm_weight=None, norm_gate=None,
                    norm_eps: float = 1e-6, out=None, scale: float = 1.0):
    """One token for every sequence (or, with ``cu_seqlens``, a few), the states updated in place
    in their slots of the pool ``state``.  Arguments as gdr_packed_fwd's.  Returns ``out``."""
    n_seqs = q.shape[0] if cu_seqlens is None else cu_seqlens.numel() - 1
    if out is None:
        out = _new_rows(v, q.dtype)
    fields, ins, pool = _packed(q, k, v, n_seqs, cu_seqlens, beta, log_alpha, state, state_index, has_state, qk_norm,
                                qk_eps, norm_weight, norm_gate, norm_eps, out, scale, B.GDR_IMPL_AUTO)
    st = _lib().gdr_packed_step(_packed_desc(*fields), ins, pool, out.data_ptr(), _raw_stream(q.get_device()))
    if st:
        B._raise(st)
    return out


@_placed
def gdr_rms_norm(x, *, weight=None, residual=None, gate=None, out_dtype=None, out=None, scales=None, residual_out=None,
                 eps: float = 1e-6) -> Tuple[object, Optional[object], Optional[object]]:
    """RMS norm of the rows of ``x`` [rows, D]: of ``x + residual`` where a residual is given,
    times ``weight`` [D] and silu(``gate``) [rows, D].  ``out_dtype``: None (x's), torch.int8 or
    torch.float8_e4m3fn, then with a scale per row.  ``stream``: the stream to launch on (the
    current one by default).  Returns (out, scales, residual_out)."""
    rows, D = shape = x.shape
    index, io = x.get_device(), x.dtype
    code, kind = _IO.get(io), _OUT.get(out_dtype)
    if code is None:
        raise TypeError(f"unsupported io dtype {io} (float32, bfloat16 or float16)")
    if kind is None:
        raise TypeError(f"unsupported output dtype {out_dtype} (None, int8 or float8_e4m3fn)")
    xs = _rows("x", x, shape, D, io, index)
    rs = 0 if residual is None else _rows("residual", residual, shape, D, io, index)
    zs = 0 if gate is None else _rows("gate", gate, shape, D, io, index)
    if out is None:
        out = _new_rows(x, out_dtype or io)
        y = out.data_ptr()
    else:
        y = _flat("out", out, shape, (out_dtype or io,), index)
    if scales is None and kind != GDR_OUT_IO:
        scales = x.new_empty(rows, dtype=torch.float32)
        sc = scales.data_ptr()
    else:
        sc = _flat("scales", scales, (rows,), _F32, index)
    if residual_out is None and residual is not None:
        residual_out = _new_rows(x, io)
        total = residual_out.data_ptr()
    else:
        total = _flat("residual_out", residual_out, shape, (io,), index)
    st = _lib().gdr_rms_norm(
        _norm_desc(rows, D, code, kind, float(eps), xs, rs, zs, 0), x.data_ptr(),
        None if residual is None else residual.data_ptr(), _flat("weight", weight, (D,), (io,), index),
        None if gate is None else gate.data_ptr(), y, sc, total, _raw_stream(index))
    if st:
        B._raise(st)
    return out, scales, residual_out


@_placed
def gdr_rms_norm_bwd(x, dy, *, weight=None, gate=None, d_residual=None, want_dweight: bool = True, eps: float = 1e-6,
                     workspace=None) -> dict:
    """Gradient of gdr_rms_norm's output in x's dtype.  ``x`` [rows, D] is the normalised sum
    (``residual_out`` where there was a residual), ``dy`` its loss gradient, ``d_residual`` the
    gradient that reaches the sum from elsewhere.  Returns a dict: dx (of x and of the residual),
    dweight [D] fp32 (with ``weight`` and ``want_dweight``) and dgate (with ``gate``)."""
    rows, D = shape = x.shape
    index, io = x.get_device(), x.dtype
    code = _IO.get(io)
    if code is None:
        raise TypeError(f"unsupported io dtype {io} (float32, bfloat16 or float16)")
    xs, ds = _rows("x", x, shape, D, io, index), _rows("dy", dy, shape, D, io, index)
    rs = 0 if d_residual is None else _rows("d_residual", d_residual, shape, D, io, index)
    zs = 0 if gate is None else _rows("gate", gate, shape, D, io, index)
    desc = _norm_desc(rows, D, code, GDR_OUT_IO, float(eps), xs, rs, zs, ds)
    g = {"dx": _new_rows(x, io)}
    ws, nbytes = None, 0
    if weight is not None and want_dweight:
        g["dweight"] = x.new_empty(D, dtype=torch.float32)
        workspace, ws, nbytes = _scratch(workspace, gdr_rms_norm_bwd_workspace_size(desc), index, x.device)
    if gate is not None:
        g["dgate"] = _new_rows(x, io)
    st = _lib().gdr_rms_norm_bwd(
        desc, x.data_ptr(), dy.data_ptr(), _flat("weight", weight, (D,), (io,), index),
        None if gate is None else gate.data_ptr(), None if d_residual is None else d_residual.data_ptr(),
        g["dx"].data_ptr(), g["dweight"].data_ptr() if "dweight" in g else None,
        g["dgate"].data_ptr() if gate is not None else None, ws, nbytes, _raw_stream(index))
    if st:
        B._raise(st)
    return g
