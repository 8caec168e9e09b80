"""Bindings of the operators around the recurrence (C ABI: include/gdn.h).

A recurrent layer takes its projections through ``gdn_causal_conv``, runs a
recurrence over the tokens (``gdn_step_record`` or ``gdn_selective_scan``) and
normalises the result with ``gdn_gated_norm``; ``gdn_sample`` draws tokens,
and the count of those that match a draft is the ``accepted`` of the replay
calls.  As with the other calls, these functions check tensor metadata,
allocate missing outputs and forward pointers and the current stream (or
``stream``, to which the allocations then belong).

``lengths`` is an int32 device tensor [B]: the steps that each sequence has
(clamped to 0..T).  ``y`` is not written at or past it.  A sequence is rolled
back by repeating a call from its earlier state with ``lengths=accepted`` and
``write_y=False``.
"""
from __future__ import annotations

import ctypes
import functools
from collections import namedtuple

import torch

import linear_attention_recurrence_step_gb300 as _pkg

from . import DTYPE_CODES, _check, _empty, _need, _need_workspace, load

ConvOutputs = namedtuple("ConvOutputs", "y state_out")
ScanOutputs = namedtuple("ScanOutputs", "y state_out")
NormOutputs = namedtuple("NormOutputs", "y residual_out")
SampleOutputs = namedtuple("SampleOutputs", "token logprob")

ACTIVATIONS = {None: 0, "none": 0, "silu": 1}
_raw_stream = torch._C._cuda_getCurrentRawStream


def _stream(dev, stream) -> int:
    if stream is None:
        return _raw_stream(dev)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


# The checks below run on every call, and a short kernel takes no longer than
# they do: each first tries the one comparison that a good argument passes,
# and leaves the wording of the error to _need.
def _lib():
    return _pkg._lib or load()


def _dense(t, name, shape, dtype, dev):
    """The pointer of a dense tensor on CUDA device `dev` (None for None), or the error of ``_need``."""
    if t is None:
        return None
    try:
        if t.shape == shape and t.dtype is dtype and t.get_device() == dev and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _need(t, name, shape, dtype, torch.device("cuda", dev))
    return t.data_ptr()


def _device_of(t, name):
    """The CUDA device index of a floating tensor, the current one."""
    try:
        if t.dtype in DTYPE_CODES and t.is_cuda:
            dev = t.get_device()
            if _pkg._one_device or _pkg._is_current(dev):
                return dev
            raise _pkg._other_device(dev)
    except AttributeError:
        raise TypeError(f"{name} must be a torch.Tensor") from None
    if t.dtype not in DTYPE_CODES:
        raise ValueError(f"unsupported dtype {t.dtype}")
    raise ValueError(f"{name} is on {t.device}, expected a CUDA device")


def _shape(t, name, dims, what):
    """The shape of a tensor of `dims` dimensions."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != dims:
        raise ValueError(f"{name} must be {what} (shape {tuple(t.shape)})")
    return t.shape


def _strided(t, name, shape, dtype, dev):
    """Batch and step strides of a [B,T,...] tensor whose inner dimensions are dense."""
    try:
        good = t.shape == shape and t.dtype is dtype and t.get_device() == dev
    except AttributeError:
        raise TypeError(f"{name} must be a torch.Tensor") from None
    if not good:
        at = torch.device("cuda", dev)
        _need(t.contiguous() if t.device == at else t, name, shape, dtype, at)
    dense = 1
    if t.is_contiguous():
        for n in shape[2:]:
            dense *= n
        return dense * shape[1], dense
    st = t.stride()
    for i in range(len(shape) - 1, 1, -1):
        if st[i] != dense and shape[i] != 1:
            raise ValueError(f"{name}'s dimensions after the second must be dense (strides {st})")
        dense *= shape[i]
    # a stride of a dimension of one is never used: give one that keeps rows apart
    step = st[1] if shape[1] > 1 else dense
    return (st[0] if shape[0] > 1 else step * shape[1]), step


def _rows(t, name, inner_dims, must=True):
    """Row stride of a tensor [..., inner] whose leading dimensions collapse into
    one; of another, the error (or None, unless it `must`)."""
    shape = t.shape
    lead = len(shape) - inner_dims
    dense = 1
    if t.is_contiguous():
        for n in shape[lead:]:
            dense *= n
        return dense
    st = t.stride()
    for i in range(len(shape) - 1, lead - 1, -1):
        if st[i] != dense and shape[i] != 1:
            if not must:
                return None
            raise ValueError(f"{name}'s last dimension(s) must be dense (strides {st})")
        dense *= shape[i]
    row, count = None, 1
    for i in range(lead - 1, -1, -1):
        if shape[i] == 1:
            continue
        if row is None:
            row = st[i]
        elif st[i] != row * count:
            if not must:
                return None
            raise ValueError(f"{name}'s leading dimensions must collapse into one (strides {st})")
        count *= shape[i]
    return dense if row is None else row


def gdn_causal_conv(x, weight, state_in=None, *, bias=None, lengths=None, activation="silu", y=None,
                    state_out=None, write_y: bool = True, stream=None) -> ConvOutputs:
    """Short causal convolution over [B,T,C] with its state.

    ``weight`` is [C,W] (W from 2 to 8, tap W-1 on the current step),
    ``state_in`` the last W-1 inputs [B,W-1,C] (None: zeros).  ``x`` may be a
    slice of a wider projection.  ``state_out=state_in`` runs in place;
    ``write_y=False`` only moves the state."""
    dev = _device_of(x, "x")
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {sorted(map(str, ACTIVATIONS))}")
    dt = x.dtype
    try:
        B, T, C = x.shape
        _, W = weight.shape
    except (AttributeError, ValueError):
        B, T, C = _shape(x, "x", 3, "[B,T,C]")
        W = _shape(weight, "weight", 2, "[C,W]")[1]
    sb, st = _strided(x, "x", (B, T, C), dt, dev)
    if write_y:
        if y is None:
            y = _empty((B, T, C), dt, x.device, stream)
    elif y is not None:
        raise ValueError("y is given but write_y is False")
    if state_out is None:
        state_out = _empty((B, W - 1, C), dt, x.device, stream)
    status = _lib().gdn_causal_conv(
        x.data_ptr(), _dense(weight, "weight", (C, W), dt, dev), _dense(bias, "bias", (C,), dt, dev),
        _dense(state_in, "state_in", (B, W - 1, C), dt, dev), _dense(lengths, "lengths", (B,), torch.int32, dev),
        _dense(y, "y", (B, T, C), dt, dev), _dense(state_out, "state_out", (B, W - 1, C), dt, dev),
        B, T, C, W, sb, st, ACTIVATIONS[activation], DTYPE_CODES[dt], _stream(dev, stream))
    if status:
        _check(status, "gdn_causal_conv")
    return ConvOutputs(y, state_out)


class _ScanStrides(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("x_b", "x_t", "dt_b", "dt_t", "B_b", "B_t", "C_b", "C_t")]


def gdn_selective_scan_workspace_size(B: int, T: int, H: int, P: int, N: int) -> int:
    """Bytes of device workspace gdn_selective_scan needs (0 for invalid sizes)."""
    return int(load().gdn_selective_scan_workspace_size(B, T, H, P, N))


_scan_workspace = functools.lru_cache(maxsize=256)(gdn_selective_scan_workspace_size)  # a function of the sizes alone


def gdn_selective_scan(x, dt, A, B, C, state_in=None, *, D=None, dt_bias=None, softplus: bool = True,
                       lengths=None, y=None, state_out=None, write_y: bool = True, workspace=None,
                       stream=None) -> ScanOutputs:
    """Selective state space scan with one decay per head and step.

    x [B,T,H,P], dt [B,T,H], B and C [B,T,G,N] (element type of x, slices of
    wider projections allowed), A, D and dt_bias [H] float32, state
    [B,H,P,N] float32 (None: zeros).  ``workspace`` (a device tensor of at
    least ``gdn_selective_scan_workspace_size(B, T, H, P, N)`` bytes) is
    allocated when not given."""
    dev = _device_of(x, "x")
    et = x.dtype
    try:
        nb, T, H, P = x.shape
        _, _, G, N = B.shape
    except (AttributeError, ValueError):
        nb, T, H, P = _shape(x, "x", 4, "[B,T,H,P]")
        _, _, G, N = _shape(B, "B", 4, "[B,T,G,N]")
    strides = _ScanStrides(*_strided(x, "x", (nb, T, H, P), et, dev), *_strided(dt, "dt", (nb, T, H), et, dev),
                           *_strided(B, "B", (nb, T, G, N), et, dev), *_strided(C, "C", (nb, T, G, N), et, dev))
    if write_y:
        if y is None:
            y = _empty((nb, T, H, P), et, x.device, stream)
    elif y is not None:
        raise ValueError("y is given but write_y is False")
    shape = (nb, H, P, N)
    if state_out is None:
        state_out = _empty(shape, torch.float32, x.device, stream)
    if workspace is None:
        need = _scan_workspace(nb, T, H, P, N)
        if need > 16:
            workspace = _empty(need, torch.uint8, x.device, stream)
    else:
        _need_workspace(workspace, x.device)
    f32 = torch.float32
    status = _lib().gdn_selective_scan(
        x.data_ptr(), dt.data_ptr(), _dense(A, "A", (H,), f32, dev), B.data_ptr(), C.data_ptr(),
        _dense(D, "D", (H,), f32, dev), _dense(dt_bias, "dt_bias", (H,), f32, dev),
        _dense(state_in, "state_in", shape, f32, dev), _dense(lengths, "lengths", (nb,), torch.int32, dev),
        _dense(y, "y", (nb, T, H, P), et, dev), _dense(state_out, "state_out", shape, f32, dev),
        nb, T, H, P, G, N, ctypes.byref(strides), 1 if softplus else 0,
        None if workspace is None else workspace.data_ptr(),
        0 if workspace is None else workspace.numel() * workspace.element_size(),
        DTYPE_CODES[et], _stream(dev, stream))
    if status:
        _check(status, "gdn_selective_scan")
    return ScanOutputs(y, state_out)


def gdn_gated_norm(x, weight, *, gate=None, gate_first: bool = False, residual=None,
                   residual_scale: float = 1.0, eps: float = 1e-6, y=None, residual_out=None,
                   stream=None) -> NormOutputs:
    """Root-mean-square norm of x [..., D] with its gate and residual sum.

    ``weight`` is [D], or [K,D] for x [...,K,D] (one row per head).  ``gate``
    multiplies by silu(gate) after the norm, or before it with
    ``gate_first``.  With ``residual`` the norm is of ``residual +
    residual_scale * x``, which is also returned.  x and gate may be slices
    of wider rows [..., D] or of wider tokens [..., K, D]."""
    dev = _device_of(x, "x")
    dt, shape = x.dtype, x.shape
    if not isinstance(weight, torch.Tensor) or weight.dim() not in (1, 2):
        raise ValueError("weight must be a tensor [D] or [K,D]")
    if not shape:
        raise ValueError("x must be [..., D]")
    D = shape[-1]
    per_head = weight.dim() == 2
    if gate is not None and (not isinstance(gate, torch.Tensor) or gate.shape != shape or gate.dtype is not dt
                             or gate.get_device() != dev):
        _need(gate.contiguous() if isinstance(gate, torch.Tensor) and gate.device == x.device else gate, "gate", shape,
              dt, x.device)
    # a shared weight: rows [..., D], if x and gate are both that; else tokens of
    # K heads each [..., K, D]
    if not per_head and x.is_contiguous() and (gate is None or gate.is_contiguous()):
        K, xs, gs = 1, D, D
    else:
        K, xs = 1, None if per_head else _rows(x, "x", 1, len(shape) < 2)
        gs = xs if gate is None or xs is None else _rows(gate, "gate", 1, len(shape) < 2)
        if gs is None:
            if len(shape) < 2:
                raise ValueError("x must be [..., K, D]")
            K = shape[-2]
            xs = _rows(x, "x", 2)
            gs = xs if gate is None else _rows(gate, "gate", 2)
    M = x.numel() // (K * D) if x.numel() else 0
    if y is None:
        y = _empty(shape, dt, x.device, stream)
    if residual is not None and residual_out is None:
        residual_out = _empty(shape, dt, x.device, stream)
    elif residual is None and residual_out is not None:
        raise ValueError("residual_out is given but residual is not")
    status = _lib().gdn_gated_norm(
        x.data_ptr(), _dense(weight, "weight", (K, D) if per_head else (D,), dt, dev),
        None if gate is None else gate.data_ptr(), _dense(residual, "residual", shape, dt, dev),
        _dense(y, "y", shape, dt, dev), _dense(residual_out, "residual_out", shape, dt, dev),
        M, K, D, xs, gs, K if per_head else 1, 1 if gate_first else 0, residual_scale, eps,
        DTYPE_CODES[dt], _stream(dev, stream))
    if status:
        _check(status, "gdn_gated_norm")
    return NormOutputs(y, residual_out)


def _setting(v, name, shape, dtype, dev, kind):
    """(pointer, value) of a setting given per row (a device tensor) or for all rows."""
    if isinstance(v, torch.Tensor):
        return _dense(v, name, shape, dtype, dev), 0
    return None, kind(v)


def gdn_sample(logits, noise, *, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, token=None, logprob=None,
               stream=None) -> SampleOutputs:
    """One token per row of logits [..., V] from standard exponential noise.

    ``noise`` (float32, the shape of logits) is given, e.g. by
    ``torch.empty(...).exponential_()``.  Each setting is a number, or a
    device tensor with one value per row (int32 for top_k, else float32).
    Returns the tokens (int32, -1 where every logit is -inf) and their log
    probability under the softmax at the row's temperature, before the cuts."""
    dev = _device_of(logits, "logits")
    dt, shape = logits.dtype, logits.shape
    if not shape:
        raise ValueError("logits must be [..., V]")
    V, lead = shape[-1], shape[:-1]
    ls = _rows(logits, "logits", 1)
    if not isinstance(noise, torch.Tensor) or noise.shape != shape or noise.dtype is not torch.float32 \
            or noise.get_device() != dev:
        _need(noise, "noise", shape, torch.float32, logits.device)
    ns = _rows(noise, "noise", 1)
    if token is None:
        token = _empty(lead, torch.int32, logits.device, stream)
    if logprob is None:
        logprob = _empty(lead, torch.float32, logits.device, stream)
    f32 = torch.float32
    tp, tv = _setting(temperature, "temperature", lead, f32, dev, float)
    kp, kv = _setting(top_k, "top_k", lead, torch.int32, dev, int)
    pp, pv = _setting(top_p, "top_p", lead, f32, dev, float)
    mp, mv = _setting(min_p, "min_p", lead, f32, dev, float)
    status = _lib().gdn_sample(
        logits.data_ptr(), noise.data_ptr(), tp, kp, pp, mp, tv, kv, pv, mv,
        _dense(token, "token", lead, torch.int32, dev), _dense(logprob, "logprob", lead, f32, dev),
        logits.numel() // V if V else 0, V, ls, ns, DTYPE_CODES[dt], _stream(dev, stream))
    if status:
        _check(status, "gdn_sample")
    return SampleOutputs(token, logprob)
