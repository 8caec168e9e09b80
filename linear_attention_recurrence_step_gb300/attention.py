"""Bindings of the operators of an attention layer (C ABI: include/gdn.h).

A hybrid model's attention layer keeps its keys and values in pages of 4-bit
values (``gdn_kv_cache``).  A serving step takes the places of its new tokens
from ``gdn_page_slots``, turns queries and keys with ``gdn_rotary``, writes with
``gdn_kv_append`` and attends with ``gdn_kv_attention``:

    s = gdn_page_slots(lengths, add, held, ring_state, block_table, ring, T=T, page=page)
    r = gdn_rotary(q, s.positions, inv_freq, k=k)
    gdn_kv_append(r.k, v, s.slots, cache)
    y = gdn_kv_attention(r.q, cache, block_table, s.lengths_out, new=s.granted).y

``s.granted`` is also the ``lengths`` of the recurrent layers' calls.  To roll a
sequence back, shorten its length: its pages stay held, and the next call
writes over what was rejected.  As with the other calls, these functions check
tensor metadata, allocate missing outputs and forward pointers and the current
stream (or ``stream``, to which the allocations then belong).
"""
from __future__ import annotations

import ctypes
import functools
import math
from collections import namedtuple

import torch

import linear_attention_recurrence_step_gb300 as _pkg

from . import DTYPE_CODES, _check, _empty, _need, _need_workspace, load
from .layer import _dense, _device_of, _lib, _shape, _stream, _strided

SlotOutputs = namedtuple("SlotOutputs", "slots positions granted lengths_out held_out ring_state_out")
RotaryOutputs = namedtuple("RotaryOutputs", "q k")
KvOutputs = namedtuple("KvOutputs", "k v")
AttentionOutputs = namedtuple("AttentionOutputs", "y lse")

ROTARY_LAYOUTS = {"half": 0, "interleaved": 1}


def _int_device(t, name):
    """The CUDA device index of an int32 tensor, the current one."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not torch.int32:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {torch.int32}")
    if not t.is_cuda:
        raise ValueError(f"{name} is on {t.device}, expected a CUDA device")
    dev = t.get_device()
    if not (_pkg._one_device or _pkg._is_current(dev)):
        raise _pkg._other_device(dev)
    return dev


def gdn_page_slots(lengths, add, held, ring_state, block_table, ring, *, T: int, page: int, slots=None,
                   positions=None, granted=None, lengths_out=None, held_out=None, ring_state_out=None,
                   stream=None) -> SlotOutputs:
    """Block tables and slots of a step's tokens, from the requests' lengths.

    int32 device tensors: ``lengths`` and ``held`` [B] (tokens and pages of each
    sequence), ``add`` [B] (tokens to add, at most T; negative: the sequence
    ends; None: T for each), ``block_table`` [B,width] and ``ring`` [pages] (both
    changed in place), ``ring_state`` [2] (first free place of the ring, free
    pages).  Returns slots and positions [B,T] (-1: no token), the tokens
    ``granted``, and the new lengths, held pages and ring state;
    ``lengths_out=lengths`` and so on run in place."""
    dev = _int_device(lengths, "lengths")
    B = _shape(lengths, "lengths", 1, "[B]")[0]
    width = _shape(block_table, "block_table", 2, "[B,width]")[1]
    pages = _shape(ring, "ring", 1, "[pages]")[0]
    T, page = int(T), int(page)
    i32 = torch.int32
    at = lengths.device

    def out(t, shape):
        return _empty(shape, i32, at, stream) if t is None else t

    if T > 0 and B > 0:
        slots, positions, granted = out(slots, (B, T)), out(positions, (B, T)), out(granted, (B,))
        lengths_out, held_out, ring_state_out = out(lengths_out, (B,)), out(held_out, (B,)), out(ring_state_out, (2,))
    status = _lib().gdn_page_slots(
        _dense(lengths, "lengths", (B,), i32, dev), _dense(add, "add", (B,), i32, dev),
        _dense(held, "held", (B,), i32, dev), _dense(ring_state, "ring_state", (2,), i32, dev),
        _dense(block_table, "block_table", (B, width), i32, dev), _dense(ring, "ring", (pages,), i32, dev),
        _dense(slots, "slots", (B, T), i32, dev), _dense(positions, "positions", (B, T), i32, dev),
        _dense(granted, "granted", (B,), i32, dev), _dense(lengths_out, "lengths_out", (B,), i32, dev),
        _dense(held_out, "held_out", (B,), i32, dev), _dense(ring_state_out, "ring_state_out", (2,), i32, dev),
        B, T, width, pages, page, _stream(dev, stream))
    if status:
        _check(status, "gdn_page_slots")
    return SlotOutputs(slots, positions, granted, lengths_out, held_out, ring_state_out)


def rotary_frequencies(R: int, base: float = 10000.0, *, scaling: str | None = None, factor: float = 1.0,
                       trained: int | None = None, low: float = 1.0, high: float = 32.0, device=None):
    """(inv_freq [R/2] float32, scale) for ``gdn_rotary``.

    ``scaling`` stretches a context of ``trained`` tokens by ``factor``:
    ``None`` not at all; ``"linear"`` divides every frequency by the factor;
    ``"base"`` raises the base so that the lowest frequency is divided by it;
    ``"parts"`` divides the frequencies that make fewer than ``low`` turns over
    the trained context, keeps those above ``high`` and goes over from one to
    the other linearly in the turns; ``"parts_scaled"`` does so linearly in the
    frequency's index and scales by 1 + log(factor)/10 (the scores by its
    square)."""
    if R <= 0 or R % 2:
        raise ValueError("R must be even and > 0")
    if scaling not in (None, "linear", "base", "parts", "parts_scaled"):
        raise ValueError('scaling must be None, "linear", "base", "parts" or "parts_scaled"')
    if not factor >= 1.0:
        raise ValueError("factor must be at least 1")
    if not base > (1.0 if scaling == "parts_scaled" else 0.0):
        raise ValueError('base must be above 0, and above 1 for "parts_scaled"')
    i = torch.arange(0, R, 2, dtype=torch.float64)
    scale = 1.0
    if scaling == "base" and R > 2:
        base = base * factor ** (R / (R - 2))
    f = base ** -(i / R)
    if scaling == "linear":
        f = f / factor
    if scaling in ("parts", "parts_scaled"):
        if not trained or trained < 0 or not 0 < low < high:
            raise ValueError('"parts" needs trained > 0 and 0 < low < high')
        if scaling == "parts":
            keep = (trained * f / (2 * math.pi) - low) / (high - low)
        else:
            index = lambda turns: R * math.log(trained / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
            first = max(math.floor(index(high)), 0)
            last = min(math.ceil(index(low)), R - 1)
            keep = 1 - (i / 2 - first) / max(last - first, 1e-3)
            scale = 1 + 0.1 * math.log(factor)
        keep = keep.clamp(0, 1)
        f = f * (keep + (1 - keep) / factor)
    return f.float().to(device), scale


class _RotaryStrides(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("q_b", "q_t", "k_b", "k_t", "q_out_b", "q_out_t", "k_out_b", "k_out_t")]


def gdn_rotary(q, positions, inv_freq, *, k=None, layout: str = "half", scale: float = 1.0, inverse: bool = False,
               q_out=None, k_out=None, stream=None) -> RotaryOutputs:
    """Rotary positions of q [B,T,Hq,D] and k [B,T,Hk,D].

    ``positions`` [B,T] int32 (a token with a negative one is not written),
    ``inv_freq`` [R/2] float32: the first R channels of a head are turned, in
    pairs (i, i + R/2) of the ``layout`` "half" or (2i, 2i + 1) of
    "interleaved".  All four tensors may be slices of wider rows; ``q_out=q``
    and ``k_out=k`` run in place; ``inverse`` turns back."""
    dev = _device_of(q, "q")
    if layout not in ROTARY_LAYOUTS:
        raise ValueError(f"layout must be one of {sorted(ROTARY_LAYOUTS)}")
    dt = q.dtype
    B, T, Hq, D = _shape(q, "q", 4, "[B,T,Hq,D]")
    R = 2 * _shape(inv_freq, "inv_freq", 1, "[R/2]")[0]
    if q_out is None:
        q_out = _empty((B, T, Hq, D), dt, q.device, stream)
    qs, qos = _strided(q, "q", (B, T, Hq, D), dt, dev), _strided(q_out, "q_out", (B, T, Hq, D), dt, dev)
    Hk, kp, kop, ks, kos = 0, None, None, (0, 0), (0, 0)
    if k is not None:
        Hk = _shape(k, "k", 4, "[B,T,Hk,D]")[2]
        if k_out is None:
            k_out = _empty((B, T, Hk, D), dt, q.device, stream)
        ks, kos = _strided(k, "k", (B, T, Hk, D), dt, dev), _strided(k_out, "k_out", (B, T, Hk, D), dt, dev)
        kp, kop = k.data_ptr(), k_out.data_ptr()
    elif k_out is not None:
        raise ValueError("k_out is given but k is not")
    strides = _RotaryStrides(*qs, *ks, *qos, *kos)
    status = _lib().gdn_rotary(
        q.data_ptr(), kp, _dense(positions, "positions", (B, T), torch.int32, dev),
        _dense(inv_freq, "inv_freq", (R // 2,), torch.float32, dev), q_out.data_ptr(), kop, B, T, Hq, Hk, D, R,
        ctypes.byref(strides), ROTARY_LAYOUTS[layout], scale, 1 if inverse else 0, DTYPE_CODES[dt],
        _stream(dev, stream))
    if status:
        _check(status, "gdn_rotary")
    return RotaryOutputs(q_out, k_out)


def gdn_kv_cache(pages: int, H: int, page: int, D: int, *, device="cuda") -> torch.Tensor:
    """An empty cache (zeros) of `pages` pages of `page` tokens for H key heads
    of D channels: uint8 [pages, H, page, 9 D/8]."""
    if page not in (16, 32, 64, 128) or D not in (64, 128, 256):
        raise ValueError("page must be 16, 32, 64 or 128, and D 64, 128 or 256")
    return torch.zeros(pages, H, page, 9 * D // 8, dtype=torch.uint8, device=device)


def _cache(cache, dev):
    """pages, H, page and D of a cache on CUDA device `dev`."""
    pages, H, page, row = _shape(cache, "cache", 4, "[pages,H,page,9 D/8]")
    _dense(cache, "cache", (pages, H, page, row), torch.uint8, dev)
    if row % 9:
        raise ValueError(f"cache must be [pages,H,page,9 D/8] (shape {tuple(cache.shape)})")
    return pages, H, page, row // 9 * 8


def gdn_kv_append(k, v, slots, cache, *, k_scale=None, v_scale=None, stream=None) -> None:
    """Writes k and v [B,T,H,D] (slices of wider rows allowed) to the slots
    [B,T] int32 of the cache; a token with a negative slot is not written.
    ``k_scale`` and ``v_scale`` [H] float32 are the heads' scales (None: 1)."""
    dev = _device_of(k, "k")
    dt = k.dtype
    pages, H, page, D = _cache(cache, dev)
    B, T = _shape(k, "k", 4, "[B,T,H,D]")[:2]
    ks, vs = _strided(k, "k", (B, T, H, D), dt, dev), _strided(v, "v", (B, T, H, D), dt, dev)
    f32 = torch.float32
    status = _lib().gdn_kv_append(
        k.data_ptr(), v.data_ptr(), _dense(slots, "slots", (B, T), torch.int32, dev), cache.data_ptr(),
        _dense(k_scale, "k_scale", (H,), f32, dev), _dense(v_scale, "v_scale", (H,), f32, dev), B, T, H, D, page, pages,
        *ks, *vs, DTYPE_CODES[dt], _stream(dev, stream))
    if status:
        _check(status, "gdn_kv_append")


def gdn_kv_read(cache, slots, *, dtype=torch.bfloat16, k_scale=None, v_scale=None, k=None, v=None,
                stream=None) -> KvOutputs:
    """Keys and values [..., H, D] of the slots [...] int32, in ``dtype``; the
    rows of a negative slot are not written."""
    dev = _int_device(slots, "slots")
    if dtype not in DTYPE_CODES:
        raise ValueError(f"unsupported dtype {dtype}")
    pages, H, page, D = _cache(cache, dev)
    shape = (*slots.shape, H, D)
    if k is None:
        k = _empty(shape, dtype, slots.device, stream)
    if v is None:
        v = _empty(shape, dtype, slots.device, stream)
    f32 = torch.float32
    status = _lib().gdn_kv_read(
        cache.data_ptr(), _dense(slots, "slots", tuple(slots.shape), torch.int32, dev),
        _dense(k_scale, "k_scale", (H,), f32, dev), _dense(v_scale, "v_scale", (H,), f32, dev),
        _dense(k, "k", shape, dtype, dev), _dense(v, "v", shape, dtype, dev), slots.numel(), H, D, page, pages,
        DTYPE_CODES[dtype], _stream(dev, stream))
    if status:
        _check(status, "gdn_kv_read")
    return KvOutputs(k, v)


def gdn_kv_attention_workspace_size(B: int, T: int, Hq: int, H: int, D: int) -> int:
    """Bytes of device workspace gdn_kv_attention needs (0 for invalid sizes)."""
    return int(load().gdn_kv_attention_workspace_size(B, T, Hq, H, D))


_workspace_size = functools.lru_cache(maxsize=256)(gdn_kv_attention_workspace_size)  # a function of the sizes alone


def gdn_kv_attention(q, cache, block_table, lengths, *, new=None, scale: float | None = None, window: int = 0,
                     k_scale=None, v_scale=None, y=None, lse=None, return_lse: bool = False, workspace=None,
                     stream=None) -> AttentionOutputs:
    """Attention of the new tokens q [B,T,Hq,D] over the cache.

    ``lengths`` [B] int32 counts the tokens in the cache, the new ones among
    them; sequence b has ``new[b]`` new tokens (None: T), the last ones of its
    length, and nothing is written past them.  Token t sees the tokens up to its
    own, the last ``window`` of them if that is not 0.  ``scale`` defaults to
    1/sqrt(D).  ``lse`` [B,T,Hq] float32 (given, or with ``return_lse``) takes the
    log-sum-exp of the scores.  ``workspace`` (a device tensor of at least
    ``gdn_kv_attention_workspace_size(B, T, Hq, H, D)`` bytes) is allocated when
    not given."""
    dev = _device_of(q, "q")
    dt = q.dtype
    B, T, Hq, D = _shape(q, "q", 4, "[B,T,Hq,D]")
    pages, H, page, Dc = _cache(cache, dev)
    if Dc != D:
        raise ValueError(f"q has heads of {D} channels, the cache of {Dc}")
    width = _shape(block_table, "block_table", 2, "[B,width]")[1]
    sb, st = _strided(q, "q", (B, T, Hq, D), dt, dev)
    if y is None:
        y = _empty((B, T, Hq, D), dt, q.device, stream)
    if lse is None and return_lse:
        lse = _empty((B, T, Hq), torch.float32, q.device, stream)
    if workspace is None:
        need = _workspace_size(B, T, Hq, H, D)
        if need > 16:
            workspace = _empty(need, torch.uint8, q.device, stream)
    else:
        _need_workspace(workspace, q.device)
    i32, f32 = torch.int32, torch.float32
    status = _lib().gdn_kv_attention(
        q.data_ptr(), cache.data_ptr(), _dense(block_table, "block_table", (B, width), i32, dev),
        _dense(lengths, "lengths", (B,), i32, dev), _dense(new, "new", (B,), i32, dev),
        _dense(k_scale, "k_scale", (H,), f32, dev), _dense(v_scale, "v_scale", (H,), f32, dev),
        _dense(y, "y", (B, T, Hq, D), dt, dev), _dense(lse, "lse", (B, T, Hq), f32, dev), B, T, Hq, H, D, width, page,
        pages, sb, st, 1 / math.sqrt(D) if scale is None else scale, window,
        None if workspace is None else workspace.data_ptr(),
        0 if workspace is None else workspace.numel() * workspace.element_size(), DTYPE_CODES[dt], _stream(dev, stream))
    if status:
        _check(status, "gdn_kv_attention")
    return AttentionOutputs(y, lse)
