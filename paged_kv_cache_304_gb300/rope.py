"""Norm and rotation of queries and keys, alone or with the KV-cache write.

Argument marshalling only; the contract of each call stands in
``include/pkv.h``.
"""

from __future__ import annotations

import ctypes
import math

import torch

from . import _cache_dims, _dev, _ints, _launch, _rows, _same_device
from .q4 import Q4Cache, _cache

HEAD_DIM = 128


class _Struct(ctypes.Structure):
    _fields_ = [("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p), ("freqs", ctypes.c_void_p),
                ("positions", ctypes.c_void_p), ("position_axis_stride", ctypes.c_int64), ("eps", ctypes.c_float),
                ("rope_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("num_axes", ctypes.c_int32),
                ("sections", ctypes.c_int32 * 3)]


def rope_frequencies(rope_dim: int, base: float = 10000.0, device="cuda", inv_freq=None) -> torch.Tensor:
    """The `freqs` of the calls below: int64 [rope_dim/2], rotation per position in 2^-64 turns.

    inv_freq: rotation per position in radians of every pair (a sequence or
    tensor of rope_dim/2 numbers) for scaled variants; default
    base^(-2i/rope_dim).  Computed once per model, in 64 bits on the host.
    """
    if rope_dim < 0 or rope_dim % 2:
        raise ValueError("rope_dim must be even and not negative")
    if inv_freq is None:
        inv_freq = [float(base) ** (-2.0 * i / rope_dim) for i in range(rope_dim // 2)]
    elif isinstance(inv_freq, torch.Tensor):
        inv_freq = inv_freq.detach().double().cpu().tolist()
    if len(inv_freq) != rope_dim // 2:
        raise ValueError("inv_freq must have rope_dim / 2 entries")
    turns = []
    for f in inv_freq:
        if not math.isfinite(f):
            raise ValueError("inv_freq must be finite")
        t = round(math.fmod(f / (2 * math.pi), 1.0) * 2.0**64) % 2**64
        turns.append(t - 2**64 if t >= 2**63 else t)
    return torch.tensor(turns, dtype=torch.int64, device=device)


def _describe(n, dev, q_weight, k_weight, eps, freqs, positions, interleaved, sections) -> _Struct:
    for t, name in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        if t is not None:
            _dev(t, name, torch.bfloat16)
            if t.shape != (HEAD_DIM,) or not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous [{HEAD_DIM}]")
    if freqs is None:
        rot, axes, stride, sections = 0, 1, 0, (0,)
    else:
        _dev(freqs, "freqs", torch.int64)
        _dev(positions, "positions", torch.int32)
        if freqs.dim() != 1 or not freqs.is_contiguous():
            raise ValueError("freqs must be contiguous [rope_dim / 2]")
        rot = 2 * int(freqs.shape[0])
        if positions.dim() not in (1, 2) or positions.shape[-1] != n or (n > 1 and positions.stride(-1) != 1):
            raise ValueError("positions must be [N] or [axes, N] with contiguous rows")
        axes = int(positions.shape[0]) if positions.dim() == 2 else 1
        stride = positions.stride(0) if positions.dim() == 2 and axes > 1 else 0
        if sections is None:
            if axes != 1:
                raise ValueError("several position axes need sections")
            sections = (rot // 2,)
        if len(sections) != axes or axes > 3:
            raise ValueError("sections must have one entry per position axis (1 to 3)")
    _same_device(dev, q_weight=q_weight, k_weight=k_weight, freqs=freqs, positions=positions if freqs is not None else None)
    ptr = [0 if t is None else t.data_ptr() for t in (q_weight, k_weight, freqs, positions if rot else None)]
    return _Struct(*ptr, stride, float(eps), rot, int(bool(interleaved)), axes, (ctypes.c_int32 * 3)(*sections))


def _q_out(q, t):
    if t is None:
        t = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
    n, h, stride = _rows(t, "output", int(q.shape[1]))
    if n != q.shape[0] or t.device != q.device:
        raise ValueError("an output must be shaped like its input, on the same device")
    return t, stride


def qk_norm_rope(q: torch.Tensor, k: torch.Tensor, q_weight, k_weight, eps: float, freqs, positions,
                 interleaved: bool = False, sections=None, q_out: torch.Tensor | None = None,
                 k_out: torch.Tensor | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """RMS norm per head and rotation of q [N, Hq, 128] and k [N, Hkv, 128] (bf16, rows may be strided).

    q_weight, k_weight: [128] bf16, or None to leave those rows unnormalised.
    freqs: from rope_frequencies(), or None for no rotation.  positions: [N]
    int32, or [axes, N] with sections (pairs per axis).  interleaved: rotate
    pairs (2i, 2i + 1) instead of (i, i + rope_dim/2).  q_out, k_out may be q
    and k themselves.
    """
    n, hq, qs = _rows(q, "q")
    nk, hkv, ks = _rows(k, "k")
    if nk != n:
        raise ValueError("q and k must have the same number of tokens")
    _same_device(q.device, k=k)
    q_out, qos = _q_out(q, q_out)
    k_out, kos = _q_out(k, k_out)
    nr = _describe(n, q.device, q_weight, k_weight, eps, freqs, positions, interleaved, sections)
    _launch("pkv_qk_norm_rope", q.device, q.data_ptr(), qs, k.data_ptr(), ks, n, hq, hkv, HEAD_DIM,
            ctypes.addressof(nr), q_out.data_ptr(), qos, k_out.data_ptr(), kos)
    return q_out, k_out


def qk_norm_rope_write(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, q_weight, k_weight, eps: float, freqs,
                       positions, slot_mapping: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                       interleaved: bool = False, sections=None, q_out: torch.Tensor | None = None) -> torch.Tensor:
    """qk_norm_rope, with its keys and v [N, Hkv, 128] written into the bf16 caches at slot_mapping; returns q_out."""
    for t, name in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        _dev(t, name, torch.bfloat16)
    nb, bs, hkv, d = _cache_dims(k_cache)
    if v_cache.shape != k_cache.shape or not v_cache.is_contiguous():
        raise ValueError("v_cache must match k_cache")
    n, hq, qs, ks, vs = _qkv(q, k, v, slot_mapping, hkv)
    _same_device(q.device, k_cache=k_cache, v_cache=v_cache)
    q_out, qos = _q_out(q, q_out)
    nr = _describe(n, q.device, q_weight, k_weight, eps, freqs, positions, interleaved, sections)
    _launch("pkv_qk_norm_rope_write", q.device, q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs, n, hq,
            ctypes.addressof(nr), slot_mapping.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), nb, bs, hkv, d,
            q_out.data_ptr(), qos)
    return q_out


def qk_norm_rope_write_q4(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, q_weight, k_weight, eps: float, freqs,
                          positions, slot_mapping: torch.Tensor, cache: Q4Cache, interleaved: bool = False,
                          sections=None, q_out: torch.Tensor | None = None) -> torch.Tensor:
    """qk_norm_rope, with its keys and v quantised into the 4-bit cache at slot_mapping; returns q_out."""
    n, hq, qs, ks, vs = _qkv(q, k, v, slot_mapping, _cache(cache).num_kv_heads)
    if cache.device != q.device:
        raise ValueError(f"cache is on {cache.device}, expected {q.device}")
    q_out, qos = _q_out(q, q_out)
    nr = _describe(n, q.device, q_weight, k_weight, eps, freqs, positions, interleaved, sections)
    _launch("pkv_qk_norm_rope_write_q4", q.device, q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs, n, hq,
            ctypes.addressof(nr), slot_mapping.data_ptr(), cache._ref, q_out.data_ptr(), qos)
    return q_out


def _qkv(q, k, v, slot_mapping, hkv):
    n, hq, qs = _rows(q, "q")
    nk, _, ks = _rows(k, "k", hkv)
    nv, _, vs = _rows(v, "v", hkv)
    _ints(q.device, slot_mapping=slot_mapping)
    _same_device(q.device, k=k, v=v)
    if nk != n or nv != n or slot_mapping.shape != (n,):
        raise ValueError("q, k, v and slot_mapping must have the same number of tokens")
    return n, hq, qs, ks, vs
