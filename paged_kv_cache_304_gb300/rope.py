"""Norm and rotation of queries and keys, alone or with the KV-cache write.

Argument marshalling only; the contract of each call stands in
``include/pkv.h``.
"""

from __future__ import annotations

import math
import struct

import torch

from . import _dense, _ints, _launch, _rows, _wrong
from .q4 import Q4Cache, _cache

HEAD_DIM = 128
# pkv_norm_rope: q_weight, k_weight, freqs, positions, position_axis_stride, eps, rope_dim, interleaved, num_axes,
# sections[3]
_PACK = struct.Struct("@4Pqf3i3i").pack


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


def _weight(t, name: str, dev: int) -> int:
    return 0 if t is None else _dense(t, name, (HEAD_DIM,), dev)


def _describe(n, dev, q_weight, k_weight, eps, freqs, positions, interleaved, sections) -> bytes:
    wq, wk = _weight(q_weight, "q_weight", dev), _weight(k_weight, "k_weight", dev)
    if freqs is None:
        return _PACK(wq, wk, 0, 0, 0, eps, 0, bool(interleaved), 1, 0, 0, 0)
    if (not isinstance(freqs, torch.Tensor) or freqs.dtype != torch.int64 or freqs.get_device() != dev
            or len(freqs.shape) != 1 or not freqs.is_contiguous()):
        _wrong(freqs, "freqs", torch.int64, dev, "contiguous [rope_dim / 2]")
    if not isinstance(positions, torch.Tensor) or positions.dtype != torch.int32 or positions.get_device() != dev:
        _wrong(positions, "positions", torch.int32, dev, "")
    half = freqs.shape[0]
    shape, stride = positions.shape, positions.stride()
    if len(shape) not in (1, 2) or shape[-1] != n or (n > 1 and stride[-1] != 1):
        raise ValueError("positions must be [N] or [axes, N] with contiguous rows")
    axes, step = (shape[0], stride[0]) if len(shape) == 2 else (1, 0)
    if sections is None:
        if axes != 1:
            raise ValueError("several position axes need sections")
        sections = (half,)
    if len(sections) != axes or axes > 3:
        raise ValueError("sections must have one entry per position axis (1 to 3)")
    return _PACK(wq, wk, freqs.data_ptr(), positions.data_ptr(), step if axes > 1 else 0, eps, 2 * half,
                 bool(interleaved), axes, *sections, *(0,) * (3 - axes))


def _like(t: torch.Tensor, out, name: str, dev: int, n: int, h: int):
    """An output of [n, h, 128]: (tensor, pointer, token stride)."""
    if out is None:
        out = torch.empty(t.shape, dtype=torch.bfloat16, device=t.device)
        return out, out.data_ptr(), h * HEAD_DIM
    p, _, _, stride = _rows(out, name, dev, n, h)
    return out, p, stride


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
    qp, n, hq, qs = _rows(q, "q")
    dev = q.get_device()
    kp, _, hkv, ks = _rows(k, "k", dev, n)
    q_out, qo, qos = _like(q, q_out, "q_out", dev, n, hq)
    k_out, ko, kos = _like(k, k_out, "k_out", dev, n, hkv)
    _launch("pkv_qk_norm_rope", dev, qp, qs, kp, ks, n, hq, hkv, HEAD_DIM,
            _describe(n, dev, q_weight, k_weight, eps, freqs, positions, interleaved, sections), qo, qos, ko, kos)
    return q_out, k_out


def qk_norm_rope_write(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, q_weight, k_weight, eps: float, freqs,
                       positions, slot_mapping: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                       interleaved: bool = False, sections=None, q_out: torch.Tensor | None = None) -> torch.Tensor:
    """qk_norm_rope, with its keys and v [N, Hkv, 128] written into the bf16 caches at slot_mapping; returns q_out."""
    qp, n, hq, qs = _rows(q, "q")
    dev = q.get_device()
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 4:
        _wrong(k_cache, "k_cache", torch.bfloat16, dev, "[num_blocks, block_size, num_kv_heads, 128]")
    shape = k_cache.shape
    nb, bs, hkv, d = shape
    kp, _, _, ks = _rows(k, "k", dev, n, hkv)
    vp, _, _, vs = _rows(v, "v", dev, n, hkv)
    q_out, qo, qos = _like(q, q_out, "q_out", dev, n, hq)
    _launch("pkv_qk_norm_rope_write", dev, qp, qs, kp, ks, vp, vs, n, hq,
            _describe(n, dev, q_weight, k_weight, eps, freqs, positions, interleaved, sections),
            _ints(slot_mapping, "slot_mapping", dev, n), _dense(k_cache, "k_cache", shape, dev),
            _dense(v_cache, "v_cache", shape, dev), nb, bs, hkv, d, qo, qos)
    return q_out


def qk_norm_rope_write_q4(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, q_weight, k_weight, eps: float, freqs,
                          positions, slot_mapping: torch.Tensor, cache: Q4Cache, interleaved: bool = False,
                          sections=None, q_out: torch.Tensor | None = None) -> torch.Tensor:
    """qk_norm_rope, with its keys and v quantised into the 4-bit cache at slot_mapping; returns q_out."""
    dev, hkv = _cache(cache)._index, cache.num_kv_heads
    qp, n, hq, qs = _rows(q, "q", dev)
    kp, _, _, ks = _rows(k, "k", dev, n, hkv)
    vp, _, _, vs = _rows(v, "v", dev, n, hkv)
    q_out, qo, qos = _like(q, q_out, "q_out", dev, n, hq)
    _launch("pkv_qk_norm_rope_write_q4", dev, qp, qs, kp, ks, vp, vs, n, hq,
            _describe(n, dev, q_weight, k_weight, eps, freqs, positions, interleaved, sections),
            _ints(slot_mapping, "slot_mapping", dev, n), cache._ref, qo, qos)
    return q_out
