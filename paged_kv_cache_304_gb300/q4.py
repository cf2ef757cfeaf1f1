"""The 4-bit cache: storage, write, read-back and attention.

Argument marshalling only, like the package's other calls; the format and the
contract of each call stand in ``include/pkv.h``.
"""

from __future__ import annotations

import ctypes
import math

import torch

from . import _dev, _ints, _launch, _rows, _same_device, load

HEAD_DIM = 128
GROUP = 16


class _Struct(ctypes.Structure):
    _fields_ = [("k_data", ctypes.c_void_p), ("k_scales", ctypes.c_void_p), ("v_data", ctypes.c_void_p),
                ("v_scales", ctypes.c_void_p), ("k_scale", ctypes.c_float), ("v_scale", ctypes.c_float),
                ("num_blocks", ctypes.c_int32), ("block_size", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32)]


class Q4Cache:
    """One layer's K and V held in 4 bits.

    k_data, v_data: uint8 [num_blocks, block_size, num_kv_heads, 64], two codes
    to a byte; k_scales, v_scales: uint8 or float8_e4m3fn [num_blocks,
    block_size, num_kv_heads, 8], one scale per 16 dims; k_scale, v_scale: the
    tensor scales.  The tensors stay the caller's: slices of one allocation for
    all layers will do.  The object is a handle on them: it keeps them alive, and
    their storage must not be resized while it is in use.
    """

    def __init__(self, k_data: torch.Tensor, k_scales: torch.Tensor, v_data: torch.Tensor, v_scales: torch.Tensor,
                 k_scale: float = 1.0, v_scale: float = 1.0):
        for t, n in ((k_data, "k_data"), (v_data, "v_data")):
            _dev(t, n, torch.uint8)
        for t, n in ((k_scales, "k_scales"), (v_scales, "v_scales")):
            _dev(t, n)
            if t.dtype not in (torch.uint8, torch.float8_e4m3fn):
                raise TypeError(f"{n} must be torch.uint8 or torch.float8_e4m3fn, got {t.dtype}")
        if k_data.dim() != 4 or k_data.shape[3] != HEAD_DIM // 2:
            raise ValueError("k_data must be [num_blocks, block_size, num_kv_heads, 64]")
        nb, bs, hkv, _ = (int(x) for x in k_data.shape)
        for t, n, last in ((k_data, "k_data", HEAD_DIM // 2), (v_data, "v_data", HEAD_DIM // 2),
                           (k_scales, "k_scales", HEAD_DIM // GROUP), (v_scales, "v_scales", HEAD_DIM // GROUP)):
            if tuple(t.shape) != (nb, bs, hkv, last) or not t.is_contiguous():
                raise ValueError(f"{n} must be contiguous [{nb}, {bs}, {hkv}, {last}]")
        _same_device(k_data.device, k_scales=k_scales, v_data=v_data, v_scales=v_scales)
        self.k_data, self.k_scales, self.v_data, self.v_scales = k_data, k_scales, v_data, v_scales
        self.k_scale, self.v_scale = float(k_scale), float(v_scale)
        if not (self.k_scale > 0 and self.v_scale > 0 and math.isfinite(self.k_scale) and math.isfinite(self.v_scale)):
            raise ValueError("tensor scales must be finite and positive")
        self.num_blocks, self.block_size, self.num_kv_heads, self.device = nb, bs, hkv, k_data.device
        self._struct = _Struct(k_data.data_ptr(), k_scales.data_ptr(), v_data.data_ptr(), v_scales.data_ptr(),
                               self.k_scale, self.v_scale, nb, bs, hkv, HEAD_DIM)
        self._ref = ctypes.addressof(self._struct)

    @classmethod
    def empty(cls, num_blocks: int, num_kv_heads: int, device, k_scale: float = 1.0, v_scale: float = 1.0,
              block_size: int = 256) -> "Q4Cache":
        """A cache of zeros (every slot reads as zero)."""
        d = torch.zeros((2, num_blocks, block_size, num_kv_heads, HEAD_DIM // 2), dtype=torch.uint8, device=device)
        s = torch.zeros((2, num_blocks, block_size, num_kv_heads, HEAD_DIM // GROUP), dtype=torch.uint8,
                        device=device)
        return cls(d[0], s[0], d[1], s[1], k_scale, v_scale)


def _cache(c) -> Q4Cache:
    if not isinstance(c, Q4Cache):
        raise TypeError(f"cache must be a Q4Cache, got {type(c).__name__}")
    return c


def kv_cache_write_q4(k: torch.Tensor, v: torch.Tensor, slot_mapping: torch.Tensor, cache: Q4Cache) -> None:
    """Quantise k, v [N, Hkv, 128] (bf16, rows may be strided) into the cache at slot_mapping [N]; -1 is skipped."""
    dev = _cache(cache).device
    n, _, ks = _rows(k, "k", cache.num_kv_heads)
    nv, _, vs = _rows(v, "v", cache.num_kv_heads)
    _ints(dev, slot_mapping=slot_mapping)
    _same_device(dev, k=k, v=v)
    if nv != n or slot_mapping.shape != (n,):
        raise ValueError("k, v and slot_mapping must have the same number of tokens")
    _launch("pkv_kv_cache_write_q4", dev, k.data_ptr(), ks, v.data_ptr(), vs, slot_mapping.data_ptr(), n, cache._ref)


def kv_cache_read_q4(cache: Q4Cache, slots: torch.Tensor, k_out: torch.Tensor | None = None,
                     v_out: torch.Tensor | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """The rows that slots [N] (int32) hold, as bf16 k, v [N, Hkv, 128]; slot -1 gives zeros."""
    dev = _cache(cache).device
    _ints(dev, slots=slots)
    if slots.dim() != 1:
        raise ValueError("slots must be [N]")
    shape = (int(slots.shape[0]), cache.num_kv_heads, HEAD_DIM)
    k_out, v_out = _out(k_out, "k_out", shape, dev), _out(v_out, "v_out", shape, dev)
    _launch("pkv_kv_cache_read_q4", dev, cache._ref, slots.data_ptr(), shape[0], k_out.data_ptr(), v_out.data_ptr())
    return k_out, v_out


def _out(t, name, shape, dev):
    if t is None:
        return torch.empty(shape, dtype=torch.bfloat16, device=dev)
    _dev(t, name, torch.bfloat16)
    if tuple(t.shape) != tuple(shape) or not t.is_contiguous() or t.device != dev:
        raise ValueError(f"{name} must be a contiguous bf16 tensor of shape {tuple(shape)} on {dev}")
    return t


def _workspace(n: int, device) -> torch.Tensor:
    return torch.empty(max(256, n), dtype=torch.uint8, device=device)


def _workspace_arg(t: torch.Tensor, dev):
    _dev(t, "workspace")
    if not t.is_contiguous() or t.device != dev:
        raise ValueError(f"workspace must be a contiguous tensor on {dev}")
    return t.data_ptr(), t.numel() * t.element_size()


def decode_q4_workspace(batch: int, num_q_heads: int, num_kv_heads: int, device) -> torch.Tensor:
    """A workspace for paged_attn_decode_q4 (uninitialised; one per call that may run at the same time)."""
    with torch.cuda.device(device):
        n = int(load().pkv_decode_q4_workspace_bytes(batch, num_q_heads, num_kv_heads))
    return _workspace(n, device)


def paged_attn_decode_q4(q: torch.Tensor, cache: Q4Cache, context_lens: torch.Tensor, block_tables: torch.Tensor,
                         scale: float, out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                         max_context_len: int | None = None) -> torch.Tensor:
    """Decode attention over the 4-bit cache; arguments as in paged_attn_decode."""
    dev = _cache(cache).device
    _dev(q, "q", torch.bfloat16)
    _same_device(dev, q=q)
    _ints(dev, context_lens=context_lens, block_tables=block_tables)
    if q.dim() != 3 or q.shape[2] != HEAD_DIM or not q.is_contiguous():
        raise ValueError("q must be contiguous [B, Hq, 128]")
    b, hq = int(q.shape[0]), int(q.shape[1])
    if block_tables.dim() != 2 or block_tables.shape[0] != b or context_lens.shape != (b,):
        raise ValueError("block_tables must be [B, max_blocks] and context_lens [B]")
    out = _out(out, "out", q.shape, dev)
    if workspace is None:
        workspace = decode_q4_workspace(b, hq, cache.num_kv_heads, dev)
    wp, wb = _workspace_arg(workspace, dev)
    maxb = int(block_tables.shape[1])
    if max_context_len is None:
        max_context_len = maxb * cache.block_size
    _launch("pkv_paged_attn_decode_q4", dev, q.data_ptr(), cache._ref, context_lens.data_ptr(),
            block_tables.data_ptr(), maxb, b, hq, int(max_context_len), float(scale), out.data_ptr(), wp, wb)
    return out


def prefill_q4_workspace(total_q: int, num_seqs: int, max_seqlen_q: int, max_seqlen_k: int, num_q_heads: int,
                         num_kv_heads: int, device) -> torch.Tensor:
    """A workspace for paged_attn_prefill_q4 of these sizes (uninitialised)."""
    with torch.cuda.device(device):
        n = int(load().pkv_prefill_q4_workspace_bytes(total_q, num_seqs, max_seqlen_q, max_seqlen_k, num_q_heads,
                                                      num_kv_heads))
    return _workspace(n, device)


def paged_attn_prefill_q4(q: torch.Tensor, cache: Q4Cache, cu_seqlens_q: torch.Tensor, cu_seqlens_k: torch.Tensor,
                          block_tables: torch.Tensor, scale: float, max_seqlen_q: int, max_seqlen_k: int,
                          out: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Varlen causal prefill attention over the 4-bit cache; arguments as in paged_attn_prefill."""
    dev = _cache(cache).device
    _dev(q, "q", torch.bfloat16)
    _same_device(dev, q=q)
    _ints(dev, cu_seqlens_q=cu_seqlens_q, cu_seqlens_k=cu_seqlens_k, block_tables=block_tables)
    if q.dim() != 3 or q.shape[2] != HEAD_DIM or not q.is_contiguous():
        raise ValueError("q must be contiguous [T, Hq, 128]")
    total, hq = int(q.shape[0]), int(q.shape[1])
    s = int(cu_seqlens_q.numel()) - 1
    if (s < 0 or cu_seqlens_q.dim() != 1 or cu_seqlens_k.shape != (s + 1,) or block_tables.dim() != 2
            or block_tables.shape[0] != s):
        raise ValueError("cu_seqlens_q and cu_seqlens_k must be [S+1] and block_tables [S, max_blocks]")
    out = _out(out, "out", q.shape, dev)
    if workspace is None:
        workspace = prefill_q4_workspace(total, s, int(max_seqlen_q), int(max_seqlen_k), hq, cache.num_kv_heads, dev)
    wp, wb = _workspace_arg(workspace, dev)
    _launch("pkv_paged_attn_prefill_q4", dev, q.data_ptr(), cache._ref, cu_seqlens_q.data_ptr(),
            cu_seqlens_k.data_ptr(), block_tables.data_ptr(), int(block_tables.shape[1]), s, total, int(max_seqlen_q),
            int(max_seqlen_k), hq, float(scale), out.data_ptr(), wp, wb)
    return out
