"""Forking, freeing, compacting and copying the blocks of a cache.

Argument marshalling only; the contract of each call stands in
``include/pkv.h``.  A pool's bookkeeping is a block table and a length per
sequence and ref_count [num_blocks] (int32, 0 = free).
"""

from __future__ import annotations

import math

import torch

from . import _dev, _ints, _launch, _table


def _pool(block_tables, context_lens, ref_count):
    """(device, S, max_blocks, num_blocks, pointers of the three)."""
    _dev(ref_count, "ref_count", torch.int32)
    dev = ref_count.get_device()
    rp = _ints(ref_count, "ref_count", dev)
    tp = _table(block_tables, "block_tables", dev)
    s, maxb = block_tables.shape
    return dev, s, maxb, ref_count.shape[0], tp, _ints(context_lens, "context_lens", dev, s), rp


def _outputs(out, names, shapes, device, dev):
    if out is None:
        out = tuple(torch.empty(s, dtype=torch.int32, device=device) for s in shapes)
    elif len(out) != len(names):
        raise ValueError(f"out must hold {', '.join(names)}")
    return tuple(out), [(_ints if len(s) == 1 else _table)(t, n, dev, *s) for t, n, s in zip(out, names, shapes)]


def fork_blocks(block_tables: torch.Tensor, context_lens: torch.Tensor, parents: torch.Tensor,
                ref_count: torch.Tensor, out=None):
    """Children of sequences parents [n]: (child_tables, child_lens, copy_src, copy_dst), all int32.

    Full blocks are shared (ref_count rises); a partly filled last block gets a
    free one of its own and a pair of copy_src, copy_dst for copy_blocks.  `out`
    may hold the four tensors to write into.
    """
    dev, s, maxb, nb, tp, lp, rp = _pool(block_tables, context_lens, ref_count)
    pp = _ints(parents, "parents", dev)
    n = parents.shape[0]
    out, ptrs = _outputs(out, ("child_tables", "child_lens", "copy_src", "copy_dst"), ((n, maxb), (n,), (n,), (n,)),
                         ref_count.device, dev)
    _launch("pkv_fork_blocks", dev, tp, lp, s, maxb, pp, n, rp, nb, *ptrs)
    return out


def free_blocks(block_tables: torch.Tensor, context_lens: torch.Tensor, ref_count: torch.Tensor) -> None:
    """Give back the blocks of every row: each loses one reference in ref_count."""
    dev, s, maxb, nb, tp, lp, rp = _pool(block_tables, context_lens, ref_count)
    _launch("pkv_free_blocks", dev, tp, lp, s, maxb, rp, nb)


def compact_blocks(block_tables: torch.Tensor, context_lens: torch.Tensor, ref_count: torch.Tensor, out=None):
    """Plan the moves that make the live blocks 0 .. n-1.

    Returns (new_tables, new_ref_count, copy_src, copy_dst, num_moves); hand
    copy_src and copy_dst [num_blocks // 2] (-1 behind the moves) to
    copy_blocks.  `out` may hold the five tensors to write into, the first two
    being block_tables and ref_count themselves if wanted.
    """
    dev, s, maxb, nb, tp, lp, rp = _pool(block_tables, context_lens, ref_count)
    out, ptrs = _outputs(out, ("new_tables", "new_ref_count", "copy_src", "copy_dst", "num_moves"),
                         ((s, maxb), (nb,), (nb // 2,), (nb // 2,), (1,)), ref_count.device, dev)
    _launch("pkv_compact_blocks", dev, tp, lp, s, maxb, rp, nb, *ptrs)
    return out


def copy_blocks(cache: torch.Tensor, src: torch.Tensor, dst: torch.Tensor, block_dim: int = 0) -> None:
    """Copy blocks src[i] -> dst[i] in a cache of any type.

    cache: contiguous, its dim `block_dim` counting blocks; the dims before it
    (K/V, layers) are planes that are all copied, the dims behind it are a
    block's contents.  src, dst: int32 [n]; pairs of -1 are skipped.
    """
    _dev(cache, "cache")
    dev, shape = cache.get_device(), cache.shape
    if not cache.is_contiguous() or not 0 <= block_dim < len(shape):
        raise ValueError("cache must be contiguous with block_dim one of its dims")
    sp = _ints(src, "src", dev)
    n = src.shape[0]
    planes, nb = math.prod(shape[:block_dim]), shape[block_dim]
    size = math.prod(shape[block_dim + 1:]) * cache.element_size()
    _launch("pkv_copy_blocks", dev, cache.data_ptr(), planes, nb * size, nb, size, sp, _ints(dst, "dst", dev, n), n)
