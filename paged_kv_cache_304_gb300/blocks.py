"""Forking, freeing, compacting and copying the blocks of a cache.

Argument marshalling only; the contract of each call stands in
``include/pkv.h``.  A pool's bookkeeping is a block table and a length per
sequence and ref_count [num_blocks] (int32, 0 = free).
"""

from __future__ import annotations

import math

import torch

from . import _dev, _ints, _launch


def _pool(block_tables, context_lens, ref_count):
    _dev(ref_count, "ref_count", torch.int32)
    dev = ref_count.device
    _ints(dev, block_tables=block_tables, context_lens=context_lens, ref_count=ref_count)
    if block_tables.dim() != 2 or context_lens.shape != (block_tables.shape[0],) or ref_count.dim() != 1:
        raise ValueError("block_tables must be [S, max_blocks], context_lens [S] and ref_count [num_blocks]")
    return dev, int(block_tables.shape[0]), int(block_tables.shape[1]), int(ref_count.shape[0])


def _outputs(out, names, shapes, dev):
    if out is None:
        return tuple(torch.empty(s, dtype=torch.int32, device=dev) for s in shapes)
    if len(out) != len(names):
        raise ValueError(f"out must hold {', '.join(names)}")
    for t, n, s in zip(out, names, shapes):
        _ints(dev, **{n: t})
        if tuple(t.shape) != s:
            raise ValueError(f"{n} must be of shape {s}")
    return tuple(out)


def fork_blocks(block_tables: torch.Tensor, context_lens: torch.Tensor, parents: torch.Tensor,
                ref_count: torch.Tensor, out=None):
    """Children of sequences parents [n]: (child_tables, child_lens, copy_src, copy_dst), all int32.

    Full blocks are shared (ref_count rises); a partly filled last block gets a
    free one of its own and a pair of copy_src, copy_dst for copy_blocks.  `out`
    may hold the four tensors to write into.
    """
    dev, s, maxb, nb = _pool(block_tables, context_lens, ref_count)
    _ints(dev, parents=parents)
    if parents.dim() != 1:
        raise ValueError("parents must be [n]")
    n = int(parents.shape[0])
    out = _outputs(out, ("child_tables", "child_lens", "copy_src", "copy_dst"), ((n, maxb), (n,), (n,), (n,)), dev)
    _launch("pkv_fork_blocks", dev, block_tables.data_ptr(), context_lens.data_ptr(), s, maxb, parents.data_ptr(), n,
            ref_count.data_ptr(), nb, *(t.data_ptr() for t in out))
    return out


def free_blocks(block_tables: torch.Tensor, context_lens: torch.Tensor, ref_count: torch.Tensor) -> None:
    """Give back the blocks of every row: each loses one reference in ref_count."""
    dev, s, maxb, nb = _pool(block_tables, context_lens, ref_count)
    _launch("pkv_free_blocks", dev, block_tables.data_ptr(), context_lens.data_ptr(), s, maxb, ref_count.data_ptr(), nb)


def compact_blocks(block_tables: torch.Tensor, context_lens: torch.Tensor, ref_count: torch.Tensor, out=None):
    """Plan the moves that make the live blocks 0 .. n-1.

    Returns (new_tables, new_ref_count, copy_src, copy_dst, num_moves); hand
    copy_src and copy_dst [num_blocks // 2] (-1 behind the moves) to
    copy_blocks.  `out` may hold the five tensors to write into, the first two
    being block_tables and ref_count themselves if wanted.
    """
    dev, s, maxb, nb = _pool(block_tables, context_lens, ref_count)
    out = _outputs(out, ("new_tables", "new_ref_count", "copy_src", "copy_dst", "num_moves"),
                   ((s, maxb), (nb,), (nb // 2,), (nb // 2,), (1,)), dev)
    _launch("pkv_compact_blocks", dev, block_tables.data_ptr(), context_lens.data_ptr(), s, maxb,
            ref_count.data_ptr(), nb, *(t.data_ptr() for t in out))
    return out


def copy_blocks(cache: torch.Tensor, src: torch.Tensor, dst: torch.Tensor, block_dim: int = 0) -> None:
    """Copy blocks src[i] -> dst[i] in a cache of any type.

    cache: contiguous, its dim `block_dim` counting blocks; the dims before it
    (K/V, layers) are planes that are all copied, the dims behind it are a
    block's contents.  src, dst: int32 [n]; pairs of -1 are skipped.
    """
    _dev(cache, "cache")
    dev = cache.device
    _ints(dev, src=src, dst=dst)
    if not cache.is_contiguous() or not 0 <= block_dim < cache.dim():
        raise ValueError("cache must be contiguous with block_dim one of its dims")
    if src.dim() != 1 or dst.shape != src.shape:
        raise ValueError("src and dst must be [n]")
    shape = tuple(int(x) for x in cache.shape)
    planes, nb = math.prod(shape[:block_dim]), shape[block_dim]
    size = math.prod(shape[block_dim + 1:]) * cache.element_size()
    _launch("pkv_copy_blocks", dev, cache.data_ptr(), planes, nb * size, nb, size, src.data_ptr(), dst.data_ptr(),
            int(src.shape[0]))
