"""The 4-bit reference itself, pinned by hand-worked rows (CPU)."""

import numpy as np
import torch

from tests import q4_ref


def test_e4m3_table():
    t = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, q4_ref.E4M3)


def test_hand_worked_group():
    """amax 6 gives scale 1; every code, a tie (0.25 -> 0, 0.75 -> 1, 5 -> 4) and the packing order."""
    x = torch.zeros(1, 128)
    x[0, :16] = torch.tensor([6, -6, 4, 3, 2, 1.5, 1, 0.5, 0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    data, scales = q4_ref.quantise(q4_ref.bf16(x))
    assert scales[0, 0] == 0x38 and (scales[0, 1:] == 0).all()
    assert list(data[0, :8]) == [0x7 | 0xF << 4, 0x6 | 0x5 << 4, 0x4 | 0x3 << 4, 0x2 | 0x1 << 4, 0x0 | 0x0 << 4,
                                 0x2 | 0x2 << 4, 0x4 | 0x4 << 4, 0x6 | 0x6 << 4]
    assert list(q4_ref.values(data, scales)[0, 8:16]) == [0, 0, 1, 1, 2, 2, 4, 4]


def test_held_values_are_exact_in_half_precision():
    """Every code times every scale fits fp16 and bf16, which the kernels rely on."""
    prod = np.outer(q4_ref.CODES, q4_ref.E4M3)
    t = torch.from_numpy(prod)
    assert torch.equal(t.half().double(), t) and torch.equal(t.bfloat16().double(), t)


def test_special_values():
    x = torch.ones(3, 128)
    x[0, 3] = float("nan")
    x[1, 20] = float("-inf")
    x[2] = 1e-30
    v = q4_ref.values(*q4_ref.quantise(q4_ref.bf16(x)))
    # a group of ones: 1/6 lies between 10/64 and 11/64 and is nearer to 11/64, so 1 is held as 6 * 11/64
    assert np.isnan(v[0, :16]).all() and (v[0, 16:] == 66 / 64).all()
    assert v[1, 20] == -6 * 448 and (v[1, 16:20] == 0).all()
    assert (v[2] == 0).all()


def test_reference_attention_matches_torch():
    g = torch.Generator().manual_seed(0)
    q, k, v = (torch.randn(s, generator=g, dtype=torch.float64) for s in ((5, 4, 128), (9, 2, 128), (9, 2, 128)))
    out, _ = q4_ref.attention(q, k, v, 0.1, 5)
    mask = torch.arange(9)[None] < (5 + torch.arange(5))[:, None]
    ref = torch.nn.functional.scaled_dot_product_attention(
        q.transpose(0, 1), k.repeat_interleave(2, 1).transpose(0, 1), v.repeat_interleave(2, 1).transpose(0, 1),
        attn_mask=mask, scale=0.1).transpose(0, 1)
    assert np.abs(out - ref.numpy()).max() < 1e-12
