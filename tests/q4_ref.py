"""Reference of the 4-bit format and of attention over it, in 64 bits (numpy and
torch on the CPU); shares no code with the library."""

from __future__ import annotations

import numpy as np
import torch

CODES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# the 127 finite e4m3 magnitudes by byte
E4M3 = np.array([(b & 7) / 8 * 2.0**-6 if b >> 3 == 0 else (1 + (b & 7) / 8) * 2.0 ** ((b >> 3) - 7)
                 for b in range(127)])


def bf16(x) -> torch.Tensor:
    return torch.as_tensor(x).to(torch.bfloat16)


def _nearest(values, x):
    """Index of the value nearest to x >= 0, ties to the even index."""
    hi = np.clip(np.searchsorted(values, x), 1, len(values) - 1)
    lo = hi - 1
    dl, dh = x - values[lo], values[hi] - x
    pick_hi = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    return np.where(pick_hi, hi, lo)


def quantise(x: torch.Tensor, ts: float = 1.0):
    """Rows [..., 128] (bf16) to (codes uint8 [..., 64], scale bytes [..., 8])."""
    y = (x.float().numpy() * (np.float32(1.0) / np.float32(ts))).astype(np.float32)
    y = y.reshape(*x.shape[:-1], 8, 16)
    with np.errstate(all="ignore"):
        amax = np.abs(y).max(-1, keepdims=True)  # a NaN stays
        q = np.minimum(amax / np.float32(6.0), np.float32(448.0)).astype(np.float64)
        sb = np.where(np.isnan(q), 127, _nearest(E4M3, np.nan_to_num(q)))
        s = np.where(sb == 127, np.nan, E4M3[np.minimum(sb, 126)])
        z = np.abs(y.astype(np.float64)) / np.where(s > 0, s, 1.0)
        code = _nearest(CODES, np.minimum(np.nan_to_num(z, nan=6.0, posinf=6.0), 6.0))
    code = np.where(s > 0, code | np.where(np.signbit(y), 8, 0), 0)
    code = np.where(np.isnan(s), 7, code).astype(np.uint8).reshape(*x.shape[:-1], 128)
    return code[..., 0::2] | (code[..., 1::2] << 4), sb.astype(np.uint8)[..., 0]


def values(data, scales, ts: float = 1.0) -> np.ndarray:
    """What packed codes and scale bytes stand for, in 64 bits."""
    data, scales = np.asarray(data), np.asarray(scales)
    n = np.stack((data & 15, data >> 4), -1).reshape(*data.shape[:-1], 128).astype(int)
    x = CODES[n & 7] * np.where(n & 8, -1.0, 1.0)
    mag = np.where((scales & 127) == 127, np.nan, E4M3[np.minimum(scales & 127, 126)])
    return x * np.repeat(np.where(scales & 128, -mag, mag), 16, -1) * np.float64(np.float32(ts))


def attention(q, k, v, scale, first_visible_end):
    """Rows q [n, Hq, 128] against k, v [L, Hkv, 128] (64 bits); row j sees keys
    0 .. first_visible_end + j - 1.  Returns (out, allowance) of shape [n, Hq, 128]:
    allowance bounds |error| of an fp32-accumulated result whose probabilities
    are rounded to fp16 and whose output is rounded to bf16.

    With A = sum p|v| / sum p the parts are: the output's rounding 2^-8 |o|; a
    probability's 2^-11 p, in the product only, so 2^-11 A; a score's error e
    (accumulation of 128 products, 2^-17 sum|q k| with room for the order of
    the sums, times scale, and 2^-21 of the exponent for ex2) changes p by a
    factor exp(+-e) above and below the fraction, 2 e A; sums over L keys in
    fp32 2^-18 A; probabilities below the fp16 range lose at most 2^-25 of the
    largest, L 2^-25 max|v|.
    """
    n, hq, _ = q.shape
    L, hkv, _ = k.shape
    q, k, v = (torch.as_tensor(x).double() for x in (q, k, v))
    out = torch.zeros((n, hq, 128), dtype=torch.float64)
    tol = torch.zeros_like(out)
    keys = torch.arange(L)
    for h in range(hq):
        kh, vh = k[:, h // (hq // hkv)], v[:, h // (hq // hkv)]
        x = q[:, h] @ kh.T * scale
        hidden = keys[None] >= (first_visible_end + torch.arange(n))[:, None]
        x = x.masked_fill(hidden, -torch.inf)
        p = torch.softmax(x, -1)
        o, a = p @ vh, p @ vh.abs()
        e = (q[:, h].abs() @ kh.abs().T * scale * 2.0**-17).masked_fill(hidden, 0).amax(-1, keepdim=True)
        span = (x.amax(-1, keepdim=True) - x.masked_fill(hidden, torch.inf).amin(-1, keepdim=True)).clamp(min=1)
        e = e + span * 2.0**-21
        out[:, h] = o
        tol[:, h] = 2.0**-8 * o.abs() + (2.0**-11 + 2 * e + 2.0**-18) * a + L * 2.0**-25 * vh.abs().max()
    return out.numpy(), tol.numpy()


def check(got: torch.Tensor, ref: np.ndarray, tol: np.ndarray, what: str):
    g = got.double().cpu().numpy()
    assert np.isfinite(g).all(), f"{what}: non-finite output"
    over = np.abs(g - ref) - tol
    assert (over <= 0).all(), (f"{what}: {int((over > 0).sum())} of {over.size} outside, worst by {over.max():.3g} "
                               f"at {np.unravel_index(over.argmax(), over.shape)}")
