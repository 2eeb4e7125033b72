"""Rotary positions and the 4-bit latent cache, numpy fp64.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``): it shares no code with
the CUDA path.

A pair (a, b) of a token at position p is turned by the angle p f:
    y_a = amplitude (x_a cos - x_b sin),  y_b = amplitude (x_b cos + x_a sin).
A 4-bit row is 256 bytes of e2m1 codes (two a byte, the even channel low), 64
bf16 shared channels and 32 e4m3 scales, one for 16 channels; a channel stands
for code * scale * 2^exponent.
"""
from __future__ import annotations

from typing import List, Tuple

import numpy as np

from .latent import LATENT, PE, ROW

ROW4 = LATENT // 2 + 2 * PE + LATENT // 16
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])                       # codes 0 .. 7; 8 .. 15 their negatives
CODE_VALUE = np.concatenate([E2M1, -E2M1])


def e4m3_values() -> np.ndarray:
    """What the 256 bytes of an e4m3 number stand for (NaN: 0x7f and 0xff)."""
    out = np.empty(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        v = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        out[b] = (-1 if b & 128 else 1) * (np.nan if e == 15 and m == 7 else v)
    return out


E4M3 = e4m3_values()


def nearest_even(x: np.ndarray, grid: np.ndarray) -> np.ndarray:
    """Index of the grid's number nearest to x >= 0, the even index at a border;
    past the last number: the last."""
    mid = (grid[1:] + grid[:-1]) / 2
    i = np.searchsorted(mid, x, side="left")                        # borders below x
    at_border = (i < len(mid)) & (x == mid[np.minimum(i, len(mid) - 1)])
    return np.where(at_border & (i % 2 == 1), i + 1, i)


def frequencies(d: int, base: float) -> np.ndarray:
    """Radians a position of each pair, in extended precision."""
    i = np.arange(d // 2, dtype=np.longdouble)
    return np.longdouble(base) ** (-2 * i / np.longdouble(d))


def rotate(x: np.ndarray, pos: np.ndarray, freq: np.ndarray, amplitude: float = 1.0, interleaved: bool = False,
           inverse: bool = False) -> np.ndarray:
    """x [T, ..., d] turned by the tokens' positions [T]."""
    x = np.asarray(x, dtype=np.float64)
    d = x.shape[-1]
    angle = np.asarray(pos, dtype=np.longdouble)[:, None] * np.asarray(freq, dtype=np.longdouble)
    two_pi = 2 * np.arctan2(np.longdouble(0), np.longdouble(-1))
    angle = (angle - two_pi * np.floor(angle / two_pi)).astype(np.float64)
    shape = (len(pos),) + (1,) * (x.ndim - 2) + (d // 2,)
    c, s = amplitude * np.cos(angle).reshape(shape), amplitude * np.sin(angle).reshape(shape)
    if inverse:
        s = -s
    a, b = (slice(0, None, 2), slice(1, None, 2)) if interleaved else (slice(0, d // 2), slice(d // 2, None))
    y = np.empty(x.shape)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def positions(seq_lens: List[int], cu: List[int]) -> np.ndarray:
    """Positions of the packed new tokens."""
    return np.concatenate([np.arange(cu[b + 1] - cu[b]) + seq_lens[b] - (cu[b + 1] - cu[b])
                           for b in range(len(seq_lens))]).astype(np.int64)


def quantise(c: np.ndarray, exponent: int = 0) -> Tuple[np.ndarray, np.ndarray]:
    """Latents [..., 512] (bf16 values) as (codes 0 .. 15, scale bytes), uint8."""
    g = np.asarray(c, dtype=np.float64).reshape(c.shape[:-1] + (LATENT // 16, 16)) * 2.0 ** -exponent
    top = np.abs(g).max(-1)
    nan = np.isnan(top)
    scale = nearest_even(np.where(nan, 0.0, top) / 6, E4M3[:127]).astype(np.uint8)
    s = E4M3[scale][..., None]
    with np.errstate(invalid="ignore", divide="ignore"):
        y = np.where(s > 0, np.abs(g) / s, 0.0)
    code = nearest_even(np.where(np.isnan(y), 0.0, y), E2M1) + 8 * np.signbit(g)
    return code.astype(np.uint8).reshape(c.shape), np.where(nan, 0x7F, scale).astype(np.uint8)


def values(codes: np.ndarray, scales: np.ndarray, exponent: int = 0) -> np.ndarray:
    """What codes [..., 512] with scale bytes [..., 32] stand for."""
    return CODE_VALUE[codes] * np.repeat(E4M3[scales], 16, axis=-1) * 2.0 ** exponent


def pack(codes: np.ndarray, pe_bits: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """Rows [..., 416] uint8; pe_bits [..., 64] uint16 (bf16)."""
    pair = codes.reshape(codes.shape[:-1] + (LATENT // 2, 2))
    pe = np.stack([pe_bits & 255, pe_bits >> 8], axis=-1).reshape(pe_bits.shape[:-1] + (2 * PE,))
    return np.concatenate([pair[..., 0] | pair[..., 1] << 4, pe.astype(np.uint8), scales], axis=-1)


def unpack(rows: np.ndarray, exponent: int = 0) -> np.ndarray:
    """What rows [..., 416] uint8 stand for, [..., 576]."""
    c, pe, sc = rows[..., :LATENT // 2], rows[..., LATENT // 2:-(LATENT // 16)], rows[..., -(LATENT // 16):]
    codes = np.stack([c & 15, c >> 4], axis=-1).reshape(rows.shape[:-1] + (LATENT,))
    bits = pe[..., 0::2].astype(np.uint32) | pe[..., 1::2].astype(np.uint32) << 8
    pe = (bits << 16).view(np.float32).astype(np.float64)
    return np.concatenate([values(codes, sc, exponent), pe], axis=-1)


assert ROW4 == 416 and ROW == 576
