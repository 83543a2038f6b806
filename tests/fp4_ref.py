"""Microscaled fp4 in float64 numpy, from the definition in include/ck.h: what the tests of the
fp4 operators compare with.  It shares no code with the library."""
from __future__ import annotations

import numpy as np
import torch

MX, NV = 0, 1
BLOCK = {MX: 32, NV: 16}
GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
                 for e in range(16) for m in range(8)][:127])


def nearest(q, table):
    """Index of the entry of an ascending table nearest to q >= 0, the even one at a tie."""
    q = np.asarray(q, dtype=np.float64)
    i = np.clip(np.searchsorted(table, q, side="right") - 1, 0, len(table) - 2)
    lo, hi = table[i], table[i + 1]
    mid = (lo + hi) / 2          # exact: neighbours of a few bits
    up = (q > mid) | ((q == mid) & (i % 2 == 1))
    return np.where(up, i + 1, i)


def to64(x: torch.Tensor) -> np.ndarray:
    return x.detach().to("cpu", torch.float64).numpy()


def quantize(x: torch.Tensor, fmt: int, t=None):
    """(codes (M, K) in 0..15, scale bytes (M, K / block)) of a 2-D tensor; t: fp32 or None."""
    v = to64(x)
    M, K = v.shape
    b = BLOCK[fmt]
    v = v.reshape(M, K // b, b)
    amax = np.abs(v).max(-1) if M else np.zeros((0, K // b))
    bad = ~np.isfinite(amax)
    a = np.where(bad, 1.0, amax)
    with np.errstate(all="ignore"):
        if fmt == MX:
            e = np.where(a == 0, -200, np.floor(np.log2(np.where(a == 0, 1.0, a))))
            # log2 may land on the neighbour of an exact power: settle it by comparison
            e = np.where((a > 0) & (np.exp2(e) > a), e - 1, e)
            e = np.where((a > 0) & (np.exp2(e + 1) <= a), e + 1, e)
            e = np.clip(e - 2, -127, 127)
            byte = (e + 127).astype(np.int64)
            unit = np.exp2(e)
            nan_byte = 0xFF
        else:
            t32 = np.float32(1.0 if t is None else t)
            if not (t32 > 0 and np.isfinite(t32)):
                bad = np.ones_like(bad)
                t32 = np.float32(1.0)
            c = np.float64(np.float32(6.0) * t32)
            byte = nearest(np.minimum(a / c, 1e6), E4M3)
            unit = (E4M3[byte].astype(np.float32) * t32).astype(np.float64)
            nan_byte = 0x7F
        av = np.where(bad[..., None], 0.0, np.abs(v))
        q = np.where(unit[..., None] == 0, 0.0, av / np.where(unit == 0, 1.0, unit)[..., None])
        code = nearest(np.minimum(q, 100.0), GRID) | (np.signbit(v).astype(np.int64) << 3)
    code = np.where((bad | (unit == 0))[..., None], 0, code)
    byte = np.where(bad, nan_byte, byte)
    return code.reshape(M, K).astype(np.uint8), byte.astype(np.uint8)


def pack(code: np.ndarray) -> np.ndarray:
    return (code[..., 0::2] | (code[..., 1::2] << 4)).astype(np.uint8)


def unpack(packed: np.ndarray) -> np.ndarray:
    return np.stack([packed & 15, packed >> 4], -1).reshape(*packed.shape[:-1], -1)


def code_values(code: np.ndarray) -> np.ndarray:
    return np.where(code & 8, -1.0, 1.0) * GRID[code & 7]


def scale_values(byte: np.ndarray, fmt: int) -> np.ndarray:
    byte = byte.astype(np.int64)
    if fmt == MX:
        return np.where(byte == 255, np.nan, np.exp2(byte - 127.0))
    v = np.append(E4M3, np.nan)[byte & 127]
    return np.where(byte & 128, -v, v)


def values(code: np.ndarray, byte: np.ndarray, fmt: int) -> np.ndarray:
    """Codes times their block scales, without the tensor scale."""
    return code_values(code) * np.repeat(scale_values(byte, fmt), BLOCK[fmt], axis=-1)


def tile_index(rows, blocks: int, first=0):
    """Byte positions (len(rows), blocks) of the scales of rows counted from tile row `first`."""
    r = np.asarray(rows)[:, None]
    c = np.arange(blocks)[None, :]
    kt = -(-blocks // 4)
    return ((first + r // 128) * kt + c // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + c % 4


def tile(byte: np.ndarray) -> np.ndarray:
    """Scale bytes (M, C) as tiles, zero past M and C."""
    M, C = byte.shape
    out = np.zeros(-(-M // 128) * -(-C // 4) * 512, np.uint8)
    out[tile_index(np.arange(M), C)] = byte
    return out


def untile(tiles: np.ndarray, M: int, C: int) -> np.ndarray:
    return tiles[tile_index(np.arange(M), C)]


def expert_scale_index(offsets, blocks: int):
    """For rows sorted by expert: (rows, byte positions (len(rows), blocks))."""
    rows, idx = [], []
    for e in range(len(offsets) - 1):
        n = offsets[e + 1] - offsets[e]
        if n > 0:
            rows.append(np.arange(offsets[e], offsets[e + 1]))
            idx.append(tile_index(np.arange(n), blocks, offsets[e] // 128 + e))
    if not rows:
        return np.zeros(0, np.int64), np.zeros((0, blocks), np.int64)
    return np.concatenate(rows), np.concatenate(idx)
