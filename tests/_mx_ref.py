"""Plain references of the norm, the MX quantizations and the grouped products:
numpy, in 64 bits except where the definition itself rounds to 32."""
import numpy as np
import torch

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def to_bf16(v: np.ndarray) -> np.ndarray:
    """float32 values rounded to bf16, as float32."""
    return torch.from_numpy(np.ascontiguousarray(v, dtype=np.float32)).to(torch.bfloat16).float().numpy()


def block_exponents(v: np.ndarray, top: int) -> np.ndarray:
    """E8M0 bytes of the 32-element blocks of v [R, C] (float32): 255 for a
    block with a NaN or an infinity, 0 for a zero block."""
    m = np.abs(v).reshape(v.shape[0], -1, 32).max(-1)              # NaN propagates
    _, e = np.frexp(np.where(np.isfinite(m) & (m > 0), m, 1.0).astype(np.float64))
    byte = np.clip(e - 1 - top, -127, 127) + 127
    byte = np.where(m == 0, 0, byte)
    return np.where(np.isfinite(m), byte, 255).astype(np.uint8)


def mxfp4(v: np.ndarray):
    """Row-major codes [R, C/2] and scales [R, C/32] of float32 v [R, C]: each
    magnitude to the nearest grid value, ties to the even code."""
    byte = block_exponents(v, 2)
    with np.errstate(invalid="ignore", over="ignore"):
        a = v.astype(np.float64) * np.exp2(127.0 - np.repeat(byte, 32, 1).astype(np.float64))
    mag = np.abs(a)
    code = np.zeros(v.shape, np.uint8)
    for c in range(7):
        mid = (GRID[c] + GRID[c + 1]) / 2
        code += (mag >= mid) if c % 2 else (mag > mid)
    code |= (np.signbit(v).astype(np.uint8) << 3)
    code[np.repeat(byte, 32, 1) == 255] = 0
    return code[:, 0::2] | (code[:, 1::2] << 4), byte


def e4m3_table() -> np.ndarray:
    """The 127 non-negative finite E4M3 values, in code order."""
    c = np.arange(127)
    e, m = c >> 3, c & 7
    return np.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * np.exp2(e - 7.0))


def mxfp8(v: np.ndarray):
    """Row-major E4M3 codes [R, C] and scales [R, C/32] of float32 v [R, C]."""
    byte = block_exponents(v, 8)
    with np.errstate(invalid="ignore", over="ignore"):
        a = np.abs(v.astype(np.float64) * np.exp2(127.0 - np.repeat(byte, 32, 1).astype(np.float64)))
    tab = e4m3_table()
    a = np.nan_to_num(np.minimum(a, 448.0))
    hi = np.clip(np.searchsorted(tab, a), 1, 126)
    lo = hi - 1
    dl, dh = a - tab[lo], tab[hi] - a
    code = np.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo).astype(np.uint8)
    code |= np.signbit(v).astype(np.uint8) << 7
    code[np.repeat(byte, 32, 1) == 255] = 0
    return code, byte


def mxfp4_values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """float64 values of row-major MXFP4 codes and scales."""
    c = np.stack((codes & 15, codes >> 4), -1).reshape(codes.shape[0], -1)
    s = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127))
    return np.where(c & 8, -1.0, 1.0) * GRID[c & 7] * np.repeat(s, 32, 1)


def mxfp8_values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    s = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127))
    tab = np.append(e4m3_table(), np.nan)
    return np.where(codes & 128, -1.0, 1.0) * tab[codes & 127] * np.repeat(s, 32, 1)


def rmsnorm(x: np.ndarray, r, w: np.ndarray, eps: float):
    """(h, rstd, y) of float32-held bf16 inputs, each rounded as defined."""
    h = x if r is None else to_bf16(x + r)
    with np.errstate(all="ignore"):
        mean = (h.astype(np.float64) ** 2).sum(1) / h.shape[1]
        rstd = (1.0 / np.sqrt(mean + eps)).astype(np.float32)
        y = (h * rstd[:, None]).astype(np.float32) * w.astype(np.float32)
    return h, rstd, y.astype(np.float32)
