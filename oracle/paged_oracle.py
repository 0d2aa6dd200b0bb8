"""The paged latent cache and its attention in numpy, 64 bits, from their definitions.

Shares no code with the CUDA path.  Row formats: "f16" rows are 576 fp16 values (latent 0..511, RoPE key 512..575);
"e4m3" rows are 656 bytes (512 codes, 64 fp16 RoPE values, 16 scale bytes: value = code * 2^(s - 127))."""
from __future__ import annotations

import numpy as np

LAT, ROPE, ROW, ROW8 = 512, 64, 576, 656


def e4m3_values() -> np.ndarray:
    """The 256 values of the e4m3 codes (sign, 4 exponent bits with bias 7, 3 mantissa bits; 0x7F is NaN)."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0)) * np.where(c & 128, -1.0, 1.0)
    v[[0x7F, 0xFF]] = np.nan
    return v


def e4m3_round(x: np.ndarray) -> np.ndarray:
    """Codes (uint8) of x (|x| <= 448) to the nearest value, ties to the even code."""
    grid = e4m3_values()[:0x7F]
    y = np.abs(x)
    hi = np.clip(np.searchsorted(grid, y), 1, len(grid) - 1)
    lo = hi - 1
    up = (grid[hi] - y < y - grid[lo]) | ((grid[hi] - y == y - grid[lo]) & (hi % 2 == 0))
    return (np.where(up, hi, lo) | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def quantise(lat: np.ndarray):
    """Latents [n, 512] -> codes [n, 512] and scale bytes [n, 16]."""
    x = lat.astype(np.float64).reshape(-1, 16, 32)
    amax = np.abs(x).max(-1)
    e = np.full(amax.shape, 7)
    for k in range(6, -16, -1):
        e = np.where(amax <= 448.0 * 2.0 ** k, k, e)
    y = np.clip(x * 2.0 ** -e[..., None], -448.0, 448.0)
    return e4m3_round(y).reshape(-1, LAT), (e + 127).astype(np.uint8)


def pack_rows(lat: np.ndarray, rope: np.ndarray, e4m3: bool) -> np.ndarray:
    """Rows as raw bytes: [n, 1152] or [n, 656]."""
    if not e4m3:
        return np.concatenate([lat, rope], 1).astype(np.float16).view(np.uint8)
    codes, scales = quantise(lat)
    return np.concatenate([codes, rope.astype(np.float16).view(np.uint8), scales], 1)


def row_values(raw: np.ndarray, e4m3: bool) -> np.ndarray:
    """The 576 values of raw rows, in 64 bits."""
    if not e4m3:
        return np.ascontiguousarray(raw).view(np.float16).astype(np.float64)
    lat = e4m3_values()[raw[:, :LAT]].reshape(-1, 16, 32) * 2.0 ** (raw[:, 640:].astype(np.float64) - 127)[..., None]
    rope = np.ascontiguousarray(raw[:, LAT:640]).view(np.float16).astype(np.float64)
    return np.concatenate([lat.reshape(-1, LAT), rope], 1)


def rope_rows(k_pe: np.ndarray, pos: np.ndarray, freq_base: float, freq_scale: float) -> np.ndarray:
    i = np.arange(ROPE // 2)
    a = pos.astype(np.float64)[:, None] * (np.float64(freq_scale) * np.float64(freq_base) ** (-2.0 * i / ROPE))
    x, y = k_pe[:, 0::2].astype(np.float64), k_pe[:, 1::2].astype(np.float64)
    out = np.empty(k_pe.shape)
    out[:, 0::2] = x * np.cos(a) - y * np.sin(a)
    out[:, 1::2] = x * np.sin(a) + y * np.cos(a)
    return out


def visible(p: int, n: int, window: int, n_sink: int) -> np.ndarray:
    j = np.arange(n)
    return (j <= p) & ((window == 0) | (j > p - window) | (j < n_sink))


def attend(q: np.ndarray, rows: np.ndarray, p0: int, window: int, n_sink: int, scale: float):
    """q [n, H, 576] at positions p0, p0 + 1, ..; rows [L, 576] -> (o [n, H, 512], sum_j p_j |c_j| [n, H, 512],
    the number of visible keys [n])."""
    o, a, cnt = [], [], []
    for i in range(q.shape[0]):
        see = np.flatnonzero(visible(p0 + i, rows.shape[0], window, n_sink))
        s = scale * (q[i] @ rows[see].T)
        w = np.exp(s - s.max(-1, keepdims=True))
        w /= w.sum(-1, keepdims=True)
        o.append(w @ rows[see, :LAT])
        a.append(w @ np.abs(rows[see, :LAT]))
        cnt.append(len(see))
    return np.array(o), np.array(a), np.array(cnt)
