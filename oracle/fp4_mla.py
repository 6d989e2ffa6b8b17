"""CPU ORACLE of the 4-bit MLA rows and the attention over them -- TEST INFRASTRUCTURE ONLY.
Plain numpy in float64.

A row is 416 B: 256 B of e2m1 codes (dim 2i in the low nibble of byte i), 32 B of e4m3 scales (one
per 16 dims), 128 B of bf16 RoPE values; latent = e2m1 x e4m3 x g, g a power of two. A row is
written with, per block of 16 values y = x / g: scale = e4m3(max |y| / 6), code = e2m1(y / scale),
nearest, halfway to the even code, saturating; scale 0 gives codes 0; a NaN or an infinity gives
scale NaN (0x7F) and codes 0.

Attention, per query over the rows j that it sees: s_j = sm (q[:512] . latent_j + q[512:] . rope_j),
o = softmax(s) . latent, lse = log sum exp s; nothing seen: o = 0, lse = -inf. A window query at
token p sees t <= p with t < sinks or t > p - window.
"""
from __future__ import annotations

import numpy as np

from .sparse_mla import bf16_decode, e4m3_decode

ROW, LATENT, ROPE, BLOCK = 416, 512, 64, 16
DIMS = LATENT + ROPE
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
E4M3 = e4m3_decode(np.arange(127))  # 0 .. 448, ascending


def nearest_code(x: np.ndarray, values: np.ndarray) -> np.ndarray:
    """Index of the nearest of `values` (ascending from 0); halfway goes to the even index, past the
    end to the last."""
    hi = np.clip(np.searchsorted(values, x, side="left"), 0, len(values) - 1)
    lo = np.maximum(hi - 1, 0)
    up, down = values[hi] - x, x - values[lo]
    take_low = (down < up) | ((down == up) & (lo % 2 == 0))
    return np.where(take_low, lo, hi)


def pack(kv_bits: np.ndarray, g: float) -> np.ndarray:
    """bf16 bit patterns [n, 576] -> rows [n, 416]."""
    n = kv_bits.shape[0]
    y = bf16_decode(kv_bits[:, :LATENT]).reshape(n, -1, BLOCK) / g
    bad = ~np.isfinite(y).all(-1)
    y = np.where(bad[..., None], 0.0, y)
    scale = nearest_code(np.abs(y).max(-1) / 6, E4M3)
    s = E4M3[scale][..., None]
    q = np.divide(y, s, out=np.zeros_like(y), where=s > 0)
    code = nearest_code(np.abs(q), E2M1) | np.where(np.signbit(q) & (s > 0), 8, 0)
    code[bad] = 0
    code = code.reshape(n, LATENT).astype(np.uint8)
    out = np.empty((n, ROW), np.uint8)
    out[:, :256] = code[:, 0::2] | (code[:, 1::2] << 4)
    out[:, 256:288] = np.where(bad, 0x7F, scale)
    out[:, 288:] = np.ascontiguousarray(kv_bits[:, LATENT:]).view(np.uint8)
    return out


def unpack(rec: np.ndarray, g: float):
    """Rows [n, 416] -> (latent [n, 512], rope [n, 64])."""
    code = np.stack((rec[:, :256] & 15, rec[:, :256] >> 4), -1).reshape(-1, LATENT)
    val = E2M1[code & 7] * np.where(code & 8, -1.0, 1.0)
    scale = np.repeat(e4m3_decode(rec[:, 256:288]), BLOCK, axis=1)
    return val * scale * g, bf16_decode(np.ascontiguousarray(rec[:, 288:]).view("<u2"))


def attend(q: np.ndarray, lat: np.ndarray, rope: np.ndarray, sm: float):
    """q [M, 576] over rows [n]: (o [M, 512], lse [M], and for error bounds the weighted magnitudes
    sum_j p_j |latent_j| [M, 512] and the largest sm sum_d |q_d v_jd| [M])."""
    if lat.shape[0] == 0:
        z = np.zeros((q.shape[0], LATENT))
        return z, np.full(q.shape[0], -np.inf), z, np.zeros(q.shape[0])
    k = np.concatenate((lat, rope), 1)
    s = sm * (q @ k.T)
    top = s.max(1, keepdims=True)
    e = np.exp(s - top)
    z = e.sum(1, keepdims=True)
    p = e / z
    return p @ lat, (top + np.log(z))[:, 0], p @ np.abs(lat), (abs(sm) * (np.abs(q) @ np.abs(k).T)).max(1)


def window_tokens(p: int, window: int, sinks: int) -> np.ndarray:
    t = np.arange(max(p + 1, 0))
    return t[(t < sinks) | (t > p - window)]
