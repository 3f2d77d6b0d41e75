"""Rows of the device row cache, attention over them, and the 8-bit norm, in
float64.

TEST INFRASTRUCTURE ONLY.  Only the tests may import this module.  It shares no
code with the CUDA library: it states the definitions with numpy.

A latent row is c^KV[512] + k^R[64].  Formats: "bf16" (1152 bytes), "compact"
(656 bytes, see compact_row) and "q4" (400 bytes): 256 bytes of e2m1 codes,
value 2i in the low half of byte i; 16 exponent bytes, block j of 32 values
scaled by 2^(byte - 127); 64 RoPE values as bf16.  A block's scale is the
smallest power of two at or above fl32(amax / 6), 1 for an all-zero block, its
exponent within -23..13.
"""
from __future__ import annotations

import numpy as np

from oracle import compact_row as X

LATENT, ROPE, ROW = 512, 64, 576
ROW_BYTES = {"bf16": 1152, "compact": 656, "q4": 400}
BLOCK = 32
MIN_EXP, MAX_EXP = -23, 13
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([X.e4m3_value(c) for c in range(0x7F)])


def bf16_value(bits: np.ndarray) -> np.ndarray:
    return (np.ascontiguousarray(bits, dtype=np.uint16).astype(np.uint32) << 16).view(
        np.float32).astype(np.float64)


def power_at_least(x: np.ndarray) -> np.ndarray:
    """Exponent of the smallest power of two >= x > 0; 0 where x is 0."""
    m, e = np.frexp(np.asarray(x, dtype=np.float64))
    return np.where(np.asarray(x) > 0, e - (m == 0.5), 0).astype(np.int64)


def block_exps(y: np.ndarray, size: int, top: float) -> np.ndarray:
    """[n][blocks] scale exponents of blocks of `size` values (the last block may be shorter)."""
    n, dim = y.shape
    pad = -(-dim // size) * size - dim
    a = np.abs(np.pad(y, ((0, 0), (0, pad)))).reshape(n, -1, size).max(axis=2)
    return power_at_least((a.astype(np.float32) / np.float32(top)))


def nearest_code(a: np.ndarray, levels: np.ndarray) -> np.ndarray:
    """Code of the nearest level of magnitudes a: the even one of two as near, the last above all."""
    i = np.clip(np.searchsorted(levels, a), 1, len(levels) - 1)
    down, up = a - levels[i - 1], levels[i] - a
    return np.where((down < up) | ((down == up) & (i % 2 == 1)), i - 1, i)


def q4_encode(y: np.ndarray) -> tuple[np.ndarray, np.ndarray]:
    """float64 [n][512] -> (packed codes uint8 [n][256], exponent bytes uint8 [n][16])."""
    e = np.clip(block_exps(y, BLOCK, 6.0), MIN_EXP, MAX_EXP)
    u = y / np.repeat(2.0 ** e, BLOCK, axis=1)
    code = nearest_code(np.abs(u), E2M1) + 8 * np.signbit(u)
    return (code[:, 0::2] + 16 * code[:, 1::2]).astype(np.uint8), (e + 127).astype(np.uint8)


def q4_decode(packed: np.ndarray, exps: np.ndarray) -> np.ndarray:
    code = np.empty((packed.shape[0], 2 * packed.shape[1]), dtype=np.int64)
    code[:, 0::2], code[:, 1::2] = packed & 15, packed >> 4
    v = E2M1[code & 7] * np.where(code & 8, -1.0, 1.0)
    e = np.clip(exps.astype(np.int64) - 127, MIN_EXP, MAX_EXP)
    return v * np.repeat(2.0 ** e, BLOCK, axis=1)


def row_values(rows: np.ndarray, fmt: str) -> np.ndarray:
    """uint8 [n][row bytes] -> float64 [n][576]."""
    rows = np.ascontiguousarray(rows)
    if fmt == "bf16":
        return bf16_value(rows.view(np.uint16))
    rope = bf16_value(np.ascontiguousarray(rows[:, -128:]).view(np.uint16))
    if fmt == "compact":
        full = np.concatenate([E4M3, [np.nan]])
        c = rows[:, :512]
        scale = np.ascontiguousarray(rows[:, 512:528]).view(np.float32).astype(np.float64)
        y = full[c & 127] * np.where(c & 128, -1.0, 1.0) * np.repeat(scale, 128, axis=1)
    else:
        y = q4_decode(rows[:, :256], rows[:, 256:272])
    return np.concatenate([y, rope], axis=1)


def rms_norm(x: np.ndarray, gamma: np.ndarray, eps: float) -> np.ndarray:
    x = x.astype(np.float64)
    r = 1.0 / np.sqrt((x * x).mean(axis=1, keepdims=True) + float(np.float32(eps)))
    return x * r * gamma.astype(np.float64)


def rotate(k: np.ndarray, pos: np.ndarray, inv_freq, halves: bool) -> np.ndarray:
    """k [n][64] turned by pos * inv_freq, 32 pairs (2i, 2i+1) or (i, i + 32)."""
    k = k.astype(np.float64)
    z = k[:, :32] + 1j * k[:, 32:] if halves else k[:, 0::2] + 1j * k[:, 1::2]
    angle = np.longdouble(1) * pos.astype(np.int64)[:, None] * np.asarray(inv_freq, dtype=np.float64)
    turn = 2 * np.longdouble("3.14159265358979323846264338327950288")
    angle = (angle - turn * np.floor(angle / turn)).astype(np.float64)
    z = z * (np.cos(angle) + 1j * np.sin(angle))
    out = np.empty_like(k)
    if halves:
        out[:, :32], out[:, 32:] = z.real, z.imag
    else:
        out[:, 0::2], out[:, 1::2] = z.real, z.imag
    return out


def attention(q: np.ndarray, k: np.ndarray, sm_scale: float, keep: np.ndarray):
    """One query set over one set of rows: q [rows][576], k [n][576], keep
    [rows][n] bool.  Returns (out [rows][512], lse [rows], weighted |v| [rows][512])."""
    z = (q @ k.T) * float(np.float32(sm_scale))
    z = np.where(keep, z, -np.inf)
    top = z.max(axis=1, initial=-np.inf)
    base = np.where(np.isfinite(top), top, 0.0)
    p = np.where(keep, np.exp(z - base[:, None]), 0.0)
    total = p.sum(axis=1)
    safe = np.where(total > 0, total, 1.0)
    out = (p @ k[:, :LATENT]) / safe[:, None]
    size = (p @ np.abs(k[:, :LATENT])) / safe[:, None]
    with np.errstate(divide="ignore"):
        lse = np.where(total > 0, base + np.log(safe), -np.inf)
    return out, lse, size


def norm_quant(h: np.ndarray, gamma: np.ndarray, eps: float):
    """(y float64 [n][dim], scale exponents [n][ceil(dim / 128)])."""
    y = rms_norm(h, gamma, eps)
    return y, np.maximum(block_exps(y, 128, 448.0), -126)
