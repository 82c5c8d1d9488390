"""Float64 NumPy definitions of the latent cache's operators (rotary positions, the fp8 number
format, latent attention), written apart from the GPU code.  Slow and plain.
"""
from __future__ import annotations

import math

import numpy as np

LAT, ROPE = 512, 64


def rope_frequencies(theta: float, dim: int, kind: str = "none", factor: float = 1.0, orig_len: int = 0,
                     beta_fast: float = 32.0, beta_slow: float = 1.0) -> np.ndarray:
    """Inverse frequencies of the dim/2 pairs: plain, position interpolation, or YaRN."""
    out = np.zeros(dim // 2)
    if kind == "yarn":
        at = lambda turns: dim * math.log(orig_len / (turns * 2 * math.pi)) / (2 * math.log(theta))  # noqa: E731
        lo, hi = max(0, math.floor(at(beta_fast))), min(dim - 1, math.ceil(at(beta_slow)))
    for i in range(dim // 2):
        f = theta ** (-2.0 * i / dim)
        if kind == "linear":
            f = f / factor
        elif kind == "yarn":
            r = min(1.0, max(0.0, (i - lo) / (hi - lo))) if hi > lo else float(i > lo)
            f = f * (1 - r) + f / factor * r
        out[i] = f
    return out


def rope(x: np.ndarray, cos: np.ndarray, sin: np.ndarray, interleaved: bool, inverse: bool) -> np.ndarray:
    """x [..., dim] turned pair by pair; cos and sin [..., dim/2] broadcast against x's leading dims."""
    half = x.shape[-1] // 2
    y = np.empty_like(x, dtype=np.float64)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        c, s = cos[..., i], -sin[..., i] if inverse else sin[..., i]
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., a] * s + x[..., b] * c
    return y


def e4m3_values() -> np.ndarray:
    """The value of each of the 256 codes (0x7F and 0xFF are NaN)."""
    v = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = (m / 8.0) * 2.0 ** -6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7)
        v[c] = math.nan if (c & 127) == 127 else (-x if c & 128 else x)
    return v


def scale_exponent(amax: float) -> int:
    """Smallest e in [-100, 7] with amax <= 448 * 2^e (7 where none is)."""
    for e in range(-100, 8):
        if amax <= 448.0 * 2.0 ** e:
            return e
    return 7


def fp8_encode(x: np.ndarray):
    """x [n, 512] -> (codes uint8 [n, 512], scale bytes uint8 [n, 4])."""
    table = e4m3_values()[:127]               # the non-negative codes 0 .. 126, ascending
    n = x.shape[0]
    codes = np.zeros((n, LAT), dtype=np.uint8)
    scale = np.zeros((n, 4), dtype=np.uint8)
    for t in range(n):
        for g in range(4):
            v = x[t, 128 * g:128 * (g + 1)]
            if not np.all(np.isfinite(v)):
                scale[t, g] = 255
                codes[t, 128 * g:128 * (g + 1)] = 127
                continue
            e = scale_exponent(float(np.max(np.abs(v))))
            scale[t, g] = e + 127
            a = np.minimum(np.abs(v) * 2.0 ** -e, 448.0)
            hi = np.clip(np.searchsorted(table, a), 0, 126)
            lo = np.maximum(hi - 1, 0)
            # nearest; halfway goes to the even code
            dl, dh = a - table[lo], table[hi] - a
            c = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
            codes[t, 128 * g:128 * (g + 1)] = c | np.where(np.signbit(v), 128, 0)
    return codes, scale


def fp8_decode(codes: np.ndarray, scale: np.ndarray) -> np.ndarray:
    """Codes and scale bytes back to values; bytes above 134 are NaN."""
    f = np.where(scale > 134, math.nan, 2.0 ** (scale.astype(np.float64) - 127))
    return e4m3_values()[codes] * np.repeat(f, 128, axis=1)


def latent_attn_row(q: np.ndarray, kv: np.ndarray, tau: float):
    """q [H, 576] over kv [n, 576]: (out [H, 512], lse [H], A [H, 512] = sum_j w_j |v_j|,
    B [H] = max_j tau sum_d |q_d kv_jd|)."""
    H = q.shape[0]
    if kv.shape[0] == 0:
        return np.zeros((H, LAT)), np.full(H, -np.inf), np.zeros((H, LAT)), np.zeros(H)
    s = tau * (q @ kv.T)
    m = s.max(axis=1, keepdims=True)
    p = np.exp(s - m)
    tot = p.sum(axis=1, keepdims=True)
    w = p / tot
    return w @ kv[:, :LAT], (m + np.log(tot))[:, 0], w @ np.abs(kv[:, :LAT]), tau * (np.abs(q) @ np.abs(kv).T).max(axis=1)
