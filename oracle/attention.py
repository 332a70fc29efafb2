"""The attention step beside the Engram forward -- oracle side, test infrastructure only.

Query/key norm and rotation, the paged cache and its 8-bit format, attention of
one new token per sequence, and the 4-bit weight's product, each from its
formula in float64 with one rounding where a value is stored.
"""

from __future__ import annotations

import numpy as np

from .mx import MX_BLOCK, e8m0_mx_scale, _e4m3_rne
from .numerics import bf16_value, e4m3fn_value

E2M1_VALUES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


# ---------------------------------------------------------------- norm and rotation

def qk_norm_rope(x_bits, weight_bits, eps, positions, inv_freq, interleaved):
    """Heads x bf16 [T, H, D] normed and rotated: (float64 results, float64 sums of the
    magnitudes of each result's two terms, for error bounds)."""
    x = bf16_value(x_bits)
    y = x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps) * bf16_value(weight_bits)
    half = len(inv_freq)
    angle = np.asarray(positions, np.float64)[:, None, None] * np.asarray(inv_freq, np.float64)
    i = np.arange(half)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    a, b = y[..., ia], y[..., ib]
    out, mag = y.copy(), np.abs(y)
    out[..., ia] = a * np.cos(angle) - b * np.sin(angle)
    out[..., ib] = b * np.cos(angle) + a * np.sin(angle)
    mag[..., ia] = mag[..., ib] = np.abs(a) + np.abs(b)
    return out, mag


# ---------------------------------------------------------------- the cache

def quantize_cache(bits):
    """bf16 [..., D] as the 8-bit cache holds it: (codes [..., D], scales [..., D / 32]).

    Per 32 values the smallest power of two 2**e, e >= -95, with amax / 2**e <= 448 (amax
    over the finite values; e = 0 where it is 0); codes to nearest even; infinities and
    NaN become the format's NaN.
    """
    bits = np.asarray(bits, np.uint16)
    x = bf16_value(bits).reshape(*bits.shape[:-1], -1, MX_BLOCK)
    finite = np.isfinite(x)
    amax = np.max(np.where(finite, np.abs(x), 0.0), axis=-1)
    m, e = np.frexp(amax)                             # amax = m * 2**e, 448 = 0.875 * 2**9
    e = np.where(amax > 0, np.maximum(e - 9 + (m > 0.875), -95), 0)
    scaled = np.where(finite, x, 0.0) / np.ldexp(1.0, e)[..., None]
    codes = np.where(finite, _e4m3_rne(scaled), 0x7F | (np.signbit(x) * 0x80))
    return codes.astype(np.uint8).reshape(bits.shape), (e + 127).astype(np.uint8)


def cache_values(codes, scales):
    """float64 values of 8-bit cache rows [..., D] with scales [..., D / 32]."""
    v = e4m3fn_value(codes)
    return v * np.repeat(e8m0_mx_scale(scales), MX_BLOCK, axis=-1)


def cache_rows(data, scales, slots):
    """float64 [T, heads, D] of the places `slots` of cache tensor data [pages, heads, ps, D]."""
    ps = data.shape[2]
    slots = np.asarray(slots)
    d = data[slots // ps, :, slots % ps]
    if scales is None:
        return bf16_value(d)
    return cache_values(d, scales[slots // ps, :, slots % ps])


# ---------------------------------------------------------------- attention

def paged_attention(k, v, k_scales, v_scales, q_bits, table, lens, max_len, scale, window=0):
    """(out, lse, spread, logit): float64 out [n, hq, D] and lse [n, hq]; for error bounds
    spread = sum p |v| / sum p like out, and the largest scale * sum |q_d k_d| like lse."""
    pages, hkv, ps, D = k.shape
    n, hq, _ = q_bits.shape
    q = bf16_value(q_bits).reshape(n, hkv, hq // hkv, D)
    out = np.zeros((n, hkv, hq // hkv, D))
    spread = np.zeros_like(out)
    lse = np.full((n, hkv, hq // hkv), -np.inf)
    logit = np.zeros((n, hkv, hq // hkv))
    for s in range(n):
        length = min(max(int(lens[s]), 0), max_len, table.shape[1] * ps)
        p = np.arange(max(0, length - window) if window else 0, length)
        page = table[s][p // ps].astype(np.int64) if len(p) else p
        ok = (page >= 0) & (page < pages)
        p, page = p[ok], page[ok]
        if not len(p):
            continue
        slots = page * ps + p % ps
        kk = cache_rows(k, k_scales, slots).transpose(1, 0, 2)        # [hkv, L, D]
        vv = cache_rows(v, v_scales, slots).transpose(1, 0, 2)
        z = q[s] @ kk.transpose(0, 2, 1) * scale
        logit[s] = (np.abs(q[s]) @ np.abs(kk).transpose(0, 2, 1)).max(-1) * abs(scale)
        top = z.max(-1, keepdims=True)
        w = np.exp(z - top)
        total = w.sum(-1, keepdims=True)
        out[s] = (w / total) @ vv
        spread[s] = (w / total) @ np.abs(vv)
        lse[s] = (top + np.log(total))[..., 0]
    return (out.reshape(n, hq, D), lse.reshape(n, hq), spread.reshape(n, hq, D),
            logit.reshape(n, hq))


# ---------------------------------------------------------------- the 4-bit weight

def quantize_mxfp4(w_bits):
    """MXFP4 copy of bf16 w [N, K]: (codes [N, K / 2], scales [N, K / 32]), OCP MX v1.0."""
    w = bf16_value(w_bits)
    N, K = w.shape
    b = w.reshape(N, K // MX_BLOCK, MX_BLOCK)
    amax = np.abs(b).max(-1)
    _, e = np.frexp(amax)
    byte = np.where(amax > 0, np.clip(e - 1 - 2 + 127, 0, 254), 127)
    x = np.abs(b) / np.ldexp(1.0, byte - 127)[..., None]
    # The nearest value, by distance; of two at one distance the even code.
    d = np.abs(np.minimum(x, 6.0)[..., None] - E2M1_VALUES)
    near = d == d.min(-1, keepdims=True)
    code = np.where(near & (np.arange(8) % 2 == 0), 2, near).argmax(-1)
    code = (code + 8 * np.signbit(b)).reshape(N, K).astype(np.uint8)
    return code[:, 0::2] | code[:, 1::2] << 4, byte.astype(np.uint8)


def mxfp4_values(codes, scales):
    """float64 [N, K] of an MXFP4 weight."""
    code = np.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[0], -1)
    v = E2M1_VALUES[code & 7] * np.where(code & 8, -1.0, 1.0)
    return v * np.repeat(e8m0_mx_scale(scales), MX_BLOCK, axis=-1)


def project_mxfp4(x_bits, codes, scales):
    """(float64 out [T, N], float64 sums of the products' magnitudes)."""
    x, w = bf16_value(x_bits), mxfp4_values(codes, scales)
    return x @ w.T, np.abs(x) @ np.abs(w).T
