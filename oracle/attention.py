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


# ---------------------------------------------------------------- several new tokens, shared prefixes, eviction

U32 = 2.0 ** -24                                       # half a step of fp32


def rules_of(window=0, cap=0.0, slopes=None, doc_starts=None, prefix_lens=None):
    return dict(window=window, cap=cap, slopes=slopes, doc_starts=doc_starts, prefix_lens=prefix_lens)


def _places(cache, table_row, length):
    """Keys and values float64 [hkv, L, D] of the places 0..length-1, and which lie on a page of the cache."""
    k, v, ks, vs = cache
    pages, _, ps, _ = k.shape
    p = np.arange(length)
    page = np.asarray(table_row)[p // ps].astype(np.int64) if length else p
    ok = (page >= 0) & (page < pages)
    slots = np.where(ok, page, 0) * ps + p % ps
    return (cache_rows(k, ks, slots).transpose(1, 0, 2), cache_rows(v, vs, slots).transpose(1, 0, 2), ok)


def _scores(q, k, scale, rules, pos, h):
    """Scores [n, L] of one head's new tokens at places pos, and how far fp32 ones may be off:
    D roundings in the product, some in the cap (2^-21 of it at most) and the bias."""
    p = np.arange(k.shape[0])
    with np.errstate(invalid="ignore", over="ignore"):
        z = q @ k.T * scale
        mag = np.abs(q) @ np.abs(k).T * abs(scale)
    off = U32 * (q.shape[1] + 4) * mag
    if rules["cap"]:
        z = rules["cap"] * np.tanh(z / rules["cap"])
        off = off + 2.0 ** -21 * np.minimum(rules["cap"], mag)
    if rules["slopes"] is not None:
        bias = float(rules["slopes"][h]) * np.abs(pos[:, None] - p)
        z, off = z - bias, off + 4 * U32 * (np.abs(bias) + np.abs(z))
    return z, off


def _seen(rules, s, tokens, pos, length, ok):
    p = np.arange(length)
    seen = p <= pos[:, None]
    if rules["window"]:
        seen &= pos[:, None] - p < rules["window"]
    if rules["prefix_lens"] is not None:
        seen |= p < int(rules["prefix_lens"][s])
    if rules["doc_starts"] is not None:
        seen &= p >= np.asarray(rules["doc_starts"])[tokens][:, None].astype(np.int64)
    return seen & ok


def _softmax_row(z, off, seen, v):
    """out, lse, sum w |v|, and the bounds that `off` gives: of out [n, D] and of lse [n]."""
    n, D = z.shape[0], v.shape[1]
    z = np.where(seen, z, -np.inf)
    some = seen.any(1)
    top = np.where(some, z.max(1, initial=-np.inf), 0.0)
    e = np.exp(z - top[:, None])
    total = e.sum(1)
    w = np.divide(e, total[:, None], out=np.zeros_like(e), where=total[:, None] > 0)
    lse = np.full(n, -np.inf)
    lse[some] = top[some] + np.log(total[some])
    used = seen.any(0)                                 # what no row sees may be anything
    w, v, off = w[:, used], v[used], np.where(seen, off, 0.0)[:, used]
    # A place that one row does not see may hold NaN that another sees.
    odd = ~np.isfinite(v)
    fine, weight = np.where(odd, 0.0, v), np.where(seen[:, used], w, 0.0)
    out, spread = weight @ fine, weight @ np.abs(fine)
    slack = (weight * off) @ np.abs(fine) + (weight * off).sum(1)[:, None] * np.abs(out)
    if odd.any():
        out = np.where((seen[:, used].astype(float) @ odd) > 0, np.nan, out)
    return out.reshape(n, D), lse, spread, slack, (weight * off).sum(1)


def chunk_attention(cache, q_bits, cu, table, lens, max_len, scale, rules=None):
    """(out, lse, spread, slack, lse_slack) of the tokens in cu; float64 [T, hq, D] or [T, hq]."""
    rules = rules or rules_of()
    hkv, ps = cache[0].shape[1:3]
    T, hq, D = q_bits.shape
    q = bf16_value(q_bits)
    out, spread, slack = np.zeros((T, hq, D)), np.zeros((T, hq, D)), np.zeros((T, hq, D))
    lse, lse_slack = np.full((T, hq), -np.inf), np.zeros((T, hq))
    for s in range(len(lens)):
        tokens = np.arange(cu[s], cu[s + 1])
        length = min(max(int(lens[s]), 0), max_len, table.shape[1] * ps)
        if not len(tokens) or not length:
            continue
        pos = length - len(tokens) + np.arange(len(tokens))
        k, v, ok = _places(cache, table[s], length)
        seen = _seen(rules, s, tokens, pos, length, ok)
        for h in range(hq):
            kk = np.where(seen.any(0)[:, None], k[h // (hq // hkv)], 0.0)
            z, off = _scores(q[tokens, h], kk, scale, rules, pos, h)
            got = _softmax_row(z, off, seen, v[h // (hq // hkv)])
            for a, x in zip((out, lse, spread, slack, lse_slack), got):
                a[tokens, h] = x
    return out, lse, spread, slack, lse_slack


def shared_prefix_attention(cache, q_bits, cu_groups, prefix_table, prefix_lens, max_prefix, table, lens, max_len, scale):
    """chunk_attention's results for one new token a sequence over its group's prefix and its own places."""
    hkv, ps = cache[0].shape[1:3]
    n, hq, D = q_bits.shape
    q = bf16_value(q_bits)
    got = [np.zeros((n, hq, D)), np.full((n, hq), -np.inf), np.zeros((n, hq, D)), np.zeros((n, hq, D)), np.zeros((n, hq))]
    prefix = [_places(cache, prefix_table[g], min(max(int(prefix_lens[g]), 0), max_prefix, prefix_table.shape[1] * ps))
              for g in range(len(prefix_lens))]
    for s in range(n):
        k, v, ok = _places(cache, table[s], min(max(int(lens[s]), 0), max_len, table.shape[1] * ps))
        for g in range(len(prefix_lens)):
            if cu_groups[g] <= s < cu_groups[g + 1]:
                k0, v0, ok0 = prefix[g]
                k, v, ok = np.concatenate([k0, k], 1), np.concatenate([v0, v], 1), np.concatenate([ok0, ok])
        if not len(ok):
            continue
        for h in range(hq):
            kk = np.where(ok[:, None], k[h // (hq // hkv)], 0.0)
            z, off = _scores(q[s, h][None], kk, scale, rules_of(), np.zeros(1), h)
            for a, x in zip(got, _softmax_row(z, off, ok[None], v[h // (hq // hkv)])):
                a[s, h] = x[0]
    return got


def cache_weights(cache, q_bits, cu, table, lens, max_len, scale, lse, stride, rules=None):
    """(weights added [n, hkv, stride], how far fp32 ones may be off)."""
    rules = rules or rules_of()
    hkv, ps = cache[0].shape[1:3]
    hq = q_bits.shape[1]
    q = bf16_value(q_bits)
    w, slack = np.zeros((len(lens), hkv, stride)), np.zeros((len(lens), hkv, stride))
    for s in range(len(lens)):
        tokens = np.arange(cu[s], cu[s + 1])
        length = min(max(int(lens[s]), 0), max_len, table.shape[1] * ps)
        if not len(tokens) or not length:
            continue
        pos = length - len(tokens) + np.arange(len(tokens))
        k, _, ok = _places(cache, table[s], length)
        seen = _seen(rules, s, tokens, pos, length, ok)
        for h in range(hq):
            kvh = h // (hq // hkv)
            z, off = _scores(q[tokens, h], np.where(seen.any(0)[:, None], k[kvh], 0.0), scale, rules, pos, h)
            ref = np.asarray(lse, np.float64)[tokens, h][:, None]
            seen_h = seen & ~np.isneginf(ref)
            e = np.where(seen_h, np.exp(np.where(seen_h, z - np.where(np.isneginf(ref), 0, ref), 0.0)), 0.0)
            off = np.where(seen_h, off + 4 * U32 * (np.abs(z) + np.abs(np.where(np.isneginf(ref), 0, ref))), 0.0)
            w[s, kvh, :length] += e.sum(0)
            # Exponentials (2 u), and the sums of the rows of 16 lanes, then of those.
            slack[s, kvh, :length] += (e * (off + (8 + len(tokens) * (hq // hkv) / 16) * U32)).sum(0)
    return w, slack


def evict(weights, lens, max_len, room, keep, sinks, recent):
    """kept int32 [n, hkv, keep]: the places that stay, in order, then -1."""
    n, hkv, _ = weights.shape
    kept = np.full((n, hkv, keep), -1, np.int32)
    for s in range(n):
        length = min(max(int(lens[s]), 0), max_len, room)
        for h in range(hkv):
            p = np.arange(length)
            if length > keep:
                w = weights[s, h, :length].astype(np.float64)
                must = (p < sinks) | (p >= length - recent)
                # Those that stay anyway, then numbers before NaN, then larger before smaller, then the first.
                order = np.lexsort((p, np.where(np.isnan(w), 0.0, -w), np.isnan(w), ~must))
                p = np.sort(order[:keep])
            kept[s, h, :len(p)] = p
    return kept
