"""The attention step's operators against oracle/attention.py (float64), on the GPU.

Tolerances, from the number of roundings (u = 2^-24 of fp32, h = 2^-8 the half step of bf16):
* norm and rotation: h |y| for the one rounding of the result, and 2^-20 (|a| + |b|) for its
  two terms: some 20 fp32 roundings in the norm, the weight, the products and their sum, sine
  and cosine being off by less than 2^-22 (the angle is reduced in fp64);
* the cache: bit for bit, both ways;
* attention: logits are off by d = D u times the largest scale * sum |q k|, so that weights
  are off by d, by h where they are rounded for the matrix cores and by 2^-18 for exponentials,
  joins and sums: (h + 2 d + 2^-18) sum p |v| / sum p, and h |out| for the result.  The log of
  the sum: d, (length / 32 + 32) u for the sum, 4 u |lse|;
* the 4-bit product: K u sum |x w|, and h |out|.
"""

import numpy as np
import pytest
import torch

import oracle
from oracle import attention as oa

pytestmark = pytest.mark.gpu

U, H = 2.0 ** -24, 2.0 ** -8


@pytest.fixture(scope="module")
def eg():
    import __graft_entry__
    __graft_entry__._ensure_built()
    import gram_hash_memory_amd
    torch.cuda.set_device(0)
    return gram_hash_memory_amd


def bits(x):
    return oracle.bf16_bits(oracle.bf16_round(np.asarray(x, np.float64)))


def dev(a):
    a = np.ascontiguousarray(a)
    return torch.from_numpy(a.view(np.int16) if a.dtype == np.uint16 else a).cuda()


def host(t):
    a = t.cpu().numpy()
    return a.view(np.uint16) if a.dtype == np.int16 else a


class Guarded:
    """A GPU buffer with sentinels around it."""

    PAD = 4096
    FILL = {torch.int16: 0x5A5A, torch.uint8: 0xA5, torch.float32: 1234.5}

    def __init__(self, shape, dtype):
        n = int(np.prod(shape))
        self.all = torch.full((n + 2 * self.PAD,), self.FILL[dtype], dtype=dtype, device="cuda")
        self.t = self.all[self.PAD:self.PAD + n].view(*shape)

    def host(self):
        edge = torch.cat([self.all[:self.PAD], self.all[-self.PAD:]])
        assert bool((edge == self.FILL[self.all.dtype]).all()), "written outside the buffer"
        return host(self.t)


def within(got_bits, want, tol):
    got = oracle.bf16_value(got_bits)
    over = np.abs(got - want) - tol
    assert np.all(np.isfinite(got)) and over.max() <= 0, \
        f"off by {np.abs(got - want).flat[over.argmax()]:.3g}, allowed {tol.flat[over.argmax()]:.3g}"


# ---------------------------------------------------------------- norm and rotation

ROPE = [  # T, q heads, kv heads, D, rot, interleaved, pad, far
    (1, 1, 1, 32, 16, False, 0, 10), (1, 32, 8, 128, 128, False, 0, 131072), (5, 3, 1, 64, 64, True, 8, 1000),
    (64, 32, 8, 128, 64, True, 0, 32768), (37, 12, 4, 96, 48, False, 24, 1000000),
    (33, 6, 2, 96, 96, True, 0, 500), (19, 5, 5, 160, 80, False, 16, 77777), (8, 16, 2, 192, 192, False, 40, 9),
    (300, 7, 1, 256, 128, True, 8, 200000), (2, 64, 8, 256, 256, False, 0, 1000000), (3, 2, 1, 224, 32, False, 0, 50),
    (1025, 8, 8, 128, 128, True, 0, 4096), (129, 24, 3, 64, 32, False, 48, 12345),
]


def rope_inputs(rng, T, hq, hkv, D, rot, pad, far):
    width = (hq + 2 * hkv) * D
    row = bits(rng.normal(size=(T, width + pad)) * rng.uniform(0.2, 4.0, size=(T, 1)))
    qw, kw = bits(1 + 0.2 * rng.normal(size=D)), bits(1 + 0.2 * rng.normal(size=D))
    pos = rng.integers(0, far, size=T).astype(np.int32)
    inv = 10000.0 ** (-2.0 * np.arange(rot // 2) / rot)
    return row, dev(row)[:, :width], qw, kw, pos, inv


@pytest.mark.parametrize("T,hq,hkv,D,rot,inter,pad,far", ROPE)
def test_qk_norm_rope(eg, T, hq, hkv, D, rot, inter, pad, far):
    rng = np.random.default_rng(T + D)
    row, qkv, qw, kw, pos, inv = rope_inputs(rng, T, hq, hkv, D, rot, pad, far)
    q, k = Guarded((T, hq, D), torch.int16), Guarded((T, hkv, D), torch.int16)
    eg.engram_qk_norm_rope(qkv, hq, hkv, D, dev(qw), dev(kw), 1e-6, dev(pos), dev(inv), inter, q.t, k.t)
    x = row[:, :(hq + hkv) * D].reshape(T, hq + hkv, D)
    for got, xs, w in ((q, x[:, :hq], qw), (k, x[:, hq:], kw)):
        want, mag = oa.qk_norm_rope(xs, w, 1e-6, pos, inv, inter)
        within(got.host(), want, H * np.abs(want) + 2.0 ** -20 * mag + 1e-38)


def test_qk_norm_rope_zero_row_and_far_positions(eg):
    """A zero head stays 0; the largest positions keep their angle; a row wider than needed."""
    rng = np.random.default_rng(0)
    T, hq, hkv, D, rot = 4, 2, 1, 64, 64
    row, qkv, qw, kw, pos, inv = rope_inputs(rng, T, hq, hkv, D, rot, 8, 9)
    qkv[1] = 0
    row[1] = 0
    pos = np.array([0, 5, 2 ** 31 - 1, -7], np.int32)
    q, k = Guarded((T, hq, D), torch.int16), Guarded((T, hkv, D), torch.int16)
    eg.engram_qk_norm_rope(qkv, hq, hkv, D, dev(qw), dev(kw), 1e-6, dev(pos), dev(inv), False, q.t, k.t)
    x = row[:, :(hq + hkv) * D].reshape(T, hq + hkv, D)
    want, mag = oa.qk_norm_rope(x[:, :hq], qw, 1e-6, pos, inv, False)
    within(q.host(), want, H * np.abs(want) + 2.0 ** -20 * mag)
    assert not oracle.bf16_value(q.host()[1]).any() and not oracle.bf16_value(k.host()[1]).any()    # either zero


# ---------------------------------------------------------------- the cache

def make_cache(eg, rng, fmt, pages, hkv, ps, D):
    """A cache full of values, as numpy (k, v, k_scales, v_scales) and on the GPU."""
    shape = (pages, hkv, ps, D)
    if fmt == "bf16":
        k, v = bits(rng.normal(size=shape)), bits(rng.normal(size=shape))
        ks = vs = None
    else:
        k, ks = oa.quantize_cache(bits(rng.normal(size=shape) * 2.0 ** rng.integers(-3, 4, size=(pages, 1, ps, 1))))
        v, vs = oa.quantize_cache(bits(rng.normal(size=shape)))
    held = [Guarded(a.shape, torch.int16 if a.dtype == np.uint16 else torch.uint8) if a is not None else None
            for a in (k, v, ks, vs)]
    for g, a in zip(held, (k, v, ks, vs)):
        if g is not None:
            g.t.copy_(dev(a))
    handle = eg.KVCache(eg.ENGRAM_CACHE_BF16 if fmt == "bf16" else eg.ENGRAM_CACHE_MXFP8,
                        *[None if g is None else g.t for g in held])
    return [k, v, ks, vs], held, handle


def put(arrays, slots, x_bits, which):
    """What a write of x [T, heads, D] leaves in the numpy cache."""
    data, scales = arrays[which], arrays[which + 2]
    ps, room = data.shape[2], data.shape[0] * data.shape[2]
    for t, s in enumerate(slots):
        if 0 <= s < room:
            if scales is None:
                data[s // ps, :, s % ps] = x_bits[t]
            else:
                data[s // ps, :, s % ps], scales[s // ps, :, s % ps] = oa.quantize_cache(x_bits[t])


def same_cache(arrays, held):
    for a, g in zip(arrays, held):
        if a is not None:
            got = g.host()
            if a.dtype == np.uint8 and a.shape[-1] % 32 == 0:      # codes: either NaN is one
                nan = (a & 0x7F) == 0x7F
                assert np.array_equal(nan, (got & 0x7F) == 0x7F)
                assert np.array_equal(np.where(nan, 0, a), np.where(nan, 0, got))
            else:
                assert np.array_equal(a, got)


CACHES = [("bf16", 8, 1, 32), ("bf16", 16, 4, 96), ("bf16", 64, 2, 256), ("bf16", 4096, 1, 64),
          ("mxfp8", 8, 1, 32), ("mxfp8", 16, 8, 128), ("mxfp8", 32, 3, 96), ("mxfp8", 128, 2, 192),
          ("mxfp8", 16, 5, 64), ("mxfp8", 8, 1, 256), ("mxfp8", 16, 2, 160), ("mxfp8", 16, 2, 224)]


@pytest.mark.parametrize("fmt,ps,hkv,D", CACHES)
@pytest.mark.parametrize("T", [1, 29])
def test_cache_write_and_read(eg, fmt, ps, hkv, D, T):
    rng = np.random.default_rng(T * D + ps)
    pages = -(-T // ps) + 2
    arrays, held, handle = make_cache(eg, rng, fmt, pages, hkv, ps, D)
    room = pages * ps
    slots = rng.permutation(room)[:T].astype(np.int64)
    if T > 4:
        slots[[1, 3]] = [-1, room]
        slots[4] = -2 ** 40
    x = bits(rng.normal(size=(T, 2 * hkv * D + 24)) * 2.0 ** rng.integers(-20, 20, size=(T, 1)))
    x[0, 0] = 0x8000                                            # -0
    row = dev(x)
    kv = row[:, :2 * hkv * D].unflatten(1, (2 * hkv, D))
    xk, xv = x[:, :2 * hkv * D].reshape(T, 2 * hkv, D)[:, :hkv], x[:, :2 * hkv * D].reshape(T, 2 * hkv, D)[:, hkv:]
    bad = torch.zeros(1, dtype=torch.int32, device="cuda")
    eg.engram_cache_write(handle, kv[:, :hkv], kv[:, hkv:], dev(slots), bad)
    put(arrays, slots, xk, 0)
    put(arrays, slots, xv, 1)
    same_cache(arrays, held)
    assert bad.item() == (2 if T > 4 else 0)

    read = rng.integers(0, room, size=2 * T + 1).astype(np.int64)
    read[0] = slots[0]
    if T > 4:
        read[[2, 5, 6]] = [-1, room + 3, -9]
    n = len(read)
    k, v = Guarded((n, hkv, D), torch.int16), Guarded((n, hkv, D), torch.int16)
    eg.engram_cache_read(handle, dev(read), k.t, v.t, bad)
    for got, which in ((k, 0), (v, 1)):
        want = oa.cache_rows(arrays[which], arrays[which + 2], np.clip(read, 0, room - 1))
        want[(read < 0) | (read >= room)] = 0
        assert np.array_equal(got.host(), bits(want))
    assert bad.item() == (4 if T > 4 else 0)


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
def test_cache_write_with_head_strides(eg, fmt):
    """Heads outermost, and a gap after each head."""
    rng = np.random.default_rng(6)
    T, hkv, D = 11, 3, 64
    arrays, held, handle = make_cache(eg, rng, fmt, 3, hkv, 8, D)
    slots = rng.permutation(24)[:T].astype(np.int64)
    a, b = bits(rng.normal(size=(hkv, T, D + 8))), bits(rng.normal(size=(T, hkv, D + 40)))
    eg.engram_cache_write(handle, dev(a)[:, :, :D].transpose(0, 1), dev(b)[:, :, :D], dev(slots))
    put(arrays, slots, a[:, :, :D].transpose(1, 0, 2), 0)
    put(arrays, slots, b[:, :, :D], 1)
    same_cache(arrays, held)


def test_cache_8_bit_rounding_of_every_value(eg):
    """Every finite bf16 value next to several block maxima; infinities and NaN."""
    every = np.arange(1 << 16, dtype=np.uint32).astype(np.uint16)
    x = every.reshape(-1, 16).repeat(2, axis=1).reshape(-1, 32)[:, :32].copy()
    x[:, 16:] = 0
    tops = [0x0000, 0x0001, 0x007F, 0x0080, 0x1234, 0x3F80, 0x43E0, 0x43E1, 0x43DF, 0x7F7F, 0x7F60, 0x7F61]
    for top in tops:
        x[:, 20] = top
        T = x.shape[0]
        arrays, held, handle = make_cache(eg, np.random.default_rng(0), "mxfp8", T // 4096, 1, 4096, 32)
        slots = np.arange(T, dtype=np.int64)
        xs = dev(x.reshape(T, 1, 32))
        eg.engram_cache_write(handle, xs, xs, dev(slots))
        put_codes, put_scales = oa.quantize_cache(x)
        for w in (0, 1):
            arrays[w] = put_codes.reshape(arrays[w].shape)
            arrays[w + 2] = put_scales.reshape(arrays[w + 2].shape)
        same_cache(arrays, held)


def test_cache_8_bit_reading_of_every_value(eg):
    """Every code under every scale byte from 1 to 254."""
    codes = np.arange(256, dtype=np.uint8).reshape(8, 32)
    k = np.broadcast_to(codes, (256, 8, 32)).reshape(256, 1, 8, 32)[:254].copy()
    scales = np.broadcast_to(np.arange(1, 255, dtype=np.uint8)[:, None, None, None], (254, 1, 8, 1)).copy()
    handle = eg.KVCache(eg.ENGRAM_CACHE_MXFP8, dev(k), dev(k), dev(scales), dev(scales))
    n = 254 * 8
    out, v = Guarded((n, 1, 32), torch.int16), Guarded((n, 1, 32), torch.int16)
    eg.engram_cache_read(handle, dev(np.arange(n, dtype=np.int64)), out.t, v.t)
    want = bits(oa.cache_values(k, scales)).reshape(n, 1, 32)
    nan = np.isnan(oracle.bf16_value(want))
    for got in (out.host(), v.host()):
        assert np.array_equal(nan, np.isnan(oracle.bf16_value(got)))
        assert np.array_equal(want[~nan], got[~nan])


@pytest.mark.parametrize("fmt,ps,T,hq,hkv,D,rot,inter", [
    ("bf16", 8, 1, 4, 2, 64, 32, False), ("bf16", 16, 21, 5, 3, 96, 48, True), ("bf16", 32, 9, 2, 1, 256, 256, False),
    ("mxfp8", 16, 17, 12, 4, 64, 32, True), ("mxfp8", 8, 40, 32, 8, 128, 128, False),
    ("mxfp8", 64, 6, 3, 3, 192, 96, False), ("mxfp8", 16, 13, 4, 1, 160, 80, False), ("mxfp8", 8, 7, 1, 1, 32, 16, False),
    ("mxfp8", 8, 500, 4, 2, 96, 96, False)])
def test_qk_norm_rope_into_the_cache(eg, fmt, ps, T, hq, hkv, D, rot, inter):
    rng = np.random.default_rng(T)
    row, qkv, qw, kw, pos, inv = rope_inputs(rng, T, hq, hkv, D, rot, 8, 5000)
    pages = -(-T // ps) + 1
    arrays, held, handle = make_cache(eg, rng, fmt, pages, hkv, ps, D)
    slots = rng.permutation(pages * ps)[:T].astype(np.int64)
    if T > 5:
        slots[[0, 4]] = [pages * ps, -1]
    bad = torch.zeros(1, dtype=torch.int32, device="cuda")
    q, k = Guarded((T, hq, D), torch.int16), Guarded((T, hkv, D), torch.int16)
    args = (qkv, hq, hkv, D, dev(qw), dev(kw), 1e-6, dev(pos), dev(inv), inter)
    eg.engram_qk_norm_rope(*args, q.t, k.t, cache=handle, slots=dev(slots), bad_slots=bad)
    x = row[:, :(hq + 2 * hkv) * D].reshape(T, hq + 2 * hkv, D)
    want, mag = oa.qk_norm_rope(x[:, hq:hq + hkv], kw, 1e-6, pos, inv, inter)
    within(k.host(), want, H * np.abs(want) + 2.0 ** -20 * mag)
    put(arrays, slots, k.host(), 0)                            # what it put there is its own k, rounded
    put(arrays, slots, x[:, hq + hkv:], 1)
    same_cache(arrays, held)
    assert bad.item() == (1 if T > 5 else 0)
    # The queries are those of a call without a cache, and k may be left out.
    q2 = Guarded((T, hq, D), torch.int16)
    eg.engram_qk_norm_rope(*args, q2.t, k.t)
    assert np.array_equal(q.host(), q2.host())
    arrays2, held2, handle2 = make_cache(eg, np.random.default_rng(T), fmt, pages, hkv, ps, D)
    eg.engram_qk_norm_rope(*args, q2.t, cache=handle2, slots=dev(slots))
    put(arrays2, slots, k.host(), 0)
    put(arrays2, slots, x[:, hq + hkv:], 1)
    same_cache(arrays2, held2)


@pytest.mark.parametrize("fmt,ps,hkv,D", [("bf16", 16, 8, 128), ("mxfp8", 16, 8, 128), ("mxfp8", 32, 3, 96),
                                          ("mxfp8", 8, 5, 224), ("bf16", 64, 1, 32), ("mxfp8", 16, 7, 64)])
def test_cache_moves_of_many_tokens(eg, fmt, ps, hkv, D):
    """Enough tokens that a thread moves several pieces; slots that are not there among them."""
    rng = np.random.default_rng(D + hkv)
    T = 2048 * 256 // (2 * hkv * (D // 8)) + 77
    pages = -(-T // ps) + 1
    arrays, held, handle = make_cache(eg, rng, fmt, pages, hkv, ps, D)
    room = pages * ps
    slots = rng.permutation(room)[:T].astype(np.int64)
    slots[[2, T // 2, T - 1]] = [-1, room, -5]
    x = bits(rng.normal(size=(T, 2 * hkv, D)))
    bad = torch.zeros(1, dtype=torch.int32, device="cuda")
    row = dev(x)
    eg.engram_cache_write(handle, row[:, :hkv], row[:, hkv:], dev(slots), bad)
    # What it should hold, the oracle's rounding applied to all tokens at once.
    ok = (slots >= 0) & (slots < room)
    at = slots[ok]
    for w, part in ((0, x[:, :hkv]), (1, x[:, hkv:])):
        if fmt == "bf16":
            arrays[w][at // ps, :, at % ps] = part[ok]
        else:
            arrays[w][at // ps, :, at % ps], arrays[w + 2][at // ps, :, at % ps] = oa.quantize_cache(part[ok])
    same_cache(arrays, held)
    k, v = Guarded((T, hkv, D), torch.int16), Guarded((T, hkv, D), torch.int16)
    eg.engram_cache_read(handle, dev(slots), k.t, v.t, bad)
    for got, which in ((k, 0), (v, 1)):
        want = oa.cache_rows(arrays[which], arrays[which + 2], np.clip(slots, 0, room - 1))
        want[~ok] = 0
        assert np.array_equal(got.host(), bits(want))
    assert bad.item() == 4


@pytest.mark.parametrize("fmt,T,hq,hkv,D,rot,inter", [
    ("mxfp8", 1500, 32, 8, 128, 128, False), ("bf16", 1400, 13, 3, 96, 48, True), ("mxfp8", 700, 64, 8, 256, 128, False),
    ("mxfp8", 4100, 5, 2, 32, 32, True)])
def test_qk_norm_rope_of_many_tokens(eg, fmt, T, hq, hkv, D, rot, inter):
    """Enough tokens that a wave takes several of a token's passes, into the cache and without one."""
    rng = np.random.default_rng(T)
    row, qkv, qw, kw, pos, inv = rope_inputs(rng, T, hq, hkv, D, rot, 8, 5000)
    ps = 16
    pages = -(-T // ps) + 1
    arrays, held, handle = make_cache(eg, rng, fmt, pages, hkv, ps, D)
    slots = rng.permutation(pages * ps)[:T].astype(np.int64)
    slots[[0, 4]] = [pages * ps, -1]
    bad = torch.zeros(1, dtype=torch.int32, device="cuda")
    q, k = Guarded((T, hq, D), torch.int16), Guarded((T, hkv, D), torch.int16)
    q2, k2 = Guarded((T, hq, D), torch.int16), Guarded((T, hkv, D), torch.int16)
    args = (qkv, hq, hkv, D, dev(qw), dev(kw), 1e-6, dev(pos), dev(inv), inter)
    eg.engram_qk_norm_rope(*args, q.t, k.t, cache=handle, slots=dev(slots), bad_slots=bad)
    eg.engram_qk_norm_rope(*args, q2.t, k2.t)
    x = row[:, :(hq + 2 * hkv) * D].reshape(T, hq + 2 * hkv, D)
    for got, xs, w in ((q, x[:, :hq], qw), (k, x[:, hq:hq + hkv], kw)):
        want, mag = oa.qk_norm_rope(xs, w, 1e-6, pos, inv, inter)
        within(got.host(), want, H * np.abs(want) + 2.0 ** -20 * mag + 1e-38)
    assert np.array_equal(q.host(), q2.host()) and np.array_equal(k.host(), k2.host())
    put(arrays, slots, k.host(), 0)
    put(arrays, slots, x[:, hq + hkv:], 1)
    same_cache(arrays, held)
    assert bad.item() == 1


# ---------------------------------------------------------------- attention

def attend(eg, rng, fmt, ps, hq, hkv, D, lens, window=0, max_len=None, spoil=True, scale=None, sharp=2.0):
    """One call against the oracle; what no sequence sees holds NaN, table entries past the end are
    garbage.  Returns (out bits, lse)."""
    n = len(lens)
    lens = np.asarray(lens, np.int32)
    max_len = int(max(0, lens.max())) if max_len is None else max_len
    scale = 1 / np.sqrt(D) if scale is None else scale
    width = max(1, -(-max_len // ps))
    need = np.minimum(-(-np.maximum(lens, 0) // ps), width)
    pages = int(need.sum()) + 1
    arrays, held, handle = make_cache(eg, rng, fmt, pages, hkv, ps, D)
    perm = rng.permutation(pages)
    table = rng.integers(-2 ** 31, 2 ** 31 - 1, size=(n, width)).astype(np.int32)
    at, seen = 0, np.zeros((pages, ps), bool)
    for s in range(n):
        table[s, :need[s]] = perm[at:at + need[s]]
        at += need[s]
        length = min(max(int(lens[s]), 0), max_len, width * ps)
        p = np.arange(max(0, length - window) if window else 0, length)
        seen[table[s][p // ps], p % ps] = True
    if spoil:
        hide = np.broadcast_to(~seen[:, None, :, None], (pages, hkv, ps, D))
        for w in (0, 1):
            arrays[w][hide] = 0x7FC1 if fmt == "bf16" else 0x7F
            arrays[w][hide & (rng.random(hide.shape) < 0.3)] = 0x7F80 if fmt == "bf16" else 0xFF
            held[w].t.copy_(dev(arrays[w]))
            if fmt != "bf16":
                arrays[w + 2][np.broadcast_to(~seen[:, None, :, None], arrays[w + 2].shape)] = 255
                held[w + 2].t.copy_(dev(arrays[w + 2]))
    q = bits(sharp * rng.normal(size=(n, hq, D)))
    out, lse = Guarded((n, hq, D), torch.int16), Guarded((n, hq), torch.float32)
    ws = Guarded((eg.engram_paged_attention_workspace_bytes(n, hq, hkv, D, max_len),), torch.uint8)
    bad = torch.zeros(1, dtype=torch.int32, device="cuda")
    eg.engram_paged_attention(handle, dev(q), dev(table), dev(lens), max_len, scale, out.t, ws.t, window=window,
                              lse=lse.t, bad_pages=bad)
    ws.host()
    assert bad.item() == 0
    check_attention(out.host(), lse.host(), arrays, q, table, lens, max_len, scale, window)
    return out.host(), lse.host()


def check_attention(out, lse, arrays, q, table, lens, max_len, scale, window):
    D = q.shape[2]
    want, want_lse, spread, logit = oa.paged_attention(*arrays, q, table, lens, max_len, scale, window)
    d = D * U * logit
    within(out, want, H * np.abs(want) + (H + 2 * d + 2.0 ** -18)[..., None] * spread + 1e-30)
    empty = np.isneginf(want_lse)
    assert np.array_equal(empty, np.isneginf(lse))
    assert not out[empty].any()
    got, ref = lse[~empty].astype(np.float64), want_lse[~empty]
    tol = d[~empty] + (max(1, max_len) / 32 + 32) * U + 4 * U * np.abs(ref)
    assert np.all(np.abs(got - ref) <= tol), np.max(np.abs(got - ref) / tol)


ATTEND = [  # fmt, page size, q heads, kv heads, D, lengths, window
    ("bf16", 16, 32, 8, 128, [500], 0), ("bf16", 8, 1, 1, 32, [1], 0), ("bf16", 16, 4, 4, 64, [0, 1, 2, 31, 32, 33], 0),
    ("bf16", 64, 6, 2, 96, [63, 64, 65, 0, 200], 0), ("bf16", 32, 16, 1, 192, [700, 5], 0),
    ("bf16", 8, 32, 1, 256, [97, 300], 0), ("bf16", 128, 3, 1, 128, [129, 1000, 0], 0),
    ("bf16", 16, 40, 1, 64, [77, 260], 0), ("bf16", 16, 100, 2, 128, [45], 0), ("bf16", 16, 5, 5, 160, [70, 3], 0),
    ("bf16", 16, 7, 7, 224, [70, 130], 0), ("bf16", 4096, 2, 1, 64, [5000, 4096], 0),
    ("mxfp8", 16, 32, 8, 128, [500, 0, 37], 0), ("mxfp8", 8, 1, 1, 32, [1, 9], 0),
    ("mxfp8", 16, 12, 4, 64, [31, 32, 33, 240], 0), ("mxfp8", 32, 4, 2, 96, [64, 65, 333], 0),
    ("mxfp8", 64, 32, 1, 192, [50, 600], 0), ("mxfp8", 8, 24, 3, 256, [23, 300], 0),
    ("mxfp8", 128, 8, 8, 128, [1200, 128, 1], 0), ("mxfp8", 16, 6, 2, 160, [90], 0), ("mxfp8", 8, 9, 3, 224, [90], 0),
    ("bf16", 16, 8, 2, 128, [300, 10, 0, 64, 65], 64), ("bf16", 8, 8, 2, 64, [300, 10, 0, 64, 65], 1),
    ("mxfp8", 16, 8, 2, 128, [1000, 10, 0, 64, 65], 50), ("mxfp8", 32, 2, 1, 96, [777, 30], 333),
    ("bf16", 16, 16, 4, 128, [9000, 123, 4000], 0), ("mxfp8", 16, 8, 8, 128, [12345], 0),
    ("bf16", 16, 4, 2, 128, [20000, 19999], 7001), ("mxfp8", 16, 8, 2, 64, list(range(0, 130)), 0),
]


@pytest.mark.parametrize("fmt,ps,hq,hkv,D,lens,window", ATTEND)
def test_paged_attention(eg, fmt, ps, hq, hkv, D, lens, window):
    attend(eg, np.random.default_rng(D + len(lens)), fmt, ps, hq, hkv, D, lens, window)


def test_paged_attention_lengths_out_of_range(eg):
    """Lengths below 0, above max_len, above the table's places; max_len far above all; max_len 0."""
    rng = np.random.default_rng(11)
    attend(eg, rng, "bf16", 16, 4, 2, 64, [-5, 90, 64], max_len=64, spoil=False)
    attend(eg, rng, "mxfp8", 16, 4, 2, 64, [3, 70], max_len=100000)
    attend(eg, rng, "bf16", 16, 4, 2, 64, [3, 70], max_len=0, spoil=False)


def test_paged_attention_extreme_logits(eg):
    """Logits of some thousands: the running maximum keeps every exponential finite."""
    rng = np.random.default_rng(12)
    attend(eg, rng, "bf16", 16, 8, 2, 128, [700, 65], sharp=300.0)
    attend(eg, rng, "mxfp8", 16, 8, 2, 128, [700, 65], sharp=300.0)
    attend(eg, rng, "bf16", 16, 8, 2, 128, [700, 65], scale=-0.3)
    attend(eg, rng, "bf16", 16, 8, 2, 128, [700, 65], scale=0.0)


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
def test_paged_attention_bad_pages_are_not_seen(eg, fmt):
    rng = np.random.default_rng(13)
    ps, hq, hkv, D, pages = 16, 8, 2, 128, 9
    arrays, held, handle = make_cache(eg, rng, fmt, pages, hkv, ps, D)
    table = rng.integers(0, pages, size=(4, 20)).astype(np.int32)
    table[0, 3], table[0, 7], table[1, 0] = -1, pages, 2 ** 31 - 1
    table[2, :] = -2 ** 31                                     # nothing left to see
    lens = np.array([300, 16, 320, 250], np.int32)
    q = bits(rng.normal(size=(4, hq, D)))
    out, lse = Guarded((4, hq, D), torch.int16), Guarded((4, hq), torch.float32)
    ws = torch.empty(eg.engram_paged_attention_workspace_bytes(4, hq, hkv, D, 320), dtype=torch.uint8, device="cuda")
    bad = torch.zeros(1, dtype=torch.int32, device="cuda")
    eg.engram_paged_attention(handle, dev(q), dev(table), dev(lens), 320, 0.1, out.t, ws, lse=lse.t, bad_pages=bad)
    assert bad.item() > 0
    check_attention(out.host(), lse.host(), arrays, q, table, lens, 320, 0.1, 0)
    assert np.isneginf(lse.host()[1:3]).all() and not out.host()[1:3].any()


def test_paged_attention_is_the_same_every_time_and_needs_no_lse(eg):
    rng = np.random.default_rng(14)
    ps, hq, hkv, D, pages = 16, 8, 2, 128, 600
    arrays, held, handle = make_cache(eg, rng, "bf16", pages, hkv, ps, D)
    table = dev(rng.permutation(pages)[None].astype(np.int32))
    lens, q = dev(np.array([pages * ps - 3], np.int32)), dev(bits(rng.normal(size=(1, hq, D))))
    outs = []
    for i in range(4):
        out = torch.empty(1, hq, D, dtype=torch.int16, device="cuda")
        ws = torch.full((eg.engram_paged_attention_workspace_bytes(1, hq, hkv, D, pages * ps),), 255 * (i % 2),
                        dtype=torch.uint8, device="cuda")
        eg.engram_paged_attention(handle, q, table, lens, pages * ps, 0.1, out, ws)
        outs.append(host(out))
    assert all(np.array_equal(outs[0], o) for o in outs[1:])


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
def test_cache_beyond_32_bit_offsets(eg, fmt):
    """Keys and values past 4 GiB (and past 2^32 values' scales) of the cache."""
    rng = np.random.default_rng(15)
    ps, hq, hkv, D = 4096, 4, 1, 256
    pages = 2200 if fmt == "bf16" else 4300                     # 4.6 GB, 4.5 GB each of keys and values
    shape = (pages, hkv, ps, D)
    data = [torch.empty(shape, dtype=torch.int16 if fmt == "bf16" else torch.uint8, device="cuda") for _ in range(2)]
    scales = [None] * 2 if fmt == "bf16" else [torch.empty(shape[:3] + (D // 32,), dtype=torch.uint8, device="cuda")
                                               for _ in range(2)]
    handle = eg.KVCache(eg.ENGRAM_CACHE_BF16 if fmt == "bf16" else eg.ENGRAM_CACHE_MXFP8, *data, *scales)
    lens = np.array([200, 130], np.int32)
    table = np.array([[pages - 1], [pages - 2]], np.int32)
    T = int(lens.sum())
    slots = np.concatenate([int(table[s, 0]) * ps + np.arange(lens[s]) for s in range(2)]).astype(np.int64)
    k, v = bits(rng.normal(size=(T, hkv, D))), bits(rng.normal(size=(T, hkv, D)))
    eg.engram_cache_write(handle, dev(k), dev(v), dev(slots))
    ko, vo = Guarded((T, hkv, D), torch.int16), Guarded((T, hkv, D), torch.int16)
    eg.engram_cache_read(handle, dev(slots), ko.t, vo.t)
    # A small cache that holds the same, for the oracle.
    small = [np.zeros((2, hkv, ps, D), np.uint16 if fmt == "bf16" else np.uint8) for _ in range(2)]
    small += [None] * 2 if fmt == "bf16" else [np.zeros((2, hkv, ps, D // 32), np.uint8) for _ in range(2)]
    at = np.concatenate([s * ps + np.arange(lens[s]) for s in range(2)])
    put(small, at, k, 0)
    put(small, at, v, 1)
    assert np.array_equal(ko.host(), bits(oa.cache_rows(small[0], small[2], at)))
    assert np.array_equal(vo.host(), bits(oa.cache_rows(small[1], small[3], at)))
    q = bits(rng.normal(size=(2, hq, D)))
    out, lse = Guarded((2, hq, D), torch.int16), Guarded((2, hq), torch.float32)
    ws = torch.empty(eg.engram_paged_attention_workspace_bytes(2, hq, hkv, D, 200), dtype=torch.uint8, device="cuda")
    eg.engram_paged_attention(handle, dev(q), dev(table), dev(lens), 200, 0.0625, out.t, ws, lse=lse.t)
    check_attention(out.host(), lse.host(), small, q, np.array([[0], [1]], np.int32), lens, 200, 0.0625, 0)


def test_paged_attention_more_sequences_than_threads(eg):
    """Many short sequences, empty ones among them, in equal runs that cut most of them."""
    rng = np.random.default_rng(40)
    lens = rng.integers(0, 700, size=700)
    lens[rng.random(700) < 0.2] = 0
    lens[[0, 1, -1]] = [0, 0, 0]
    attend(eg, rng, "mxfp8", 8, 3, 1, 32, lens, max_len=1100)


def test_paged_attention_one_long_among_short(eg):
    rng = np.random.default_rng(41)
    attend(eg, rng, "bf16", 16, 8, 2, 64, [3, 0, 20000, 1, 500, 129])
    attend(eg, rng, "mxfp8", 32, 12, 3, 96, [1, 9000, 0, 4097, 128], window=4500)


def test_paged_attention_many_head_blocks(eg):
    """More query heads a key-value head than a workgroup takes, split over the length."""
    attend(eg, np.random.default_rng(42), "bf16", 16, 70, 1, 64, [2000, 17, 0, 900])
    attend(eg, np.random.default_rng(43), "mxfp8", 16, 66, 2, 192, [1500, 800])
    attend(eg, np.random.default_rng(44), "bf16", 64, 33, 1, 256, [1500, 64])


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
def test_paged_attention_long_runs_of_shared_pages(eg, fmt):
    """Runs longer than the pages held at a time; pages shared by all sequences."""
    rng = np.random.default_rng(45)
    n, ps, hq, D, pages = 40, 8, 2, 32, 50
    arrays, held, handle = make_cache(eg, rng, fmt, pages, 1, ps, D)
    lens = rng.integers(28000, 32000, size=n).astype(np.int32)
    lens[5] = 0
    table = rng.integers(0, pages, size=(n, 32000 // ps)).astype(np.int32)
    q = bits(2.0 * rng.normal(size=(n, hq, D)))
    out, lse = Guarded((n, hq, D), torch.int16), Guarded((n, hq), torch.float32)
    ws = Guarded((eg.engram_paged_attention_workspace_bytes(n, hq, 1, D, 32000),), torch.uint8)
    eg.engram_paged_attention(handle, dev(q), dev(table), dev(lens), 32000, 0.2, out.t, ws.t, lse=lse.t)
    ws.host()
    check_attention(out.host(), lse.host(), arrays, q, table, lens, 32000, 0.2, 0)


# ---------------------------------------------------------------- the 4-bit weight

def test_quantize_mxfp4(eg):
    rng = np.random.default_rng(20)
    w = rng.normal(size=(33, 96)) * 2.0 ** rng.integers(-30, 30, size=(33, 1))
    w[0, :32] = 0
    w[1, :16] = [0, 0.25, 0.5, 0.75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, 7]
    w[2, :16] = -w[1, :16]
    w[3] = 1e-39
    w[4] = 3e38
    wb = bits(w)
    codes, scales = Guarded((33, 48), torch.uint8), Guarded((33, 3), torch.uint8)
    eg.engram_quantize_mxfp4(dev(wb), 33, 96, codes.t, scales.t)
    want_codes, want_scales = oa.quantize_mxfp4(wb)
    assert np.array_equal(scales.host(), want_scales)
    assert np.array_equal(codes.host(), want_codes)


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 33, 64, 65, 101, 128, 129, 300])
@pytest.mark.parametrize("K,N", [(32, 1), (96, 67), (128, 64), (160, 16), (1056, 130), (4096, 48), (6144, 33)])
def test_project_mxfp4(eg, T, K, N):
    rng = np.random.default_rng(T + K)
    x = bits(rng.normal(size=(T, K)))
    codes = rng.integers(0, 256, size=(N, K // 2), dtype=np.uint8)
    scales = rng.integers(110, 130, size=(N, K // 32), dtype=np.uint8)
    out = Guarded((T, N), torch.int16)
    eg.engram_project_mxfp4(dev(x), dev(codes), dev(scales), out.t, T, K, N)
    want, mag = oa.project_mxfp4(x, codes, scales)
    within(out.host(), want, H * np.abs(want) + K * U * mag)


def test_project_mxfp4_many_columns_odd_scales(eg):
    """More column tiles than compute units; scales at an odd address; the smallest and largest scales."""
    rng = np.random.default_rng(21)
    T, K, N = 3, 64, 9001
    x = bits(rng.normal(size=(T, K)))
    codes = rng.integers(0, 256, size=(N, K // 2), dtype=np.uint8)
    scales = rng.choice(np.array([0, 1, 2, 60, 127, 200, 240], np.uint8), size=(N, K // 32))
    room = torch.empty(scales.size + 1, dtype=torch.uint8, device="cuda")
    room[1:] = dev(scales).flatten()
    out = Guarded((T, N), torch.int16)
    eg.engram_project_mxfp4(dev(x), dev(codes), room[1:], out.t, T, K, N)
    want, mag = oa.project_mxfp4(x, codes, scales)
    within(out.host(), want, H * np.abs(want) + K * U * mag + 2.0 ** -133)


@pytest.mark.parametrize("K,N,shift", [(16640, 37, 0), (16640, 20, 1), (8224, 21, 0), (8320, 4, 2), (24608, 130, 3)])
@pytest.mark.parametrize("T", [5, 70])
def test_project_mxfp4_long_rows(eg, K, N, shift, T):
    """Rows of more scales than are held at a time; scales at any address."""
    rng = np.random.default_rng(K + T)
    x = bits(rng.normal(size=(T, K)))
    codes = rng.integers(0, 256, size=(N, K // 2), dtype=np.uint8)
    scales = rng.integers(110, 130, size=(N, K // 32), dtype=np.uint8)
    room = torch.empty(scales.size + shift, dtype=torch.uint8, device="cuda")
    room[shift:] = dev(scales).flatten()
    out = Guarded((T, N), torch.int16)
    eg.engram_project_mxfp4(dev(x), dev(codes), room[shift:], out.t, T, K, N)
    want, mag = oa.project_mxfp4(x, codes, scales)
    within(out.host(), want, H * np.abs(want) + K * U * mag)


def test_project_mxfp4_infinity_and_nan_stay_in_their_token(eg):
    """K that ends inside a step of 128: an infinity of one token reaches no other."""
    rng = np.random.default_rng(50)
    T, K, N = 20, 160, 48
    x = bits(rng.normal(size=(T, K)))
    codes = rng.integers(0, 256, size=(N, K // 2), dtype=np.uint8)
    scales = rng.integers(120, 130, size=(N, K // 32), dtype=np.uint8)
    y = x.copy()
    y[3, :] = 0x7F80
    y[11, 0] = 0x7FC1
    out, ref = Guarded((T, N), torch.int16), Guarded((T, N), torch.int16)
    eg.engram_project_mxfp4(dev(x), dev(codes), dev(scales), ref.t, T, K, N)
    eg.engram_project_mxfp4(dev(y), dev(codes), dev(scales), out.t, T, K, N)
    others = np.setdiff1d(np.arange(T), [3, 11])
    assert np.array_equal(out.host()[others], ref.host()[others])
    assert not np.isfinite(oracle.bf16_value(out.host()[[3, 11]])).any()


# ---------------------------------------------------------------- all of it together

def step_state(eg, seed=30):
    """A decode step of three streams: projection, norm and rotation into the cache, attention, projection."""
    rng = np.random.default_rng(seed)
    n, hq, hkv, D, rot, ps, dim = 3, 8, 2, 64, 64, 16, 256
    width = (hq + 2 * hkv) * D
    s = dict(n=n, hq=hq, hkv=hkv, D=D, dim=dim, width=width)
    for name, (N, K) in dict(wqkv=(width, dim), wo=(dim, hq * D)).items():
        w = bits(rng.normal(size=(N, K)) / np.sqrt(K))
        s[name] = (torch.empty(N, K // 2, dtype=torch.uint8, device="cuda"),
                   torch.empty(N, K // 32, dtype=torch.uint8, device="cuda"))
        eg.engram_quantize_mxfp4(dev(w), N, K, *s[name])
    lens = np.array([41, 1, 17], np.int32)
    s["arrays"], s["held"], s["cache"] = make_cache(eg, rng, "mxfp8", 8, hkv, ps, D)
    table = np.array([[5, 2, 7], [0, -1, -1], [4, 3, -1]], np.int32)
    slots = np.array([table[i, (l - 1) // ps] * ps + (l - 1) % ps for i, l in enumerate(lens)], np.int64)
    s.update(x=dev(bits(rng.normal(size=(n, dim)))), table=dev(table), lens=dev(lens), slots=dev(slots),
             pos=dev(lens - 1), inv=dev(10000.0 ** (-2.0 * np.arange(rot // 2) / rot)),
             qw=dev(bits(np.ones(D))), kw=dev(bits(np.ones(D))),
             qkv=torch.empty(n, width, dtype=torch.int16, device="cuda"),
             q=torch.empty(n, hq, D, dtype=torch.int16, device="cuda"),
             att=torch.empty(n, hq, D, dtype=torch.int16, device="cuda"),
             y=torch.empty(n, dim, dtype=torch.int16, device="cuda"),
             ws=torch.empty(eg.engram_paged_attention_workspace_bytes(n, hq, hkv, D, 48), dtype=torch.uint8,
                            device="cuda"))
    return s


def step(eg, s, stream=None):
    eg.engram_project_mxfp4(s["x"], *s["wqkv"], s["qkv"], s["n"], s["dim"], s["width"], stream=stream)
    eg.engram_qk_norm_rope(s["qkv"], s["hq"], s["hkv"], s["D"], s["qw"], s["kw"], 1e-6, s["pos"], s["inv"], False,
                           s["q"], cache=s["cache"], slots=s["slots"], stream=stream)
    eg.engram_paged_attention(s["cache"], s["q"], s["table"], s["lens"], 48, 0.125, s["att"], s["ws"], stream=stream)
    eg.engram_project_mxfp4(s["att"], *s["wo"], s["y"], s["n"], s["hq"] * s["D"], s["dim"], stream=stream)


def test_step_against_the_oracle(eg):
    """Each operator of the step on what the one before it gave."""
    s = step_state(eg)
    step(eg, s)
    x, qkv, q, att, y = (host(s[m]) for m in ("x", "qkv", "q", "att", "y"))
    want, mag = oa.project_mxfp4(x, *(host(t) for t in s["wqkv"]))
    within(qkv, want, H * np.abs(want) + s["dim"] * U * mag)
    heads = qkv.reshape(s["n"], -1, s["D"])
    want, mag = oa.qk_norm_rope(heads[:, :s["hq"]], host(s["qw"]), 1e-6, host(s["pos"]), host(s["inv"]), False)
    within(q, want, H * np.abs(want) + 2.0 ** -20 * mag)
    held = [g.host() for g in s["held"]]
    lse = oa.paged_attention(*held, q, host(s["table"]), host(s["lens"]), 48, 0.125)[1].astype(np.float32)
    check_attention(att, lse, held, q, host(s["table"]), host(s["lens"]), 48, 0.125, 0)
    want, mag = oa.project_mxfp4(att.reshape(s["n"], -1), *(host(t) for t in s["wo"]))
    within(y, want, H * np.abs(want) + s["hq"] * s["D"] * U * mag)


def test_step_on_another_stream_and_in_a_graph(eg):
    s = step_state(eg)
    step(eg, s)
    torch.cuda.synchronize()
    want = host(s["y"])
    side = torch.cuda.Stream()
    s["y"].zero_()
    side.wait_stream(torch.cuda.current_stream())
    step(eg, s, stream=side)
    side.synchronize()
    assert np.array_equal(want, host(s["y"]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(eg, s)
    inputs = [host(s["x"])] + [bits(np.random.default_rng(i).normal(size=(s["n"], s["dim"]))) for i in (1, 2)]
    for x in inputs + inputs:
        s["x"].copy_(dev(x))
        step(eg, s)
        torch.cuda.synchronize()
        eager = host(s["y"])
        s["y"].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(eager, host(s["y"]))


@pytest.mark.parametrize("kind", ["bf16", "mxfp8"])
def test_example_of_a_prompt_and_decode_steps(eg, kind):
    """Relative to the largest value: the weights' and the result's rounding, H each."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "attention_step.py")
    spec = importlib.util.spec_from_file_location("attention_step", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    worst, bad, lens = mod.run(3, kind, verbose=False)
    assert bad == 0 and lens == [p + 3 for p in mod.PROMPTS]
    assert worst <= 4 * H


def test_empty_inputs(eg):
    z = lambda *shape, dtype=torch.int16: torch.zeros(*shape, dtype=dtype, device="cuda")  # noqa: E731
    cache = eg.KVCache(eg.ENGRAM_CACHE_BF16, z(1, 1, 8, 32), z(1, 1, 8, 32))
    eg.engram_cache_write(cache, z(0, 1, 32), z(0, 1, 32), z(0, dtype=torch.int64))
    eg.engram_cache_read(cache, z(0, dtype=torch.int64), z(0, 1, 32), z(0, 1, 32))
    eg.engram_qk_norm_rope(z(0, 96), 1, 1, 32, z(32), z(32), 1e-6, z(0, dtype=torch.int32),
                           z(8, dtype=torch.float64), False, z(0, 1, 32), z(0, 1, 32))
    eg.engram_paged_attention(cache, z(0, 1, 32), z(0, 4, dtype=torch.int32), z(0, dtype=torch.int32), 0, 1.0,
                              z(0, 1, 32), z(0, dtype=torch.uint8))
    eg.engram_project_mxfp4(z(0, 64), z(5, 32, dtype=torch.uint8), z(5, 2, dtype=torch.uint8), z(0, 5), 0, 64, 5)


def test_binding_refuses(eg):
    z = lambda *shape, dtype=torch.int16: torch.zeros(*shape, dtype=dtype, device="cuda")  # noqa: E731
    i64, i32, u8 = torch.int64, torch.int32, torch.uint8
    cache = eg.KVCache(eg.ENGRAM_CACHE_BF16, z(2, 2, 8, 64), z(2, 2, 8, 64))
    with pytest.raises(ValueError, match="must be"):
        eg.engram_cache_write(cache, z(3, 2, 64), z(3, 1, 64), z(3, dtype=i64))
    with pytest.raises(ValueError, match="contiguous"):
        eg.engram_cache_write(cache, z(3, 2, 128)[:, :, ::2], z(3, 2, 64), z(3, dtype=i64))
    with pytest.raises(eg.EngramError, match="stride"):
        eg.engram_cache_write(cache, z(3, 2 * 64 + 4)[:, :128].unflatten(1, (2, 64)), z(3, 2, 64), z(3, dtype=i64))
    with pytest.raises(TypeError, match="slots"):
        eg.engram_cache_write(cache, z(3, 2, 64), z(3, 2, 64), z(3, dtype=i32))
    with pytest.raises(ValueError, match="elements"):
        eg.engram_cache_read(cache, z(3, dtype=i64), z(2, 2, 64), z(3, 2, 64))
    rope = lambda qkv, **kw: eg.engram_qk_norm_rope(  # noqa: E731
        qkv, 4, 2, 64, z(64), z(64), 1e-6, z(3, dtype=i32), z(16, dtype=torch.float64), False, z(3, 4, 64), **kw)
    with pytest.raises(ValueError, match="rows of"):
        rope(z(3, 376), k=z(3, 2, 64))
    with pytest.raises(ValueError, match="rows of"):
        rope(z(3, 384), cache=cache, slots=z(3, dtype=i64))
    with pytest.raises(eg.EngramError, match="keys need"):
        rope(z(3, 512))
    with pytest.raises(eg.EngramError, match="slots"):
        rope(z(3, 512), cache=cache)
    with pytest.raises(TypeError, match="GPU"):
        rope(torch.zeros(3, 512, dtype=torch.int16), k=z(3, 2, 64))
    with pytest.raises(ValueError, match="q must be"):
        eg.engram_paged_attention(cache, z(1, 4, 32), z(1, 2, dtype=i32), z(1, dtype=i32), 9, 1.0, z(1, 4, 32))
    with pytest.raises(ValueError, match="table"):
        eg.engram_paged_attention(cache, z(1, 4, 64), z(2, 2, dtype=i32), z(1, dtype=i32), 9, 1.0, z(1, 4, 64))
    with pytest.raises(eg.EngramError, match="multiple of kv_heads"):
        eg.engram_paged_attention(cache, z(1, 3, 64), z(1, 2, dtype=i32), z(1, dtype=i32), 9, 1.0, z(1, 3, 64))
    with pytest.raises(ValueError, match="elements"):
        eg.engram_project_mxfp4(z(2, 64), z(5, 31, dtype=u8), z(5, 2, dtype=u8), z(2, 5), 2, 64, 5)
