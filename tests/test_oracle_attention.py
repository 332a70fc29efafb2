"""Pins of oracle/attention.py (CPU): against torch's formats, closed forms and hand-worked values."""

import numpy as np
import pytest
import torch

import oracle
from oracle import attention as oa


def bits(x):
    return oracle.bf16_bits(oracle.bf16_round(np.asarray(x, np.float64)))


def test_rotation_is_a_rotation():
    """Pairs keep their length, position 0 turns nothing, a quarter turn maps (a, b) to (-b, a)."""
    rng = np.random.default_rng(1)
    x, w = bits(rng.normal(size=(3, 2, 64))), bits(np.ones(64))
    plain, _ = oa.qk_norm_rope(x, w, 0.0, [0, 0, 0], [0.3, 0.1], False)
    assert np.allclose(np.mean(plain ** 2, -1), 1.0)
    for inter in (False, True):
        i = np.arange(16)
        ia, ib = (2 * i, 2 * i + 1) if inter else (i, i + 16)
        got, _ = oa.qk_norm_rope(x, w, 0.0, [0, 1, 100003], [np.pi / 2] * 16, inter)
        assert np.array_equal(got[0], plain[0])
        assert np.allclose(got[1][:, ia], -plain[1][:, ib]) and np.allclose(got[1][:, ib], plain[1][:, ia])
        assert np.allclose(got[2][:, ia] ** 2 + got[2][:, ib] ** 2,
                           plain[2][:, ia] ** 2 + plain[2][:, ib] ** 2)
        assert np.array_equal(got[:, :, 32:], plain[:, :, 32:])


def test_cache_format_scale_rule_and_codes_against_torch():
    rng = np.random.default_rng(2)
    x = bits(rng.normal(size=(500, 96)) * 2.0 ** rng.integers(-60, 60, size=(500, 1)))
    codes, scales = oa.quantize_cache(x)
    v = oracle.bf16_value(x).reshape(500, 3, 32)
    amax, unit = np.abs(v).max(-1), np.ldexp(1.0, scales.astype(int) - 127)
    assert np.all(amax <= 448 * unit) and np.all(amax > 224 * unit)      # the smallest that holds
    want = torch.from_numpy((v / unit[..., None]).astype(np.float32)).to(torch.float8_e4m3fn)
    assert np.array_equal(codes.reshape(500, 3, 32), want.view(torch.uint8).numpy())


def test_cache_format_borders():
    x = np.zeros((6, 32))
    x[1, 0], x[2, 0], x[3, 0], x[4, 5] = 448.0, 450.0, 1e-38, np.inf
    x[4, 6], x[5, 0], x[5, 1] = -3.0, np.nan, 224.0
    codes, scales = oa.quantize_cache(bits(x))
    assert scales[:, 0].tolist() == [127, 127, 128, 32, 120, 126]
    assert codes[1, 0] == 0x7E and codes[2, 0] == 0x76 and not codes[0].any()
    # 3 / 2^-7 = 384 = 1.5 * 2^8 (768 would be too much): exponent field 15, fraction 4
    assert codes[4, 5] & 0x7F == 0x7F and codes[4, 6] == 0x80 | 15 << 3 | 4
    assert codes[5, 0] & 0x7F == 0x7F and codes[5, 1] == 0x7E


def test_attention_closed_forms():
    """Equal keys give the mean of the values; a window's out is that of the places it leaves;
    bad pages and empty sequences drop out."""
    rng = np.random.default_rng(3)
    pages, ps, D = 5, 8, 32
    k = np.broadcast_to(bits(rng.normal(size=D)), (pages, 1, ps, D)).copy()
    v = bits(rng.normal(size=(pages, 1, ps, D)))
    q = bits(rng.normal(size=(4, 2, D)))
    table = np.array([[3, 1, -1], [4, 0, -1], [2, -1, 0], [0, 1, 2]], np.int32)
    lens = [13, 16, 24, 0]
    out, lse, _, _ = oa.paged_attention(k, v, None, None, q, table, lens, 24, 0.25)
    vv = oracle.bf16_value(v)
    first = np.concatenate([vv[3, 0], vv[1, 0, :5]])
    assert np.allclose(out[0], first.mean(0))
    z = 0.25 * (oracle.bf16_value(q[0]) @ oracle.bf16_value(k[0, 0, 0]))
    assert np.allclose(lse[0], z + np.log(13))
    assert np.allclose(out[2], np.concatenate([vv[2, 0], vv[0, 0]]).mean(0))
    assert not out[3].any() and np.all(np.isneginf(lse[3]))
    out, _, _, _ = oa.paged_attention(k, v, None, None, q, table, lens, 24, 0.25, window=6)
    assert np.allclose(out[0], first[-6:].mean(0))


def test_mxfp4_hand_worked():
    w = np.zeros((2, 32))
    w[0, :8] = [6.0, -0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]             # scale 2^0; ties to even
    codes, scales = oa.quantize_mxfp4(bits(w))
    assert scales[:, 0].tolist() == [127, 127]
    assert [codes[0, 0] & 15, codes[0, 0] >> 4, codes[0, 1] & 15, codes[0, 1] >> 4,
            codes[0, 2] & 15, codes[0, 2] >> 4, codes[0, 3] & 15, codes[0, 3] >> 4] == [7, 8, 2, 2, 4, 4, 6, 6]
    assert oa.mxfp4_values(codes, scales)[0, :8].tolist() == [6, 0, 1, 1, 2, 2, 4, 4]
    # 7.9 has the exponent of 4, so the scale stays 1 and the code saturates.
    w[1, 3] = 7.875
    codes, scales = oa.quantize_mxfp4(bits(w))
    assert oa.mxfp4_values(codes, scales)[1, 3] == 6.0


@pytest.mark.parametrize("seed", [0, 1])
def test_mxfp4_values_survive_their_own_quantisation(seed):
    rng = np.random.default_rng(seed)
    codes = rng.integers(0, 256, size=(7, 48), dtype=np.uint8)
    codes[:, ::16] |= 0x07                            # a 6 in every block
    scales = rng.integers(30, 200, size=(7, 3), dtype=np.uint8)
    v = oa.mxfp4_values(codes, scales)
    again = oa.mxfp4_values(*oa.quantize_mxfp4(bits(v)))
    assert np.array_equal(v, again)
