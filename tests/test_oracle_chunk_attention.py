"""Pins of the oracle's attention of chunks and shared prefixes, places' weights and eviction (CPU)."""

import numpy as np
import pytest
import torch

import oracle
from oracle import attention as oa


def bits(x):
    return oracle.bf16_bits(oracle.bf16_round(np.asarray(x, np.float64)))


def world(rng, hkv=2, ps=8, D=32, pages=12):
    k, v = (bits(rng.normal(size=(pages, hkv, ps, D))) for _ in range(2))
    return k, v, None, None


def test_single_tokens_are_paged_attention():
    rng = np.random.default_rng(0)
    cache = world(rng)
    table = rng.permutation(12).reshape(3, 4).astype(np.int32)
    lens, q = np.array([30, 1, 17]), bits(rng.normal(size=(3, 4, 32)))
    for window in (0, 5):
        want = oa.paged_attention(*cache, q, table, lens, 32, 0.2, window)
        got = oa.chunk_attention(cache, q, np.arange(4), table, lens, 32, 0.2, oa.rules_of(window=window))
        assert np.allclose(got[0], want[0], rtol=1e-12) and np.allclose(got[1], want[1], rtol=1e-12)
        assert np.allclose(got[2], want[2], rtol=1e-12)


def test_a_chunk_is_its_tokens_one_by_one():
    rng = np.random.default_rng(1)
    cache = world(rng)
    table, q = rng.permutation(12)[None].astype(np.int32), bits(rng.normal(size=(9, 4, 32)))
    got = oa.chunk_attention(cache, q, [0, 9], table, [20], 32, 0.2)
    for i in range(9):
        one = oa.chunk_attention(cache, q[i:i + 1], [0, 1], table, [12 + i], 32, 0.2)
        assert np.allclose(got[0][i], one[0][0], rtol=1e-12) and np.allclose(got[1][i], one[1][0], rtol=1e-12)


def test_rules_by_a_dense_mask():
    """Against torch's softmax in float64 over an explicit mask and bias."""
    rng = np.random.default_rng(2)
    cache = world(rng)
    table, n, length = rng.permutation(12)[None].astype(np.int32), 20, 40
    q = bits(rng.normal(size=(n, 2, 32)))
    starts = np.array([0] * 5 + [25] * 5 + [33] * 9 + [99], np.int32)
    rules = oa.rules_of(window=7, cap=1.5, slopes=np.array([0.5, 0.1]), doc_starts=starts, prefix_lens=np.array([27]))
    out, lse, *_ = oa.chunk_attention(cache, q, [0, n], table, [length], 64, 0.3, rules)
    k, v, _ = oa._places(cache, table[0], length)
    qf = torch.from_numpy(oracle.bf16_value(q))
    for h in range(2):
        z = 1.5 * torch.tanh(qf[:, h] @ torch.from_numpy(k[h].T.copy()) * 0.3 / 1.5)
        for i in range(n):
            pos = length - n + i
            for p in range(length):
                z[i, p] -= rules["slopes"][h] * abs(pos - p)
                inside = pos - 7 < p <= pos or p < 27
                if not inside or p < starts[i]:
                    z[i, p] = -np.inf
        some = torch.isfinite(z).any(1)
        empty = starts > np.arange(length - n, length)            # a document that begins behind its token
        assert np.array_equal(some.numpy(), ~empty) and empty[[10, 19]].all()
        assert np.isneginf(lse[empty]).all() and not out[empty].any()
        want = torch.softmax(z[some], 1) @ torch.from_numpy(v[h].copy())
        assert np.allclose(out[~empty, h], want, rtol=1e-10, atol=1e-12)
        assert np.allclose(lse[~empty, h], torch.logsumexp(z[some], 1), rtol=1e-10)


def test_a_value_that_is_not_finite_reaches_its_rows_and_dimension():
    rng = np.random.default_rng(3)
    cache = world(rng)
    table, q = rng.permutation(12)[None].astype(np.int32), bits(rng.normal(size=(4, 2, 32)))
    before = oa.chunk_attention(cache, q, [0, 4], table, [30], 32, 0.2)[0]
    cache[1][table[0, 28 // 8], 1, 28 % 8, 3] = 0x7FC1
    after = oa.chunk_attention(cache, q, [0, 4], table, [30], 32, 0.2)[0]
    hit = np.isnan(after)
    assert hit[2:, 1, 3].all() and hit.sum() == 2
    assert np.array_equal(after[~hit], before[~hit])


def test_shared_prefix_is_attention_over_joined_places():
    rng = np.random.default_rng(4)
    cache = world(rng)
    perm = rng.permutation(12).astype(np.int32)
    q = bits(rng.normal(size=(3, 4, 32)))
    prefix, own = perm[None, :2], perm[2:8].reshape(3, 2)
    got = oa.shared_prefix_attention(cache, q, [0, 2], prefix, [16], 99, own, [5, 0, 9], 99, 0.2)
    joined = np.concatenate([np.repeat(prefix, 3, 0), own], 1)
    want = oa.chunk_attention(cache, q, np.arange(4), joined, [21, 16, 0], 99, 0.2)
    alone = oa.chunk_attention(cache, q, np.arange(4), own, [0, 0, 9], 99, 0.2)
    assert np.allclose(got[0][:2], want[0][:2], rtol=1e-12) and np.allclose(got[0][2], alone[0][2], rtol=1e-12)
    assert np.allclose(got[1][:2], want[1][:2], rtol=1e-12)


def test_weights_sum_to_one_a_row():
    rng = np.random.default_rng(5)
    cache = world(rng)
    table, q = rng.permutation(12)[None].astype(np.int32), bits(rng.normal(size=(6, 4, 32)))
    lse = oa.chunk_attention(cache, q, [0, 6], table, [33], 64, 0.2)[1]
    lse[2] = -np.inf
    w, slack = oa.cache_weights(cache, q, [0, 6], table, [33], 64, 0.2, lse, 40)
    assert np.isclose(w.sum(), 5 * 4) and not w[..., 33:].any() and (slack >= 0).all()
    assert w[0, 0, 32] > 0 and np.isclose(w[0].sum(1), 10).all()


@pytest.mark.parametrize("sinks,recent", [(0, 0), (1, 0), (0, 2), (2, 3)])
def test_evict_by_hand(sinks, recent):
    w = np.array([[[1, 5, 5, 0, np.nan, 5, 2, 0, 9, 0]]], np.float32)
    got = oa.evict(w, [10], 10, 99, 5, sinks, recent)[0, 0].tolist()
    assert got == {(0, 0): [1, 2, 5, 6, 8], (1, 0): [0, 1, 2, 5, 8], (0, 2): [1, 2, 5, 8, 9], (2, 3): [0, 1, 7, 8, 9]}[sinks, recent]
    assert oa.evict(w, [3], 10, 99, 5, 0, 0)[0, 0].tolist() == [0, 1, 2, -1, -1]
