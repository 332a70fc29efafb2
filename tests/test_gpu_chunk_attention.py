"""Attention of several new tokens, over shared prefixes, places' weights and eviction, on the GPU, against
oracle/attention.py (float64).

Tolerances, from the number of roundings (u = 2^-24 of fp32, h = 2^-8 the half step of bf16):
* out: h |out| for the result, h sum w |v| for the weights (rounded for the matrix cores) and 2^-17 of it for
  exponentials, sums and joins; and what the scores' own errors give, which the oracle adds up place by place
  (the products' D roundings, the cap's, the bias's);
* lse: the scores' errors, (length / 64 + 64) u for the sum, 4 u |lse|;
* weights: the scores' errors, those of lse as an fp32 number, and the rows' additions (the oracle's);
* eviction: places, lengths and what is moved bit for bit.
"""

import numpy as np
import pytest
import torch

import oracle
from oracle import attention as oa
from test_gpu_attention import H, U, Guarded, bits, dev, eg, host, make_cache  # noqa: F401 (eg: a fixture)

pytestmark = pytest.mark.gpu

NOTHING = 2 ** 31 - 1


def rules_on_gpu(eg, rules):
    on = {k: rules[k] for k in ("window", "cap")}
    for k, t in (("slopes", np.float32), ("doc_starts", np.int32), ("prefix_lens", np.int32)):
        on[k] = None if rules[k] is None else dev(np.asarray(rules[k], t))
    return eg.AttentionRules(**on)


def check(got, want, max_len):
    """out bits and lse against the oracle's."""
    out, lse = got
    ref, ref_lse, spread, slack, lse_slack = want
    value = oracle.bf16_value(out)
    nan = np.isnan(ref)
    assert np.array_equal(nan, np.isnan(value))
    tol = H * np.abs(ref) + (H + 2.0 ** -17) * spread + (1 + H) * slack + 1e-30
    over = np.where(nan, -1, np.abs(value - ref) - tol)
    assert over.max() <= 0, f"off by {np.abs(value - ref).flat[over.argmax()]:.3g}, allowed {tol.flat[over.argmax()]:.3g}"
    empty = np.isneginf(ref_lse)
    assert np.array_equal(empty, np.isneginf(lse))
    assert not out[empty].any()
    off = np.abs(lse[~empty].astype(np.float64) - ref_lse[~empty])
    tol = lse_slack[~empty] + (max_len / 64 + 64) * U + 4 * U * np.abs(ref_lse[~empty])
    assert np.all(off <= tol), np.max(off / tol)


class Chunk:
    """A cache of unrelated pages, sequences with new tokens, rules; table entries of unseen pages are garbage and
    places that no token sees hold NaN."""

    def __init__(self, eg, rng, fmt, ps, hq, hkv, D, new, lens, rules=None, sharp=2.0, scale=None, max_len=None, tail=0,
                 spoil=True):
        self.eg, self.rules = eg, {**oa.rules_of(), **(rules or {})}
        new, lens = np.asarray(new), np.asarray(lens, np.int32)
        n = len(lens)
        self.cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.T = int(self.cu[-1]) + tail                  # rows behind the last sequence
        self.max_len = int(max(0, lens.max())) if max_len is None else max_len
        self.lens, self.scale = lens, D ** -0.5 if scale is None else scale
        width = max(1, -(-self.max_len // ps))
        need = np.minimum(-(-np.maximum(lens, 0) // ps), width)
        pages = int(need.sum()) + 1
        self.arrays, self.held, self.cache = make_cache(eg, rng, fmt, pages, hkv, ps, D)
        perm = rng.permutation(pages)
        self.table = rng.integers(-2 ** 31, 2 ** 31 - 1, size=(n, width)).astype(np.int32)
        at, seen = 0, np.zeros((pages, ps), bool)
        self.seen = []
        for s in range(n):
            self.table[s, :need[s]] = perm[at:at + need[s]]
            at += need[s]
            length = min(max(int(lens[s]), 0), self.max_len, width * ps)
            tokens = np.arange(self.cu[s], self.cu[s + 1])
            pos = length - len(tokens) + np.arange(len(tokens))
            mine = oa._seen(self.rules, s, tokens, pos, length, np.ones(length, bool))
            self.seen.append(mine)
            p = np.arange(length)[mine.any(0)]
            seen[self.table[s][p // ps], p % ps] = True
        if spoil:
            hide = np.broadcast_to(~seen[:, None, :, None], (pages, hkv, ps, D))
            for w in (0, 1):
                self.arrays[w][hide] = 0x7FC1 if fmt == "bf16" else 0x7F
                self.arrays[w][hide & (rng.random(hide.shape) < 0.3)] = 0x7F80 if fmt == "bf16" else 0xFF
                if fmt != "bf16":
                    self.arrays[w + 2][np.broadcast_to(~seen[:, None, :, None], self.arrays[w + 2].shape)] = 255
            self.refresh()
            # A page none of whose places is seen: its entry may be anything.
            for s in range(n):
                for e in range(need[s]):
                    if not seen[self.table[s, e]].any() and rng.random() < 0.5:
                        self.table[s, e] = rng.choice([-1, pages, 2 ** 31 - 1])
        self.q = bits(sharp * rng.normal(size=(self.T, hq, D)))
        self.bad = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.out, self.lse = Guarded((self.T, hq, D), torch.int16), Guarded((self.T, hq), torch.float32)
        self.ws = Guarded((eg.engram_chunk_attention_workspace_bytes(self.T, n, hq, hkv, D, self.max_len),), torch.uint8)
        self.upload()

    def refresh(self):
        for g, a in zip(self.held, self.arrays):
            if g is not None:
                g.t.copy_(dev(a))

    def upload(self):
        self.on_gpu = [dev(a) for a in (self.q, self.cu, self.table, self.lens)]
        self.gpu_rules = rules_on_gpu(self.eg, self.rules)

    def run(self, stream=None):
        q, cu, table, lens = self.on_gpu
        self.eg.engram_chunk_attention(self.cache, q, cu, table, lens, self.max_len, self.scale, self.out.t, self.ws.t,
                                       rules=self.gpu_rules, lse=self.lse.t, bad_pages=self.bad, stream=stream)

    def want(self):
        # The oracle's table has no garbage.
        table = np.where((self.table >= 0) & (self.table < self.arrays[0].shape[0]), self.table, -1)
        return oa.chunk_attention(self.arrays, self.q, self.cu, table, self.lens, self.max_len, self.scale, self.rules)

    def check(self, bad=False):
        self.run()
        self.ws.host()
        out, lse = self.out.host(), self.lse.host()
        last = int(self.cu[-1])
        assert np.all(out[last:] == 0x5A5A) and np.all(lse[last:] == np.float32(1234.5)), "rows of no sequence written"
        assert (self.bad.item() > 0) == bad
        check((out[:last], lse[:last]), [x[:last] for x in self.want()], self.max_len)
        return out, lse


def docs_for(new, lens, every, pad=0):
    """doc_starts with a document every `every` places, the last `pad` tokens of each sequence seeing nothing."""
    got = []
    for n, length in zip(new, lens):
        start = np.arange(length - n, length) // every * every
        start[n - min(n, pad):] = NOTHING
        got.append(start)
    return np.concatenate(got).astype(np.int32)


CHUNKS = [  # fmt, page size, q heads, kv heads, D, new tokens, lengths
    ("bf16", 16, 1, 1, 32, [1], [1]), ("bf16", 8, 4, 2, 64, [1, 0, 3, 5], [1, 7, 3, 64]),
    ("bf16", 16, 8, 2, 128, [64, 65, 63], [64, 65, 200]), ("bf16", 64, 3, 3, 96, [40, 1], [100, 129]),
    ("bf16", 16, 16, 1, 160, [9, 20], [64, 20]), ("bf16", 32, 6, 2, 192, [33], [300]),
    ("bf16", 128, 5, 1, 224, [31, 2], [31, 130]), ("bf16", 16, 4, 4, 256, [70, 7], [70, 600]),
    ("bf16", 4096, 2, 1, 64, [10], [4200]), ("bf16", 16, 32, 8, 128, [1, 1, 1], [700, 1, 65]),
    ("mxfp8", 16, 8, 2, 128, [64, 1, 0], [64, 65, 3]), ("mxfp8", 8, 1, 1, 32, [17], [40]),
    ("mxfp8", 32, 12, 4, 64, [21, 37], [21, 37]), ("mxfp8", 16, 6, 2, 96, [100], [333]),
    ("mxfp8", 16, 3, 1, 160, [45], [90]), ("mxfp8", 64, 8, 8, 192, [5, 6], [5, 700]),
    ("mxfp8", 8, 7, 1, 224, [30], [31]), ("mxfp8", 16, 16, 2, 256, [50], [180]),
    ("bf16", 16, 40, 1, 64, [30, 2], [77, 260]),      # rows of more than a block a sequence, blocks that cut a token's heads
    ("bf16", 16, 8, 8, 128, [300], [300]), ("bf16", 16, 7, 1, 128, [150, 3], [150, 900]),
]


@pytest.mark.parametrize("fmt,ps,hq,hkv,D,new,lens", CHUNKS)
def test_chunk_attention(eg, fmt, ps, hq, hkv, D, new, lens):
    Chunk(eg, np.random.default_rng(D + sum(new)), fmt, ps, hq, hkv, D, new, lens, tail=2).check()


RULES = [
    dict(window=1), dict(window=20), dict(window=2 ** 31 - 1), dict(cap=2.0), dict(cap=30.0), dict(slopes=True),
    dict(prefix=10), dict(prefix=1000), dict(docs=16), dict(docs=50, pad=3), dict(window=30, prefix=5),
    dict(window=9, prefix=70, docs=40), dict(cap=5.0, slopes=True, window=33, prefix=3, docs=100, pad=1),
    dict(pad=1000),                                    # nothing sees anything
]


@pytest.mark.parametrize("fmt,hq,hkv,D,new,lens", [
    ("bf16", 8, 2, 64, [50, 1, 90, 0, 7], [120, 33, 90, 5, 70]), ("mxfp8", 6, 1, 128, [1, 1, 2], [200, 64, 700]),
    ("bf16", 4, 4, 256, [130], [130]), ("mxfp8", 12, 3, 96, [200, 30], [650, 700])])
@pytest.mark.parametrize("rule", RULES)
def test_chunk_attention_rules(eg, fmt, hq, hkv, D, new, lens, rule):
    rng = np.random.default_rng(len(new) + D)
    rules = {k: rule[k] for k in ("window", "cap") if k in rule}
    if "slopes" in rule:
        rules["slopes"] = (2.0 ** (-8.0 * (np.arange(hq) + 1) / hq)).astype(np.float32)
    if "prefix" in rule:
        rules["prefix_lens"] = np.array([rule["prefix"] + i for i in range(len(lens))], np.int32)
    if "docs" in rule or "pad" in rule:
        rules["doc_starts"] = docs_for(new, lens, rule.get("docs", 10 ** 6), rule.get("pad", 0))
    Chunk(eg, rng, fmt, 16, hq, hkv, D, new, lens, rules).check()


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
def test_chunk_attention_prefix_far_before_a_window(eg, fmt):
    """A few first places and a window far behind them; the pages between are no pages of the cache."""
    rng = np.random.default_rng(3)
    c = Chunk(eg, rng, fmt, 16, 8, 2, 64, [3, 40], [9000, 5000], dict(window=100, prefix_lens=np.array([4, 70])))
    c.check()
    # Documents that begin inside the prefix, behind it, and in no order.
    starts = rng.choice([0, 2, 60, 70, 71, 4000, 4990, NOTHING, -5], size=43)
    Chunk(eg, rng, fmt, 16, 8, 2, 64, [3, 40], [9000, 5000],
          dict(window=100, prefix_lens=np.array([4, 70]), doc_starts=starts.astype(np.int32))).check()


@pytest.mark.parametrize("fmt,hq,hkv,D,new,lens", [
    ("bf16", 8, 2, 128, [1, 4], [9000, 5000]), ("mxfp8", 32, 8, 128, [2], [20000]), ("bf16", 6, 1, 256, [3, 1], [4000, 77]),
    ("mxfp8", 64, 1, 64, [70, 3, 0, 9], [3000, 4000, 9, 2500]), ("bf16", 4, 2, 96, [500], [5000]),
    ("bf16", 1, 1, 32, [1] * 300, list(range(0, 3000, 10)))])
def test_chunk_attention_split_over_the_length(eg, fmt, hq, hkv, D, new, lens):
    c = Chunk(eg, np.random.default_rng(D), fmt, 16, hq, hkv, D, new, lens)
    first = c.check()
    c.ws.t.fill_(255)
    again = c.check()
    assert all(np.array_equal(a, b) for a, b in zip(first, again))


def test_chunk_attention_of_more_sequences_than_threads(eg):
    rng = np.random.default_rng(5)
    new = rng.integers(0, 4, size=1500)
    lens = new + rng.integers(0, 60, size=1500)
    lens[rng.random(1500) < 0.1] = 0                   # and more new tokens than places
    Chunk(eg, rng, "mxfp8", 8, 3, 1, 32, new, lens, dict(window=25), max_len=100).check()


def test_chunk_attention_of_many_blocks_in_a_sequence(eg):
    rng = np.random.default_rng(6)
    Chunk(eg, rng, "bf16", 16, 64, 1, 32, [1100], [1100], dict(window=70, doc_starts=docs_for([1100], [1100], 33))).check()


def test_chunk_attention_scales_and_lengths(eg):
    rng = np.random.default_rng(7)
    for kw in (dict(sharp=300.0), dict(scale=-0.3), dict(scale=0.0), dict(scale=-0.3, rules=dict(cap=3.0)),
               dict(sharp=200.0, rules=dict(cap=50.0))):
        Chunk(eg, rng, "bf16", 16, 8, 2, 128, [40, 2], [100, 70], **kw).check()
    Chunk(eg, rng, "bf16", 16, 4, 2, 64, [10, 5, 7], [-5, 90, 64], max_len=64, spoil=False).check()
    Chunk(eg, rng, "mxfp8", 16, 4, 2, 64, [3, 4], [3, 70], max_len=100000).check()
    Chunk(eg, rng, "bf16", 16, 4, 2, 64, [3, 4], [3, 70], max_len=0, spoil=False).check()
    Chunk(eg, rng, "bf16", 16, 4, 2, 64, [9, 4], [3, 0]).check()       # more new tokens than places


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_chunk_attention_values_not_finite_reach_only_rows_that_see_them(eg, fmt, D):
    """NaN and infinities in keys and values of later tokens, of other documents, past the window: rows that do not
    see them keep their results, rows that do get NaN (a NaN value: in its dimension alone)."""
    rng = np.random.default_rng(8)
    c = Chunk(eg, rng, fmt, 16, 8, 2, D, [90, 3], [150, 70], dict(window=60), spoil=False)
    before = c.check()
    ps = 16
    nan, inf = (0x7FC1, 0x7F80) if fmt == "bf16" else (0x7F, 0xFF)
    touched = np.zeros(93, bool)
    for place, what in ((149, nan), (120, inf), (64, nan), (63, nan)):
        c.arrays[1][c.table[0, place // ps], :, place % ps, [5, 40]] = what
        touched[:90] |= c.seen[0][:, place]
    c.refresh()
    out, lse = c.check() if fmt != "bf16" else (c.run(), None) and (c.out.host(), c.lse.host())
    assert np.array_equal(lse, before[1])
    value = oracle.bf16_value(out)
    hit = np.isnan(value) | np.isinf(value)
    assert np.array_equal(hit.any((1, 2)), touched)
    assert not hit[..., np.setdiff1d(np.arange(D), [5, 40])].any()
    assert np.array_equal(out[~touched], before[0][~touched])
    # Keys: all of a row that sees one.
    c.arrays[1][...] = np.where(np.isin(c.arrays[1], (nan, inf)), 0, c.arrays[1])
    c.refresh()
    c.run()
    before = c.out.host()
    c.arrays[0][c.table[0, 100 // ps], :, 100 % ps, 7] = nan
    c.refresh()
    c.run()
    out = oracle.bf16_value(c.out.host())
    touched = np.concatenate([c.seen[0][:, 100], np.zeros(3, bool)])
    assert np.isnan(out[touched]).all() and np.array_equal(c.out.host()[~touched], before[~touched])


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
@pytest.mark.parametrize("D,new", [(64, [7, 3]), (96, [4, 2]), (128, [7, 3]), (256, [7, 3])])
def test_chunk_attention_of_few_rows_values_not_finite(eg, fmt, D, new):
    """As above, where all sequences have few rows."""
    rng, ps = np.random.default_rng(11), 16
    c = Chunk(eg, rng, fmt, ps, 8, 2, D, new, [150, 70], dict(window=80), spoil=False)
    before = c.check()
    nan, inf = (0x7FC1, 0x7F80) if fmt == "bf16" else (0x7F, 0xFF)
    first = 150 - new[0] - 79                          # the first place that the first token sees
    touched = np.zeros(sum(new), bool)
    for place, what in ((149, nan), (147, inf), (first, nan), (first + 2, inf), (first - 1, nan)):
        c.arrays[1][c.table[0, place // ps], :, place % ps, [5, 17]] = what
        touched[:new[0]] |= c.seen[0][:, place]
    c.refresh()
    c.run()
    out = c.out.host()
    assert np.array_equal(c.lse.host(), before[1])
    value = oracle.bf16_value(out)
    hit = ~np.isfinite(value)
    assert np.array_equal(hit.any((1, 2)), touched) and hit[touched].any(1)[:, [5, 17]].all()
    assert not hit[..., np.setdiff1d(np.arange(D), [5, 17])].any()
    assert np.array_equal(out[~touched], before[0][~touched])
    rest = np.setdiff1d(np.arange(D), [5, 17])
    assert np.array_equal(out[..., rest], before[0][..., rest])


@pytest.mark.parametrize("fmt,D", [("bf16", 64), ("mxfp8", 128), ("bf16", 256)])
@pytest.mark.parametrize("new,length,window", [(10, 5, 2), (300, 200, 3), (300, 299, 40), (90, 1, 7)])
def test_chunk_attention_of_more_tokens_than_places_in_a_window(eg, fmt, D, new, length, window):
    """The first tokens have no place and see nothing; those behind them see places that the last ones do not."""
    rng = np.random.default_rng(12)
    Chunk(eg, rng, fmt, 16, 4, 2, D, [new], [length], dict(window=window)).check()
    docs = docs_for([new], [length], 25)
    Chunk(eg, rng, fmt, 16, 4, 2, D, [new], [length], dict(window=window, doc_starts=docs)).check()
    Chunk(eg, rng, fmt, 16, 4, 2, D, [new], [length], dict(window=window, prefix_lens=np.array([2]))).check()


@pytest.mark.parametrize("fmt,hq,hkv,D", [("bf16", 8, 2, 64), ("mxfp8", 12, 3, 128), ("bf16", 16, 2, 256)])
@pytest.mark.parametrize("rules", [{}, dict(window=700), dict(cap=4.0)])
def test_chunk_attention_of_long_and_short_chunks_at_once(eg, fmt, hq, hkv, D, rules):
    """Some sequences have a prompt's rows, some a single token's over a long context, some none."""
    rng = np.random.default_rng(13)
    c = Chunk(eg, rng, fmt, 16, hq, hkv, D, [300, 1, 2, 0, 200, 3, 1, 8, 1], [1500, 2000, 64, 5, 200, 1100, 2900, 8, 1], rules,
              tail=1)
    first = c.check()
    c.ws.t.fill_(255)
    assert all(np.array_equal(a, b) for a, b in zip(first, c.check()))


def test_chunk_attention_graphs_that_share_a_workspace(eg):
    """Two captured calls of different sizes with one workspace, replayed in turn."""
    rng = np.random.default_rng(14)
    calls = [Chunk(eg, rng, "bf16", 16, 8, 2, 128, new, lens) for new, lens in
             (([200, 30], [2000, 40]), ([1, 1, 4], [900, 3, 1200]))]
    want = [c.check() for c in calls]
    ws = max((c.ws for c in calls), key=lambda g: g.t.numel())
    graphs = []
    for c in calls:
        c.ws = ws
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            c.run()
    for i in (0, 1, 1, 0, 1, 0):
        calls[i].out.t.zero_()
        graphs[i].replay()
        torch.cuda.synchronize()
        assert np.array_equal(calls[i].out.host(), want[i][0]) and np.array_equal(calls[i].lse.host(), want[i][1])


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
def test_chunk_attention_bad_pages_are_not_seen(eg, fmt):
    rng = np.random.default_rng(9)
    c = Chunk(eg, rng, fmt, 16, 8, 2, 128, [40, 5, 3], [300, 16, 64], spoil=False)
    c.table[0, 3], c.table[0, 17], c.table[1, 0] = -1, c.arrays[0].shape[0], 2 ** 31 - 1
    c.table[2, :4] = -2 ** 31
    c.upload()
    c.check(bad=True)
    assert np.isneginf(c.lse.host()[40:48]).all()


def test_chunk_attention_of_one_token_is_that_of_paged_attention(eg):
    rng = np.random.default_rng(10)
    c = Chunk(eg, rng, "mxfp8", 16, 32, 8, 128, [1] * 5, [300, 1, 5000, 64, 0])
    out, lse = c.check()
    q, _, table, lens = c.on_gpu
    out1, lse1 = Guarded(out.shape, torch.int16), Guarded(lse.shape, torch.float32)
    ws = torch.empty(eg.engram_paged_attention_workspace_bytes(5, 32, 8, 128, c.max_len), dtype=torch.uint8, device="cuda")
    eg.engram_paged_attention(c.cache, q, table, lens, c.max_len, c.scale, out1.t, ws, lse=lse1.t)
    a, b = oracle.bf16_value(out), oracle.bf16_value(out1.host())
    assert np.all(np.abs(a - b) <= 4 * H * np.abs(b) + 4 * H)
    same = np.isneginf(lse)
    assert np.array_equal(same, np.isneginf(lse1.host()))
    assert np.all(np.abs(lse[~same] - lse1.host()[~same]) <= 1e-4)


# ---------------------------------------------------------------- shared prefixes

class Shared:
    def __init__(self, eg, rng, fmt, ps, hq, hkv, D, cu, prefixes, lens, max_prefix=None, max_len=None):
        self.eg = eg
        self.cu, self.prefixes, self.lens = (np.asarray(x, np.int32) for x in (cu, prefixes, lens))
        self.max_prefix = int(self.prefixes.max()) if max_prefix is None else max_prefix
        self.max_len = int(self.lens.max()) if max_len is None else max_len
        n, groups = len(lens), len(prefixes)
        need = [-(-np.maximum(x, 0) // ps) for x in (self.prefixes, self.lens)]
        pages = int(sum(x.sum() for x in need)) + 1
        self.arrays, self.held, self.cache = make_cache(eg, rng, fmt, pages, hkv, ps, D)
        perm, at, self.tables = rng.permutation(pages), 0, []
        seen = np.zeros((pages, ps), bool)
        for x, lengths in zip(need, (self.prefixes, self.lens)):
            t = rng.integers(-2 ** 31, 2 ** 31 - 1, size=(len(x), max(1, int(x.max())))).astype(np.int32)
            for i, c in enumerate(x):
                t[i, :c] = perm[at:at + c]
                at += c
                p = np.arange(max(0, lengths[i]))
                seen[t[i][p // ps], p % ps] = True
            self.tables.append(t)
        hide = np.broadcast_to(~seen[:, None, :, None], self.arrays[0].shape)
        for w in (0, 1):
            self.arrays[w][hide] = 0x7FC1 if fmt == "bf16" else 0x7F
            self.held[w].t.copy_(dev(self.arrays[w]))
        self.scale, self.q = D ** -0.5, bits(2.0 * rng.normal(size=(n, hq, D)))
        self.out, self.lse = Guarded((n, hq, D), torch.int16), Guarded((n, hq), torch.float32)
        self.ws = Guarded((eg.engram_shared_prefix_attention_workspace_bytes(
            n, groups, hq, hkv, D, self.max_prefix, self.max_len),), torch.uint8)
        self.bad = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.upload()

    def upload(self):
        self.on_gpu = [dev(a) for a in (self.q, self.cu, self.tables[0], self.prefixes, self.tables[1], self.lens)]

    def run(self, stream=None):
        q, cu, prefix_table, prefixes, table, lens = self.on_gpu
        self.eg.engram_shared_prefix_attention(self.cache, q, cu, prefix_table, prefixes, self.max_prefix, table, lens,
                                               self.max_len, self.scale, self.out.t, self.ws.t, lse=self.lse.t,
                                               bad_pages=self.bad, stream=stream)

    def check(self, bad=False):
        self.run()
        self.ws.host()
        assert (self.bad.item() > 0) == bad
        want = oa.shared_prefix_attention(self.arrays, self.q, self.cu, self.tables[0], self.prefixes, self.max_prefix,
                                          self.tables[1], self.lens, self.max_len, self.scale)
        got = self.out.host(), self.lse.host()
        check(got, want, self.max_prefix + self.max_len)
        return got


SHARED = [  # fmt, page size, q heads, kv heads, D, cu_groups, prefixes, own lengths
    ("bf16", 16, 32, 8, 128, [0, 8], [500], [1, 5, 64, 65, 2, 9, 30, 60]), ("bf16", 16, 1, 1, 32, [0, 1], [1], [0]),
    ("mxfp8", 16, 8, 2, 64, [0, 3, 3, 7], [100, 50, 777], [3, 0, 20, 1, 1, 90, 64]),
    ("mxfp8", 32, 16, 2, 128, [0, 70], [3000], list(range(70))), ("bf16", 8, 6, 2, 96, [2, 4], [129], [10, 0, 7, 300, 5]),
    ("bf16", 64, 4, 1, 256, [0, 2, 5], [2000, 0], [10, 700, 0, 3, 64]), ("mxfp8", 16, 5, 5, 160, [0, 4], [333], [8, 9, 10, 0]),
    ("bf16", 16, 40, 1, 192, [0, 9, 10], [600, 65], [1] * 10), ("mxfp8", 8, 3, 1, 224, [0, 50], [4000], [0] * 50),
    ("bf16", 16, 8, 8, 128, [0, 300], [70], list(range(300))), ("bf16", 128, 32, 8, 128, [0, 64], [9000], [70] * 64),
]


@pytest.mark.parametrize("fmt,ps,hq,hkv,D,cu,prefixes,lens", SHARED)
def test_shared_prefix_attention(eg, fmt, ps, hq, hkv, D, cu, prefixes, lens):
    s = Shared(eg, np.random.default_rng(D + len(lens)), fmt, ps, hq, hkv, D, cu, prefixes, lens)
    first = s.check()
    s.ws.t.fill_(255)
    assert all(np.array_equal(a, b) for a, b in zip(first, s.check()))


@pytest.mark.parametrize("fmt,hq,hkv,D", [("bf16", 8, 2, 64), ("mxfp8", 40, 1, 128)])
def test_shared_prefix_attention_of_many_groups(eg, fmt, hq, hkv, D):
    """Groups of none, one and many sequences, prefixes of all lengths, sequences of no group before and behind them."""
    rng = np.random.default_rng(22)
    sizes = np.concatenate([rng.integers(0, 4, size=60), [40]])
    cu = np.concatenate([[2], 2 + np.cumsum(sizes)])
    n = int(cu[-1]) + 3
    Shared(eg, rng, fmt, 16, hq, hkv, D, cu, rng.integers(0, 700, size=61), rng.integers(0, 90, size=n)).check()


def test_shared_prefix_attention_lengths_out_of_range_and_bad_pages(eg):
    rng = np.random.default_rng(20)
    Shared(eg, rng, "bf16", 16, 4, 2, 64, [0, 2, 3], [100, -4], [-1, 30, 64], max_prefix=5000, max_len=3000).check()
    s = Shared(eg, rng, "mxfp8", 16, 4, 2, 64, [0, 2, 3], [100, 40], [40, 30, 20])
    s.tables[0][0, 2], s.tables[1][1, 0], s.tables[1][2, :] = -1, s.arrays[0].shape[0], 2 ** 31 - 1
    s.upload()
    s.check(bad=True)


def test_shared_prefix_attention_is_that_of_paged_attention_on_joined_tables(eg):
    """A prefix that fills its pages, its page table before each sequence's own."""
    rng = np.random.default_rng(21)
    s = Shared(eg, rng, "mxfp8", 16, 8, 2, 128, [0, 4], [160], [5, 33, 70, 16])
    out, lse = s.check()
    table = np.concatenate([np.repeat(s.tables[0], 4, 0), s.tables[1]], 1)
    lens = dev((s.lens + 160).astype(np.int32))
    out1, lse1 = Guarded(out.shape, torch.int16), Guarded(lse.shape, torch.float32)
    ws = torch.empty(eg.engram_paged_attention_workspace_bytes(4, 8, 2, 128, 230), dtype=torch.uint8, device="cuda")
    eg.engram_paged_attention(s.cache, s.on_gpu[0], dev(table), lens, 230, s.scale, out1.t, ws, lse=lse1.t)
    a, b = oracle.bf16_value(out), oracle.bf16_value(out1.host())
    assert np.all(np.abs(a - b) <= 4 * H * np.abs(b) + 4 * H)
    assert np.all(np.abs(lse - lse1.host()) <= 1e-4)


# ---------------------------------------------------------------- weights

def weigh(eg, c, rng, extra=3, old=True):
    """One call of engram_cache_weights on a Chunk's inputs and its own lse, against the oracle."""
    n, hkv = len(c.lens), c.arrays[0].shape[1]
    c.run()
    lse = c.lse.host().copy()
    w = Guarded((n, hkv, c.max_len + extra), torch.float32)
    start = np.abs(rng.normal(size=w.t.shape)).astype(np.float32) * (1.0 if old else 0.0)
    w.t.copy_(dev(start))
    q, cu, table, lens = c.on_gpu
    bad = torch.zeros(1, dtype=torch.int32, device="cuda")
    eg.engram_cache_weights(c.cache, q, cu, table, lens, c.max_len, c.scale, c.lse.t, w.t, rules=c.gpu_rules, bad_pages=bad)
    t = np.where((c.table >= 0) & (c.table < c.arrays[0].shape[0]), c.table, -1)
    want, slack = oa.cache_weights(c.arrays, c.q, c.cu, t, c.lens, c.max_len, c.scale, lse, w.t.shape[2], c.rules)
    got = w.host().astype(np.float64)
    tol = slack + U * (np.abs(start) + np.abs(want)) + 1e-30
    over = np.abs(got - start - want) - tol
    assert over.max() <= 0, f"off by {np.abs(got - start - want).flat[over.argmax()]:.3g}, allowed {tol.flat[over.argmax()]:.3g}"
    for s in range(n):
        length = min(max(int(c.lens[s]), 0), c.max_len)
        assert np.array_equal(w.host()[s, :, length:], start[s, :, length:])
    return w.host(), bad.item()


@pytest.mark.parametrize("fmt,ps,hq,hkv,D,new,lens", CHUNKS)
def test_cache_weights(eg, fmt, ps, hq, hkv, D, new, lens):
    rng = np.random.default_rng(D + sum(new))
    c = Chunk(eg, rng, fmt, ps, hq, hkv, D, new, lens)
    assert weigh(eg, c, rng)[1] == 0
    first, again = (weigh(eg, c, np.random.default_rng(0), old=False)[0] for _ in range(2))
    assert np.array_equal(first, again)
    # Every head's weights of a token sum to 1.
    total = first[..., :c.max_len].sum(dtype=np.float64)
    rows = sum(int(s.any(1).sum()) for s in c.seen) * hq
    assert abs(total - rows) <= 1e-4 * max(1, rows)


@pytest.mark.parametrize("rule", RULES)
def test_cache_weights_rules(eg, rule):
    rng = np.random.default_rng(31)
    hq, new, lens = 6, [50, 1, 90, 0, 7], [120, 33, 90, 5, 300]
    rules = {k: rule[k] for k in ("window", "cap") if k in rule}
    if "slopes" in rule:
        rules["slopes"] = (2.0 ** (-8.0 * (np.arange(hq) + 1) / hq)).astype(np.float32)
    if "prefix" in rule:
        rules["prefix_lens"] = np.array([rule["prefix"] + i for i in range(len(lens))], np.int32)
    if "docs" in rule or "pad" in rule:
        rules["doc_starts"] = docs_for(new, lens, rule.get("docs", 10 ** 6), rule.get("pad", 0))
    c = Chunk(eg, rng, "mxfp8", 16, hq, 2, 96, new, lens, rules)
    assert weigh(eg, c, rng)[1] == 0


def test_cache_weights_bad_pages(eg):
    rng = np.random.default_rng(32)
    c = Chunk(eg, rng, "bf16", 16, 8, 2, 128, [4, 5], [300, 40], spoil=False)
    c.table[0, 3], c.table[1, 0] = -1, c.arrays[0].shape[0]
    c.upload()
    assert weigh(eg, c, rng)[1] > 0


# ---------------------------------------------------------------- eviction

def evict_once(eg, rng, fmt, ps, hkv, D, lens, keep, sinks, recent, weights=None, max_len=None, extra=2, to_extra=1):
    lens = np.asarray(lens, np.int32)
    n = len(lens)
    max_len = int(max(0, lens.max())) if max_len is None else max_len
    width, to_width = max(1, -(-max_len // ps)), max(1, -(-keep // ps)) + to_extra
    pages = n * (width + to_width) + 1
    arrays, held, handle = make_cache(eg, rng, fmt, pages, hkv, ps, D)
    perm = rng.permutation(pages).astype(np.int32)
    table, to = perm[:n * width].reshape(n, width).copy(), perm[n * width:n * (width + to_width)].reshape(n, to_width).copy()
    if weights is None:
        weights = np.exp(2 * rng.normal(size=(n, hkv, max_len + extra)))
        weights = np.where(weights < 0.5, 0.0, weights)          # many equal ones
    weights = np.asarray(weights, np.float32)
    new_lens = torch.full((n,), -7, dtype=torch.int32, device="cuda")
    new_weights = Guarded((n, hkv, keep + extra), torch.float32)
    kept = torch.full((n, hkv, keep), -7, dtype=torch.int32, device="cuda")
    bad = torch.zeros(1, dtype=torch.int32, device="cuda")
    eg.engram_cache_evict(handle, dev(table), dev(lens), max_len, keep, sinks, recent, dev(weights), dev(to), new_lens,
                          new_weights.t, kept, bad_pages=bad)
    room = width * ps
    want = oa.evict(weights, lens, max_len, room, keep, sinks, recent)
    assert np.array_equal(kept.cpu().numpy(), want)
    count = np.minimum(np.clip(lens, 0, min(max_len, room)), keep)
    assert np.array_equal(new_lens.cpu().numpy(), count)
    got_w = new_weights.host()
    for s in range(n):
        for h in range(hkv):
            i = np.arange(count[s])
            p = want[s, h, :count[s]]
            assert np.array_equal(got_w[s, h, :count[s]].view(np.uint32), weights[s, h][p].view(np.uint32))
            assert not got_w[s, h, count[s]:].view(np.uint32).any()
            for a in arrays:
                if a is not None:
                    a[to[s][i // ps], h, i % ps] = a[table[s][p // ps], h, p % ps]
    for a, g in zip(arrays, held):
        if a is not None:
            assert np.array_equal(a, g.host())
    assert bad.item() == 0


EVICT = [  # fmt, page size, heads, D, lengths, keep, sinks, recent
    ("bf16", 16, 2, 64, [100, 40, 0, 1], 40, 4, 8), ("bf16", 8, 1, 32, [5], 1, 0, 0), ("bf16", 8, 1, 32, [5], 1, 1, 0),
    ("bf16", 8, 1, 32, [9], 2, 1, 1), ("mxfp8", 16, 8, 128, [300, 256, 257], 256, 4, 64), ("mxfp8", 32, 3, 96, [5000], 1000, 0, 0),
    ("mxfp8", 8, 2, 192, [70, 90], 64, 32, 32), ("bf16", 64, 4, 256, [1000, 2000, 64], 500, 0, 499),
    ("mxfp8", 16, 1, 160, [9999], 4097, 100, 1), ("bf16", 16, 5, 224, [50], 49, 0, 0), ("mxfp8", 16, 2, 32, [20000, 5], 3, 1, 1),
    ("bf16", 16, 2, 96, [30, 20], 40, 4, 8), ("bf16", 16, 1, 64, [4096, 4097], 4096, 0, 0), ("bf16", 8, 3, 64, [33, 9], 0, 0, 0),
]


@pytest.mark.parametrize("fmt,ps,hkv,D,lens,keep,sinks,recent", EVICT)
def test_cache_evict(eg, fmt, ps, hkv, D, lens, keep, sinks, recent):
    evict_once(eg, np.random.default_rng(D + keep), fmt, ps, hkv, D, lens, keep, sinks, recent)


def test_cache_evict_weights_of_every_kind(eg):
    """All equal, in order, NaN, infinities, both zeros, negative ones, numbers next to each other."""
    rng = np.random.default_rng(40)
    n, length = 9, 3000
    w = np.zeros((n, 1, length), np.float32)
    w[1] = 1.0
    w[2] = np.arange(length)
    w[3] = -np.arange(length)
    w[4] = rng.choice(np.array([0.0, -0.0, np.nan, np.inf, -np.inf, 1e-45, -1e-45], np.float32), size=length)
    w[5] = np.float32(1.0) + rng.integers(0, 4, size=length) * np.float32(2.0 ** -23)
    w[6] = np.nan
    w[7] = rng.normal(size=length)
    w[8] = np.frombuffer(rng.integers(0, 2 ** 32, size=length, dtype=np.uint32).tobytes(), np.float32)
    for keep, sinks, recent in ((1000, 0, 0), (1, 0, 0), (2999, 3, 10), (1500, 700, 700)):
        evict_once(eg, rng, "bf16", 16, 1, 32, [length] * n, keep, sinks, recent, weights=w)


def test_cache_evict_lengths_out_of_range(eg):
    rng = np.random.default_rng(41)
    evict_once(eg, rng, "mxfp8", 16, 2, 64, [-3, 500, 90], 50, 2, 4, max_len=100)
    evict_once(eg, rng, "bf16", 16, 2, 64, [60, 20], 50, 2, 4, max_len=4000)
    evict_once(eg, rng, "bf16", 16, 2, 64, [0, 0], 50, 2, 4, max_len=0)


def test_cache_evict_bad_pages(eg):
    rng = np.random.default_rng(42)
    ps, hkv, D, keep = 16, 2, 64, 32
    arrays, held, handle = make_cache(eg, rng, "mxfp8", 8, hkv, ps, D)
    table, to = np.array([[0, -1, 2, 3]], np.int32), np.array([[4, 8]], np.int32)
    lens, w = np.array([64], np.int32), rng.random((1, hkv, 64)).astype(np.float32)
    z = lambda *s, dtype=torch.int32: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    bad, kept, new_w, new_lens = z(1), z(1, hkv, keep), z(1, hkv, keep, dtype=torch.float32), z(1)
    eg.engram_cache_evict(handle, dev(table), dev(lens), 64, keep, 4, 4, dev(w), dev(to), new_lens, new_w, kept, bad_pages=bad)
    want = oa.evict(w, lens, 64, 64, keep, 4, 4)
    assert np.array_equal(kept.cpu().numpy(), want) and bad.item() > 0
    for h in range(hkv):
        for i, p in enumerate(want[0, h][:ps]):            # the first new page; the second is none
            page = table[0, p // ps]
            for a, zero in zip(arrays, (0, 0, 127, 127)):
                a[4, h, i] = a[page, h, p % ps] if page >= 0 else zero
    for a, g in zip(arrays, held):
        assert np.array_equal(a, g.host())


# ---------------------------------------------------------------- all of it together

class Generation:
    """A prompt in chunks, its weights, eviction, and streams that go on from what is left."""

    def __init__(self, eg, seed=50):
        rng = np.random.default_rng(seed)
        self.eg, self.rng = eg, rng
        self.hq, self.hkv, self.D, self.ps, self.n = 8, 2, 64, 16, 5
        self.T, self.keep = 150, 64
        self.arrays, self.held, self.cache = make_cache(eg, rng, "mxfp8", 40, self.hkv, self.ps, self.D)
        perm = rng.permutation(40).astype(np.int32)
        self.prompt, self.left, self.own = (dev(x) for x in (perm[None, :10], perm[None, 10:14], perm[14:24].reshape(5, 2)))
        self.scale = self.D ** -0.5
        i32 = lambda x: dev(np.asarray(x, np.int32))  # noqa: E731
        self.cu, self.lens, self.first = i32([0, self.T]), i32([self.T]), i32([0])
        self.q = dev(bits(2 * rng.normal(size=(self.T, self.hq, self.D))))
        self.q1 = dev(bits(2 * rng.normal(size=(self.n, self.hq, self.D))))
        self.groups, self.own_lens = i32([0, self.n]), i32([3, 0, 20, 17, 1])
        z = lambda *s, dtype=torch.int16: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
        f32, u8 = torch.float32, torch.uint8
        self.out, self.lse = z(self.T, self.hq, self.D), z(self.T, self.hq, dtype=f32)
        self.w, self.new_w = z(1, self.hkv, 160, dtype=f32), z(1, self.hkv, self.keep, dtype=f32)
        self.kept, self.new_lens = z(1, self.hkv, self.keep, dtype=torch.int32), z(1, dtype=torch.int32)
        self.out1, self.lse1 = z(self.n, self.hq, self.D), z(self.n, self.hq, dtype=f32)
        self.ws = z(eg.engram_chunk_attention_workspace_bytes(self.T, 1, self.hq, self.hkv, self.D, 160), dtype=u8)
        self.ws1 = z(eg.engram_shared_prefix_attention_workspace_bytes(self.n, 1, self.hq, self.hkv, self.D, 64, 32), dtype=u8)

    def run(self, stream=None):
        eg = self.eg
        with torch.cuda.stream(stream if stream is not None else torch.cuda.current_stream()):
            self.w.zero_()
        eg.engram_chunk_attention(self.cache, self.q, self.cu, self.prompt, self.lens, 160, self.scale, self.out, self.ws,
                                  lse=self.lse, stream=stream)
        eg.engram_cache_weights(self.cache, self.q, self.cu, self.prompt, self.lens, 160, self.scale, self.lse, self.w,
                                stream=stream)
        eg.engram_cache_evict(self.cache, self.prompt, self.lens, 160, self.keep, 4, 16, self.w, self.left, self.new_lens,
                              self.new_w, self.kept, stream=stream)
        eg.engram_shared_prefix_attention(self.cache, self.q1, self.groups, self.left, self.new_lens, 64, self.own,
                                          self.own_lens, 32, self.scale, self.out1, self.ws1, lse=self.lse1, stream=stream)

    def results(self):
        torch.cuda.synchronize()
        return [host(t).copy() for t in (self.out, self.lse, self.w, self.kept, self.new_w, self.new_lens, self.out1, self.lse1)]


def test_together_against_the_oracle(eg):
    s = Generation(eg)
    s.run()
    out, lse, w, kept, new_w, new_lens, out1, lse1 = s.results()
    held = [g.host() for g in s.held]
    table = host(s.prompt)
    check((out, lse), oa.chunk_attention(held, host(s.q), [0, s.T], table, [s.T], 160, s.scale), 160)
    want, slack = oa.cache_weights(held, host(s.q), [0, s.T], table, [s.T], 160, s.scale, lse, 160)
    assert np.all(np.abs(w - want) <= slack + U * want)
    assert np.array_equal(kept, oa.evict(w, [s.T], 160, 160, s.keep, 4, 16)) and new_lens[0] == s.keep
    check((out1, lse1), oa.shared_prefix_attention(held, host(s.q1), [0, s.n], host(s.left), new_lens, 64, host(s.own),
                                                   host(s.own_lens), 32, s.scale), 96)


def test_together_on_another_stream_and_in_a_graph(eg):
    s = Generation(eg)
    s.run()
    want = s.results()
    side = torch.cuda.Stream()
    for t in (s.out, s.lse, s.out1, s.kept):
        t.zero_()
    side.wait_stream(torch.cuda.current_stream())
    s.run(stream=side)
    assert all(np.array_equal(a, b) for a, b in zip(want, s.results()))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    for i in range(4):
        s.q.copy_(dev(bits((1 + i % 3) * np.random.default_rng(i).normal(size=tuple(s.q.shape)))))
        s.lens.fill_(150 - 20 * i)
        s.run()
        want = s.results()
        for t in (s.out, s.lse, s.out1, s.kept):
            t.zero_()
        graph.replay()
        got = s.results()
        assert all(np.array_equal(a, b) for a, b in zip(want, got))


def test_together_on_two_streams_at_once(eg):
    runs = [Generation(eg, seed) for seed in (51, 52)]
    want = []
    for s in runs:
        s.run()
        want.append(s.results())
    sides = [torch.cuda.Stream() for _ in runs]
    for s in runs:
        for t in (s.out, s.lse, s.out1, s.kept):
            t.zero_()
    torch.cuda.synchronize()
    for _ in range(3):
        for s, side in zip(runs, sides):
            s.run(stream=side)
    for s, w in zip(runs, want):
        assert all(np.array_equal(a, b) for a, b in zip(w, s.results()))


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
def test_beyond_32_bit_offsets(eg, fmt):
    """All four operators on pages past 4 GiB (and past 2^32 values) of the cache."""
    rng = np.random.default_rng(60)
    ps, hq, hkv, D = 4096, 4, 1, 256
    pages = 2200 if fmt == "bf16" else 4300
    shape = (pages, hkv, ps, D)
    data = [torch.empty(shape, dtype=torch.int16 if fmt == "bf16" else torch.uint8, device="cuda") for _ in range(2)]
    scales = [None] * 2 if fmt == "bf16" else [torch.empty(shape[:3] + (D // 32,), dtype=torch.uint8, device="cuda")
                                               for _ in range(2)]
    handle = eg.KVCache(eg.ENGRAM_CACHE_BF16 if fmt == "bf16" else eg.ENGRAM_CACHE_MXFP8, *data, *scales)
    small, _, _ = make_cache(eg, rng, fmt, 3, hkv, ps, D)
    for i in range(2):                                   # the last pages hold what the small cache holds
        for big, a in zip(data + scales, small):
            if a is not None:
                big[pages - 1 - i].copy_(dev(a[i]))
    table, small_table = np.array([[pages - 1], [pages - 2]], np.int32), np.array([[0], [1]], np.int32)
    cu, lens = np.array([0, 5, 8], np.int32), np.array([200, 130], np.int32)
    q = bits(2 * rng.normal(size=(8, hq, D)))
    out, lse = Guarded((8, hq, D), torch.int16), Guarded((8, hq), torch.float32)
    ws = torch.empty(eg.engram_chunk_attention_workspace_bytes(8, 2, hq, hkv, D, 200), dtype=torch.uint8, device="cuda")
    eg.engram_chunk_attention(handle, dev(q), dev(cu), dev(table), dev(lens), 200, 0.0625, out.t, ws, lse=lse.t)
    check((out.host(), lse.host()), oa.chunk_attention(small, q, cu, small_table, lens, 200, 0.0625), 200)
    w = torch.zeros(2, hkv, 200, dtype=torch.float32, device="cuda")
    eg.engram_cache_weights(handle, dev(q), dev(cu), dev(table), dev(lens), 200, 0.0625, lse.t, w)
    want, slack = oa.cache_weights(small, q, cu, small_table, lens, 200, 0.0625, lse.host(), 200)
    assert np.all(np.abs(host(w) - want) <= slack + U * want)
    to = dev(np.array([[pages - 3], [0]], np.int32))
    z = lambda *s, dtype=torch.int32: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    kept, new_w, new_lens = z(2, hkv, 50), z(2, hkv, 50, dtype=torch.float32), z(2)
    eg.engram_cache_evict(handle, dev(table), dev(lens), 200, 50, 2, 5, w, to, new_lens, new_w, kept)
    want = oa.evict(host(w), lens, 200, ps, 50, 2, 5)
    assert np.array_equal(host(kept), want)
    for big, a in zip(data + scales, small):
        if a is not None:
            assert np.array_equal(host(big[pages - 3, 0, :50]), a[0, 0][want[0, 0]])
            assert np.array_equal(host(big[0, 0, :50]), a[1, 0][want[1, 0]])
    q1 = q[:2]
    ws = torch.empty(eg.engram_shared_prefix_attention_workspace_bytes(2, 1, hq, hkv, D, 200, 130), dtype=torch.uint8,
                     device="cuda")
    out, lse = Guarded((2, hq, D), torch.int16), Guarded((2, hq), torch.float32)
    own = np.array([3, 130], np.int32)
    eg.engram_shared_prefix_attention(handle, dev(q1), dev(np.array([0, 2], np.int32)), dev(table[:1]), dev(lens[:1]), 200,
                                      dev(table[::-1].copy()), dev(own), 130, 0.0625, out.t, ws, lse=lse.t)
    check((out.host(), lse.host()), oa.shared_prefix_attention(small, q1, [0, 2], small_table[:1], lens[:1], 200,
                                                               small_table[::-1], own, 130, 0.0625), 330)


def test_empty_inputs(eg):
    z = lambda *shape, dtype=torch.int16: torch.zeros(*shape, dtype=dtype, device="cuda")  # noqa: E731
    i32, f32, u8 = torch.int32, torch.float32, torch.uint8
    cache = eg.KVCache(eg.ENGRAM_CACHE_BF16, z(1, 1, 8, 32), z(1, 1, 8, 32))
    eg.engram_chunk_attention(cache, z(0, 1, 32), z(3, dtype=i32), z(2, 4, dtype=i32), z(2, dtype=i32), 9, 1.0, z(0, 1, 32), None)
    eg.engram_chunk_attention(cache, z(4, 1, 32), z(1, dtype=i32), z(0, 4, dtype=i32), z(0, dtype=i32), 9, 1.0, z(4, 1, 32), None)
    eg.engram_shared_prefix_attention(cache, z(0, 1, 32), z(2, dtype=i32), z(1, 1, dtype=i32), z(1, dtype=i32), 8,
                                      z(0, 4, dtype=i32), z(0, dtype=i32), 0, 1.0, z(0, 1, 32), None)
    eg.engram_cache_weights(cache, z(0, 1, 32), z(3, dtype=i32), z(2, 4, dtype=i32), z(2, dtype=i32), 9, 1.0,
                            z(0, 1, dtype=f32), z(2, 1, 9, dtype=f32))
    eg.engram_cache_evict(cache, z(0, 1, dtype=i32), z(0, dtype=i32), 9, 4, 1, 1, z(0, 1, 9, dtype=f32), z(0, 1, dtype=i32),
                          z(0, dtype=i32), z(0, 1, 4, dtype=f32), z(0, 1, 4, dtype=i32))
    # A table without a column: no places.
    out, lse = Guarded((2, 1, 32), torch.int16), Guarded((2, 1), f32)
    ws = z(eg.engram_chunk_attention_workspace_bytes(2, 1, 1, 1, 32, 9), dtype=u8)
    eg.engram_chunk_attention(cache, z(2, 1, 32), dev(np.array([0, 2], np.int32)), z(1, 0, dtype=i32),
                              dev(np.array([5], np.int32)), 9, 1.0, out.t, ws, lse=lse.t)
    assert not out.host().any() and np.isneginf(lse.host()).all()


def test_binding_refuses(eg):
    z = lambda *shape, dtype=torch.int16: torch.zeros(*shape, dtype=dtype, device="cuda")  # noqa: E731
    i32, f32, u8 = torch.int32, torch.float32, torch.uint8
    cache = eg.KVCache(eg.ENGRAM_CACHE_BF16, z(2, 2, 8, 64), z(2, 2, 8, 64))
    q, cu, table, lens, out = z(3, 4, 64), z(3, dtype=i32), z(2, 2, dtype=i32), z(2, dtype=i32), z(3, 4, 64)
    ws = z(eg.engram_chunk_attention_workspace_bytes(3, 2, 4, 2, 64, 9), dtype=u8)
    chunk = lambda **kw: eg.engram_chunk_attention(  # noqa: E731
        cache, *(kw.get(k, v) for k, v in (("q", q), ("cu", cu), ("table", table), ("lens", lens))), 9, 1.0,
        kw.get("out", out), kw.get("ws", ws), rules=kw.get("rules"), lse=kw.get("lse"))
    chunk()
    for kw, what in ((dict(q=z(3, 4, 32)), "q must be"), (dict(cu=z(4, dtype=i32)), "table must be"),
                     (dict(lens=z(1, dtype=i32)), "lens"), (dict(out=z(2, 4, 64)), "out"), (dict(lse=z(11, dtype=f32)), "lse"),
                     (dict(rules=eg.AttentionRules(slopes=z(3, dtype=f32))), "slopes"),
                     (dict(rules=eg.AttentionRules(doc_starts=z(2, dtype=i32))), "doc_starts"),
                     (dict(rules=eg.AttentionRules(prefix_lens=z(1, dtype=i32))), "prefix_lens")):
        with pytest.raises(ValueError, match=what):
            chunk(**kw)
    for kw, what in ((dict(ws=ws[:-1]), "workspace_bytes"), (dict(ws=None), "workspace"), (dict(q=z(3, 3, 64)), "multiple of kv_heads"),
                     (dict(rules=eg.AttentionRules(window=-1)), "window"), (dict(rules=eg.AttentionRules(cap=float("nan"))), "cap")):
        with pytest.raises(eg.EngramError, match=what):
            chunk(**kw)
    with pytest.raises(TypeError, match="GPU"):
        chunk(q=torch.zeros(3, 4, 64, dtype=torch.int16))
    shared = lambda **kw: eg.engram_shared_prefix_attention(  # noqa: E731
        cache, q, kw.get("cu", z(2, dtype=i32)), kw.get("prefix", z(1, 2, dtype=i32)), z(1, dtype=i32), 9,
        kw.get("table", z(3, 2, dtype=i32)), z(3, dtype=i32), 9, 1.0, out, ws)
    for kw, what in ((dict(cu=z(3, dtype=i32)), "prefix_table"), (dict(table=z(2, 2, dtype=i32)), "table")):
        with pytest.raises(ValueError, match=what):
            shared(**kw)
    weights = lambda w, lse: eg.engram_cache_weights(cache, q, cu, table, lens, 9, 1.0, lse, w)  # noqa: E731
    with pytest.raises(ValueError, match="weights must be"):
        weights(z(2, 2, 8, dtype=f32), z(3, 4, dtype=f32))
    with pytest.raises(ValueError, match="lse"):
        weights(z(2, 2, 9, dtype=f32), z(3, 3, dtype=f32))
    with pytest.raises(eg.EngramError, match="lse or weights"):
        weights(z(2, 2, 9, dtype=f32), None)
    evict = lambda **kw: eg.engram_cache_evict(  # noqa: E731
        cache, table, lens, 9, kw.get("keep", 4), kw.get("sinks", 1), 1, z(2, 2, 9, dtype=f32), kw.get("to", z(2, 1, dtype=i32)),
        z(2, dtype=i32), kw.get("new_w", z(2, 2, 20, dtype=f32)), kw.get("kept", z(2, 2, 20, dtype=i32)))
    evict()
    for kw, what in ((dict(keep=9), "to_width"), (dict(sinks=4), "sinks"), (dict(keep=-1), "sinks")):
        with pytest.raises(eg.EngramError, match=what):
            evict(**kw)
    for kw, what in ((dict(new_w=z(2, 2, 3, dtype=f32)), "new_weights"), (dict(kept=z(2, 2, 3, dtype=i32)), "kept"),
                     (dict(to=z(1, 1, dtype=i32)), "to_table")):
        with pytest.raises(ValueError, match=what):
            evict(**kw)
