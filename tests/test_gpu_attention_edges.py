"""The attention step's operators where a rounding, an infinity or the split of the work could show, on the GPU.

Against oracle/attention.py (float64), with the bounds of tests/test_gpu_attention.py (u = 2^-24 of fp32, h = 2^-8
the half step of bf16) but for the softmax's weights: held as the sum of two bf16 values, of which the second has at
most 2^-7 of the whole, they are off by 2^-7 h = 2^-15.
"""

import numpy as np
import pytest

import oracle
from oracle import attention as oa
from test_gpu_attention import (H, U, Guarded, bits, check_attention, dev, eg, host, make_cache,  # noqa: F401 (eg: a fixture)
                                rope_inputs, step, step_state, within)

pytestmark = pytest.mark.gpu


class Call:
    """One call of the attention: a cache of unrelated pages, lengths, queries; its outputs checked on request."""

    def __init__(self, eg, rng, fmt, ps, hq, hkv, D, lens, window=0, sharp=2.0, width=None):
        lens = np.asarray(lens, np.int32)
        n, self.max_len = len(lens), int(lens.max())
        width = max(1, -(-self.max_len // ps))
        need = -(-lens // ps)
        self.arrays, self.held, self.cache = make_cache(eg, rng, fmt, int(need.sum()) + 1, hkv, ps, D)
        perm = rng.permutation(int(need.sum()) + 1)
        table = np.full((n, width), -1, np.int32)
        table[np.arange(width) < need[:, None]] = perm[:need.sum()]
        self.q, self.table, self.lens, self.window, self.scale = bits(sharp * rng.normal(size=(n, hq, D))), table, lens, window, D ** -0.5
        self.on_gpu = [dev(a) for a in (self.q, table, lens)]
        self.out, self.lse = (n, hq, D), (n, hq)
        self.bytes = eg.engram_paged_attention_workspace_bytes(n, hq, hkv, D, self.max_len)
        self.eg = eg

    def run(self):
        import torch
        out, lse = Guarded(self.out, torch.int16), Guarded(self.lse, torch.float32)
        ws, bad = Guarded((self.bytes,), torch.uint8), torch.zeros(1, dtype=torch.int32, device="cuda")
        self.eg.engram_paged_attention(self.cache, *self.on_gpu, self.max_len, self.scale, out.t, ws.t,
                                       window=self.window, lse=lse.t, bad_pages=bad)
        ws.host()
        assert bad.item() == 0
        return out.host(), lse.host()

    def check(self, out, lse):
        D = self.q.shape[2]
        want, want_lse, spread, logit = oa.paged_attention(*self.arrays, self.q, self.table, self.lens, self.max_len,
                                                           self.scale, self.window)
        d = D * U * logit
        within(out, want, H * np.abs(want) + (2.0 ** -15 + 2 * d + 2.0 ** -18)[..., None] * spread + 1e-30)
        empty = np.isneginf(want_lse)
        assert np.array_equal(empty, np.isneginf(lse)) and not out[empty].any()
        got, ref = lse[~empty].astype(np.float64), want_lse[~empty]
        tol = d[~empty] + (self.max_len / 32 + 32) * U + 4 * U * np.abs(ref)
        assert np.all(np.abs(got - ref) <= tol), np.max(np.abs(got - ref) / tol)


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
@pytest.mark.parametrize("hq,hkv,D,lens", [(8, 2, 32, [500, 130, 1]), (20, 1, 32, [700, 33]), (3, 1, 96, [3000]),
                                           (32, 8, 128, [400, 129]), (32, 1, 256, [200, 1500])])
def test_paged_attention_weights_are_not_rounded_to_bf16(eg, fmt, hq, hkv, D, lens):
    """Nearly equal weights over many values: results small against the values, so that weights in 8 bits would show."""
    call = Call(eg, np.random.default_rng(D + hq), fmt, 16, hq, hkv, D, lens, sharp=0.1)
    call.check(*call.run())


def run_pieces(call, hkv, head_blocks):
    """Whole or partial (sequence, heads) pairs of each of the 256 runs, as the call deals them out."""
    units = np.repeat(-(-call.lens // 128), hkv * head_blocks)
    per = max(1, -(-int(units.sum()) // 256))
    ends = np.cumsum(units)
    held = units > 0
    first, last = (ends - units)[held] // per, (ends - 1)[held] // per
    return np.bincount(np.concatenate([np.arange(a, b + 1) for a, b in zip(first, last)]))


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
@pytest.mark.parametrize("hq,hkv,D", [(70, 1, 64), (71, 1, 32), (40, 1, 96), (66, 2, 64), (64, 1, 64), (47, 1, 96)])
def test_paged_attention_runs_of_blocks_of_differing_heads(eg, fmt, hq, hkv, D):
    """Runs of many pieces whose blocks have 32 query heads, then a few: pieces shorter than a workgroup's four
    tiles beside long ones.  The same bits every time."""
    rng = np.random.default_rng(hq + D)
    lens = np.concatenate([rng.integers(1, 128, size=25), rng.integers(0, 32, size=15), rng.integers(900, 2000, size=20)])
    call = Call(eg, rng, fmt, 16, hq, hkv, D, rng.permutation(lens))
    blocks = -(-hq // hkv // 32)
    assert call.bytes > 0 and run_pieces(call, hkv, blocks).max() > 2
    out, lse = call.run()
    call.check(out, lse)
    for _ in range(4):
        again = call.run()
        assert np.array_equal(out, again[0]) and np.array_equal(lse, again[1])


@pytest.mark.parametrize("fmt,hq,hkv,D,n,top", [("mxfp8", 3, 1, 32, 700, 2300), ("bf16", 4, 2, 64, 300, 2100),
                                                ("mxfp8", 2, 2, 32, 513, 2500)])
def test_paged_attention_many_sequences_dealt_out_in_runs(eg, fmt, hq, hkv, D, n, top):
    """More sequences than a workgroup has threads, split over their length: several of them a thread's, empty ones
    at the ends of its span and whole spans of them among them."""
    rng = np.random.default_rng(n)
    lens = rng.integers(0, top // 2, size=n)
    lens[rng.random(n) < 0.2] = 0
    per_thread = -(-n // 256)
    lens[:per_thread] = 0                                     # the first thread's
    lens[5 * per_thread - 1:5 * per_thread + 1] = 0           # one thread's last, another's first
    lens[20 * per_thread:21 * per_thread] = 0
    lens[[-1, n // 2]] = [0, top]
    call = Call(eg, rng, fmt, 8, hq, hkv, D, lens)
    assert call.bytes > 0
    call.check(*call.run())


# ---------------------------------------------------------------- norm and rotation

@pytest.mark.parametrize("hq,hkv", [((1 << 20) + 650, 2), (33, (1 << 20) + 650)])
def test_qk_norm_rope_of_a_million_heads(eg, hq, hkv):
    """A row whose passes times its waves pass 32 bits."""
    import torch
    T, D = 1, 32
    row, qkv, qw, kw, pos, inv = rope_inputs(np.random.default_rng(hkv), T, hq, hkv, D, D, 0, 5000)
    q, k = Guarded((T, hq, D), torch.int16), Guarded((T, hkv, D), torch.int16)
    eg.engram_qk_norm_rope(qkv, hq, hkv, D, dev(qw), dev(kw), 1e-6, dev(pos), dev(inv), False, q.t, k.t)
    x = row.reshape(T, -1, D)
    for got, first, n, w in ((q.host(), 0, hq, qw), (k.host(), hq, hkv, kw)):
        for h in range(0, n, 1 << 18):
            want, mag = oa.qk_norm_rope(x[:, first + h:first + min(n, h + (1 << 18))], w, 1e-6, pos, inv, False)
            within(got[:, h:h + (1 << 18)], want, H * np.abs(want) + 2.0 ** -20 * mag + 1e-38)


@pytest.mark.parametrize("hq,hkv", [(2, 2), (32, 8)])
@pytest.mark.parametrize("inter", [False, True])
def test_qk_norm_rope_infinity_spoils_its_own_pair_only(eg, hq, hkv, inter):
    """An infinity makes its head's mean infinite and all finite values 0: NaN is left of it, and of its partner
    where it is rotated."""
    import torch
    rng = np.random.default_rng(3)
    T, D, rot = 4, 64, 32
    row, qkv, qw, kw, pos, inv = rope_inputs(rng, T, hq, hkv, D, rot, 0, 1000)
    x = row.reshape(T, -1, D)
    for t, d in ((0, 40), (1, 63), (2, 5), (3, 32)):
        x[t, :, d] = 0x7F80 if t % 2 else 0xFF80
    qkv = dev(row)
    q, k = Guarded((T, hq, D), torch.int16), Guarded((T, hkv, D), torch.int16)
    eg.engram_qk_norm_rope(qkv, hq, hkv, D, dev(qw), dev(kw), 1e-6, dev(pos), dev(inv), inter, q.t, k.t)
    for got, xs, w in ((q, x[:, :hq], qw), (k, x[:, hq:hq + hkv], kw)):
        with np.errstate(invalid="ignore"):
            want, _ = oa.qk_norm_rope(xs, w, 1e-6, pos, inv, inter)
        value = oracle.bf16_value(got.host())
        assert np.array_equal(np.isnan(want), np.isnan(value))
        assert not value[~np.isnan(want)].any() and not want[~np.isnan(want)].any()


def test_qk_norm_rope_keys_are_fp64_results_rounded_to_fp32_and_bf16(eg):
    """Of 4 M keys, some 30 have an fp32 rounding half-way between two bf16 values: it goes to the even one."""
    import torch
    T, hq, hkv, D = 4096, 1, 8, 128
    row, qkv, qw, kw, pos, inv = rope_inputs(np.random.default_rng(4), T, hq, hkv, D, D, 0, 4000)
    q, k = Guarded((T, hq, D), torch.int16), Guarded((T, hkv, D), torch.int16)
    eg.engram_qk_norm_rope(qkv, hq, hkv, D, dev(qw), dev(kw), 1e-6, dev(pos), dev(inv), False, q.t, k.t)
    x = row.reshape(T, -1, D)[:, hq:hq + hkv]
    want, mag = oa.qk_norm_rope(x, kw, 1e-6, pos, inv, False)
    # The two fp64 computations are off by less than 2^-34 of their terms (angles of up to 4000 and a series
    # to 2^-41): what is nearer to a border than that may go either way.
    twice = [bits((want + e * mag).astype(np.float32)) for e in (-2.0 ** -34, 0.0, 2.0 ** -34)]
    sure = (twice[0] == twice[2]) & (np.abs(want) > 1e-30)
    assert sure.mean() > 0.999
    assert (sure & (twice[1] != bits(want))).sum() > 10          # there are such
    wrong = sure & (k.host() != twice[1])
    assert not wrong.any(), int(wrong.sum())


# ---------------------------------------------------------------- the operators together

def test_step_with_lse(eg):
    """The decode step's attention with its own log-sum-exp."""
    import torch
    s = step_state(eg)
    step(eg, s)
    out, lse = Guarded(s["att"].shape, torch.int16), Guarded(s["att"].shape[:2], torch.float32)
    eg.engram_paged_attention(s["cache"], s["q"], s["table"], s["lens"], 48, 0.125, out.t, s["ws"], lse=lse.t)
    assert np.array_equal(out.host(), host(s["att"]))
    check_attention(out.host(), lse.host(), [g.host() for g in s["held"]], host(s["q"]), host(s["table"]),
                    host(s["lens"]), 48, 0.125, 0)


def test_engram_stages_with_a_4_bit_wkv(eg):
    """Hash, rows, 4-bit projection and gate of the tiny workload: kv against the oracle's product of the same rows
    and weight, and the highway what the gate makes of that kv."""
    import torch

    import workloads
    from workloads.device import to_device
    wl = workloads.make_workload(0)
    sp, d = wl.spec, to_device(wl, "cuda")
    layer = d.layers[0]
    params, tokens = eg.HashParams.from_dict(wl.hash_params), eg.Tokens(d.cids, d.cu_seqlens)
    codes, scales = Guarded((sp.N, sp.K // 2), torch.uint8), Guarded((sp.N, sp.K // 32), torch.uint8)
    eg.engram_quantize_mxfp4(layer.wkv, sp.N, sp.K, codes.t, scales.t)
    ids = torch.empty(sp.T, sp.cols, dtype=torch.int32, device="cuda")
    rows, kv = Guarded((sp.T, sp.K), torch.int16), Guarded((sp.T, sp.N), torch.int16)
    eg.engram_hash(params, tokens, ids)
    eg.engram_rows(eg.ENGRAM_ROWS_Q2K, layer.table, None, sp.num_rows, ids, sp.cols, sp.cols, sp.T, rows.t)
    eg.engram_project_mxfp4(rows.t, codes.t, scales.t, kv.t, sp.T, sp.K, sp.N)
    h = d.h.clone()
    eg.engram_gate(h, kv.t, layer.q_weight, layer.k_weight, None, sp.T, sp.hc, sp.dim, sp.eps, sp.clamp, sp.dot_scale)
    want_codes, want_scales = oa.quantize_mxfp4(wl.layers[0].wkv)
    assert np.array_equal(codes.host(), want_codes) and np.array_equal(scales.host(), want_scales)
    want, mag = oa.project_mxfp4(rows.host(), want_codes, want_scales)
    within(kv.host(), want, H * np.abs(want) + sp.K * U * mag)
    want_h, a = oracle.gate(wl.h, kv.host(), wl.layers[0].q_weight, wl.layers[0].k_weight, None, sp.eps, sp.clamp,
                            sp.dot_scale, return_preact=True)
    # The bounds of the gate's own tests: 1e-2, and 1e-4 away from the steep part of its signed square root.
    err = np.abs(h.cpu().numpy() - want_h) / np.maximum(1.0, np.abs(want_h))
    assert err.max() <= 1e-2 and err[np.abs(a) > 1e-2].max() <= 1e-4


@pytest.mark.parametrize("kind", ["bf16", "mxfp8"])
def test_example_decodes_the_same_in_a_graph(eg, kind):
    """Five decode steps, the last four replayed: the bits of five eager ones."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "attention_step.py")
    spec = importlib.util.spec_from_file_location("attention_step", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    (a, worst), (b, _) = (mod.generate(5, kind, graph) for graph in (True, False))
    assert worst <= 4 * H and int(a.m.bad) == 0
    for name in ("cids", "h", "q", "att", "lse"):
        assert np.array_equal(host(getattr(a, name)), host(getattr(b, name))), name
    for name in ("history", "live"):
        assert np.array_equal(host(getattr(a.m, name)), host(getattr(b.m, name))), name
    with pytest.raises(ValueError, match="places"):
        mod.generate(1000, kind)
