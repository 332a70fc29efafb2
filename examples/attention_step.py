"""Two streams' prompts and a few decode steps through one layer: Engram forward and attention step.

    python examples/attention_step.py [--steps 4] [--cache mxfp8]

The streams share a paged cache.  A pass takes some tokens of each stream through the
layer: the Engram forward in place on the highway, a norm, the 4-bit QKV projection, norm
and rotation of queries and keys, keys and values into the cache, paged attention, and the
4-bit output projection added to the highway.  The prompts go through it at once, each
token attending to its stream's places up to its own (as a sequence of one new token each);
then each decode step takes every stream's next token, the lookback store carrying the ids
before it.  The decode step is captured into a HIP graph once and replayed.  After the
prompts and after the last step the attention is checked against a plain computation on
the context read back out of the cache.  Weights, embeddings and token ids are random.
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import gram_hash_memory_amd as eg  # noqa: E402
import workloads  # noqa: E402
from workloads.device import to_device  # noqa: E402

Q_HEADS, KV_HEADS, HEAD_DIM, PAGE, PAGES = 8, 2, 64, 16, 16
EPS, SCALE = 1e-6, HEAD_DIM ** -0.5
PROMPTS = (37, 21)                                  # tokens of each stream's prompt
MAX_LEN = PAGES // len(PROMPTS) * PAGE
WIDTH = (Q_HEADS + 2 * KV_HEADS) * HEAD_DIM


def bits(x):
    return x.to(torch.bfloat16).view(torch.int16)


def zeros(*shape, dtype=torch.int16):
    return torch.zeros(*shape, dtype=dtype, device="cuda")


def fp4_weight(g, n, k):
    """A random weight [n, k], quantised once as a program does when it loads one."""
    w = bits(torch.randn(n, k, generator=g, device="cuda") / k ** 0.5)
    codes, scales = zeros(n, k // 2, dtype=torch.uint8), zeros(n, k // 32, dtype=torch.uint8)
    eg.engram_quantize_mxfp4(w, n, k, codes, scales)
    return codes, scales


def make_cache(kind):
    shape = (PAGES, KV_HEADS, PAGE, HEAD_DIM)
    if kind == "bf16":
        return eg.KVCache(eg.ENGRAM_CACHE_BF16, zeros(*shape), zeros(*shape))
    u8 = torch.uint8
    scales = [torch.full((*shape[:3], HEAD_DIM // 32), 127, dtype=u8, device="cuda") for _ in range(2)]
    return eg.KVCache(eg.ENGRAM_CACHE_MXFP8, zeros(*shape, dtype=u8), zeros(*shape, dtype=u8), *scales)


class Model:
    """One layer's weights, the streams' ids (of every place they may reach) and their pages."""

    def __init__(self, kind):
        g = torch.Generator(device="cuda").manual_seed(0)
        n = len(PROMPTS)
        wl = workloads.make_workload(0)             # a small Engram layer
        self.spec, dev = wl.spec, to_device(wl, torch.device("cuda"))
        hc, dim = self.spec.hc, self.spec.dim
        self.params = eg.HashParams.from_dict(wl.hash_params)
        self.layers = [eg.Layer(eg.ENGRAM_ROWS_Q2K, ly.table, ly.scales, ly.wkv, ly.q_weight, ly.k_weight, hc, dim,
                                self.spec.cols) for ly in dev.layers]
        self.embed = torch.randn(self.spec.compressed_vocab, hc, dim, generator=g, device="cuda")
        self.ids = torch.randint(0, self.spec.compressed_vocab, (n, MAX_LEN), generator=g, device="cuda",
                                 dtype=torch.int32)
        self.wqkv, self.wo = fp4_weight(g, WIDTH, dim), fp4_weight(g, dim, Q_HEADS * HEAD_DIM)
        self.q_weight, self.k_weight = (bits(1 + 0.1 * torch.randn(HEAD_DIM, generator=g, device="cuda"))
                                        for _ in range(2))
        half = torch.arange(HEAD_DIM // 2, dtype=torch.float64, device="cuda")
        self.inv_freq = 10000.0 ** (-2.0 * half / HEAD_DIM)
        self.cache = make_cache(kind)
        # Stream s owns every n-th page; slot_of[s, p] is the cache slot of its place p.
        self.table = torch.arange(PAGES, dtype=torch.int32, device="cuda").view(-1, n).t().contiguous()
        self.slot_of = (self.table.long()[:, :, None] * PAGE + torch.arange(PAGE, device="cuda")).flatten(1)
        depth = self.spec.max_ngram - 1             # the ids before a stream's next token
        self.history, self.live = zeros(n, depth, dtype=torch.int32), zeros(n, depth, dtype=torch.uint8)
        self.bad = zeros(1, dtype=torch.int32)


class Pass:
    """The layer on T tokens; stream[i] is token i's stream.  What it reads and writes stays where it is."""

    def __init__(self, m, stream, cu_seqlens, positions):
        T, hc, dim = len(stream), m.spec.hc, m.spec.dim
        self.m, self.T, self.stream, self.positions = m, T, stream, positions
        self.cids = zeros(T, dtype=torch.int32)
        self.tokens = eg.Tokens(self.cids, cu_seqlens, lookback=m.history, lookback_live=m.live)
        self.engram_ws = zeros(eg.engram_workspace_bytes(T, 1, m.spec.cols, hc, dim), dtype=torch.uint8)
        self.h = zeros(T, hc, dim, dtype=torch.float32)
        self.qkv, self.q, self.att = zeros(T, WIDTH), zeros(T, Q_HEADS, HEAD_DIM), zeros(T, Q_HEADS, HEAD_DIM)
        self.y, self.lse = zeros(T, dim), zeros(T, Q_HEADS, dtype=torch.float32)
        self.table = m.table[stream].contiguous()   # a row for each token
        self.ws = zeros(eg.engram_paged_attention_workspace_bytes(T, Q_HEADS, KV_HEADS, HEAD_DIM, MAX_LEN),
                        dtype=torch.uint8)

    def run(self):
        m, T, dim = self.m, self.T, self.m.spec.dim
        self.cids.copy_(m.ids[self.stream, self.positions.long()])
        self.h.copy_(m.embed[self.cids.long()])
        eg.engram_forward(m.params, self.tokens, m.layers, self.h, m.spec.hc, dim, m.spec.eps, m.spec.clamp,
                          m.spec.dot_scale, self.engram_ws)
        eg.engram_history_update(self.tokens, m.history, m.live)
        x = self.h.mean(1)
        x = bits(x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS))
        eg.engram_project_mxfp4(x, *m.wqkv, self.qkv, T, dim, WIDTH)
        slots = m.slot_of[self.stream, self.positions.long()]
        eg.engram_qk_norm_rope(self.qkv, Q_HEADS, KV_HEADS, HEAD_DIM, m.q_weight, m.k_weight, EPS, self.positions,
                               m.inv_freq, False, self.q, cache=m.cache, slots=slots, bad_slots=m.bad)
        eg.engram_paged_attention(m.cache, self.q, self.table, self.positions + 1, MAX_LEN, SCALE, self.att, self.ws,
                                  lse=self.lse, bad_pages=m.bad)
        eg.engram_project_mxfp4(self.att, *m.wo, self.y, T, Q_HEADS * HEAD_DIM, dim)
        self.h.add_(self.y.view(torch.bfloat16).float()[:, None])

    def off(self):
        """How far the attention is from a plain one over the cache's places, relative to its largest value."""
        m, worst = self.m, 0.0
        for i, (s, p) in enumerate(zip(self.stream.tolist(), self.positions.tolist())):
            k, v = (zeros(p + 1, KV_HEADS, HEAD_DIM) for _ in range(2))
            eg.engram_cache_read(m.cache, m.slot_of[s, :p + 1].contiguous(), k, v, m.bad)
            k, v = (t.view(torch.bfloat16).double().repeat_interleave(Q_HEADS // KV_HEADS, 1) for t in (k, v))
            z = (self.q[i].view(torch.bfloat16).double() * k).sum(-1) * SCALE        # [p + 1, heads]
            want = (torch.softmax(z, 0)[..., None] * v).sum(0)
            got = self.att[i].view(torch.bfloat16).double()
            worst = max(worst, float((got - want).abs().max() / want.abs().max()))
        return worst


def generate(steps=4, kind="mxfp8", graph=True):
    """The prompts and `steps` decode steps: the decode pass after the last of them, and the largest error."""
    if max(PROMPTS) + steps > MAX_LEN:
        raise ValueError(f"a stream has {MAX_LEN} places: at most {MAX_LEN - max(PROMPTS)} steps")
    torch.cuda.set_device(0)
    m, n = Model(kind), len(PROMPTS)
    i32 = dict(dtype=torch.int32, device="cuda")
    ends = torch.tensor((0,) + PROMPTS, **i32).cumsum(0, dtype=torch.int32)
    stream = torch.repeat_interleave(torch.arange(n, device="cuda"), torch.tensor(PROMPTS, device="cuda"))
    prompt = Pass(m, stream, ends, torch.cat([torch.arange(p, **i32) for p in PROMPTS]))
    prompt.run()
    worst = prompt.off()

    decode = Pass(m, torch.arange(n, device="cuda"), torch.arange(n + 1, **i32), torch.tensor(PROMPTS, **i32) - 1)

    def step():
        decode.positions.add_(1)
        decode.run()

    step()                                          # once eagerly, then from the graph
    if graph:
        captured = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(captured):
            step()
    for _ in range(steps - 1):
        captured.replay() if graph else step()
    torch.cuda.synchronize()
    return decode, max(worst, decode.off())


def run(steps=4, kind="mxfp8", verbose=True):
    decode, worst = generate(steps, kind)
    lens, bad = (decode.positions + 1).tolist(), int(decode.m.bad)
    if verbose:
        print(f"{sum(PROMPTS)} prompt tokens and {steps} decode steps of {len(PROMPTS)} streams, lengths {lens}, "
              f"{kind} cache: attention off by {worst:.1e} of its largest value, {bad} bad slots or pages")
    return worst, bad, lens


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=4)
    ap.add_argument("--cache", choices=("bf16", "mxfp8"), default="mxfp8")
    a = ap.parse_args()
    worst, bad, _ = run(a.steps, a.cache)
    sys.exit(0 if worst < 1e-2 and bad == 0 else 1)
