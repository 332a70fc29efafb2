"""A prompt and a few decode steps through one layer's Engram forward and attention step.

    python examples/attention_step.py [--steps 4] [--cache mxfp8]

Two streams share a paged cache.  Their prompts go in as one chunk (norm and rotation
of queries and keys, keys and values into the cache); each decode step then runs, on the
streams' newest tokens: the Engram forward in place on the highway, the 4-bit QKV
projection, norm and rotation into the cache, paged attention, and the 4-bit output
projection added to the highway.  The decode step is captured into a HIP graph once and
replayed.  After the last step the attention is checked against a plain computation on
the context read back out of the cache.
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


def run(steps=4, kind="mxfp8", verbose=True):
    torch.cuda.set_device(0)
    g = torch.Generator(device="cuda").manual_seed(0)
    n = len(PROMPTS)
    wl = workloads.make_workload(0)                 # a small Engram layer; its first n tokens are used
    spec, dev = wl.spec, to_device(wl, torch.device("cuda"))
    hc, dim = spec.hc, spec.dim
    params = eg.HashParams.from_dict(wl.hash_params)
    layers = [eg.Layer(eg.ENGRAM_ROWS_Q2K, ly.table, ly.scales, ly.wkv, ly.q_weight, ly.k_weight, hc, dim, spec.cols)
              for ly in dev.layers]
    tokens = eg.Tokens(dev.cids[:n].contiguous(), torch.arange(n + 1, dtype=torch.int32, device="cuda"))
    engram_ws = zeros(eg.engram_workspace_bytes(n, 1, spec.cols, hc, dim), dtype=torch.uint8)

    wqkv, wo = fp4_weight(g, WIDTH, dim), fp4_weight(g, dim, Q_HEADS * HEAD_DIM)
    q_weight, k_weight = (bits(1 + 0.1 * torch.randn(HEAD_DIM, generator=g, device="cuda")) for _ in range(2))
    half = torch.arange(HEAD_DIM // 2, dtype=torch.float64, device="cuda")
    inv_freq = 10000.0 ** (-2.0 * half / HEAD_DIM)
    cache = make_cache(kind)
    # Stream s owns every n-th page; slot_of[s, p] is the cache slot of its place p.
    table = torch.arange(PAGES, dtype=torch.int32, device="cuda").view(-1, n).t().contiguous()
    slot_of = (table.long()[:, :, None] * PAGE + torch.arange(PAGE, device="cuda")).flatten(1)

    # The prompts, one chunk of tokens: keys and values go straight into the cache.
    T = sum(PROMPTS)
    x = bits(torch.randn(T, dim, generator=g, device="cuda"))
    qkv, q = zeros(T, WIDTH), zeros(T, Q_HEADS, HEAD_DIM)
    eg.engram_project_mxfp4(x, *wqkv, qkv, T, dim, WIDTH)
    positions = torch.cat([torch.arange(p, dtype=torch.int32, device="cuda") for p in PROMPTS])
    slots = torch.cat([slot_of[s, :p] for s, p in enumerate(PROMPTS)])
    bad = zeros(1, dtype=torch.int32)
    eg.engram_qk_norm_rope(qkv, Q_HEADS, KV_HEADS, HEAD_DIM, q_weight, k_weight, EPS, positions, inv_freq, False, q,
                           cache=cache, slots=slots, bad_slots=bad)

    # One decode step; everything it reads and writes stays where it is, for the graph.
    lens = torch.tensor(PROMPTS, dtype=torch.int32, device="cuda")
    h = torch.randn(n, hc, dim, generator=g, device="cuda")
    qkv, q, att, y = zeros(n, WIDTH), zeros(n, Q_HEADS, HEAD_DIM), zeros(n, Q_HEADS, HEAD_DIM), zeros(n, dim)
    x, pos, slot, lse = zeros(n, dim), zeros(n, dtype=torch.int32), zeros(n, dtype=torch.int64), \
        zeros(n, Q_HEADS, dtype=torch.float32)
    ws = zeros(eg.engram_paged_attention_workspace_bytes(n, Q_HEADS, KV_HEADS, HEAD_DIM, MAX_LEN), dtype=torch.uint8)

    def step():
        pos.copy_(lens)
        slot.copy_(slot_of.gather(1, lens.long()[:, None])[:, 0])
        lens.add_(1)
        eg.engram_forward(params, tokens, layers, h, hc, dim, spec.eps, spec.clamp, spec.dot_scale, engram_ws)
        x.copy_(bits(h[:, 0]))
        eg.engram_project_mxfp4(x, *wqkv, qkv, n, dim, WIDTH)
        eg.engram_qk_norm_rope(qkv, Q_HEADS, KV_HEADS, HEAD_DIM, q_weight, k_weight, EPS, pos, inv_freq, False, q,
                               cache=cache, slots=slot, bad_slots=bad)
        eg.engram_paged_attention(cache, q, table, lens, MAX_LEN, SCALE, att, ws, lse=lse, bad_pages=bad)
        eg.engram_project_mxfp4(att, *wo, y, n, Q_HEADS * HEAD_DIM, dim)
        h.add_(y.view(torch.bfloat16).float()[:, None])

    step()                                          # once eagerly, then from the graph
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    for _ in range(steps - 1):
        graph.replay()
    torch.cuda.synchronize()

    worst = 0.0
    for s in range(n):
        length = int(lens[s])
        k, v = (zeros(length, KV_HEADS, HEAD_DIM) for _ in range(2))
        eg.engram_cache_read(cache, slot_of[s, :length].contiguous(), k, v, bad)
        kf, vf = (t.view(torch.bfloat16).double().repeat_interleave(Q_HEADS // KV_HEADS, 1) for t in (k, v))
        z = (q[s].view(torch.bfloat16).double() * kf).sum(-1) * SCALE        # [length, heads]
        want = (torch.softmax(z, 0)[..., None] * vf).sum(0)
        worst = max(worst, float((att[s].view(torch.bfloat16).double() - want).abs().max() / want.abs().max()))
    if verbose:
        print(f"{steps} decode steps of {n} streams, lengths {lens.tolist()}, {kind} cache: "
              f"attention off by {worst:.1e} of its largest value, {int(bad)} bad slots or pages")
    return worst, int(bad), lens.tolist()


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=4)
    ap.add_argument("--cache", choices=("bf16", "mxfp8"), default="mxfp8")
    a = ap.parse_args()
    worst, bad, _ = run(a.steps, a.cache)
    sys.exit(0 if worst < 1e-2 and bad == 0 else 1)
