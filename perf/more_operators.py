"""Cases of the paged cache's attention beyond one new token per sequence, and of what keeps the cache small.

Four operators over the paged cache (bf16, or 8 bits with a scale per 32 values):
  chunk    attention of several new tokens per sequence (a prompt, a chunk of one, a few drafted tokens, one token),
           with a window, a prefix that all of a sequence's tokens see, documents, capped scores, a distance bias;
  shared   attention of one new token per sequence, for sequences that share a long prefix;
  weights  the attention weight that each place of the cache gets from new tokens, added up;
  evict    the places of largest weight of each key-value head, copied to other pages.

bf16 tensors are held as int16 bit patterns, as everywhere in the package.
"""

import math

import numpy as np
import torch

own = False

NOTHING = 2 ** 31 - 1          # a token whose document begins here sees nothing (padding)


# ---------------------------------------------------------------- cases

def _heads(hq, hkv, D, fmt, page):
    return dict(q_heads=hq, kv_heads=hkv, head_dim=D, fmt=fmt, page_size=page)


def _chunk(name, seqs, new, old, heads, kind="chunk", window=0, prefix=0, doc_len=0, pad=0, cap=0.0, bias=False):
    """new, old: (least, most) new tokens and places before them of the sequences; prefix: places that all of a
    sequence's tokens see; doc_len: places of a document (0: one document); pad: tokens at each sequence's end that
    see nothing."""
    return dict(name=name, kind=kind, seqs=seqs, new_min=new[0], new_max=new[1], old_min=old[0], old_max=old[1],
                window=window, prefix=prefix, doc_len=doc_len, pad=pad, cap=cap, bias=bias, **heads)


def listed():
    return [
        # Two short prompts, each seen whole by its own tokens: latency.
        _chunk("chunk_prompts_21_37", 2, (21, 37), (0, 0), _heads(8, 2, 64, "mxfp8", 16), prefix=37),
        # A decode step of a model with capped scores and a distance bias: one token a stream.
        _chunk("chunk_64x1_after_4095", 64, (1, 1), (899, 4095), _heads(32, 8, 128, "mxfp8", 16), cap=30.0, bias=True),
        # A prefill batch of four sequences, packed documents of 512 tokens, a few padding tokens.
        _chunk("chunk_4x2048_documents", 4, (2048, 2048), (0, 0), _heads(32, 8, 128, "bf16", 16), doc_len=512, pad=9),
        # Capped scores and wide heads, ragged prompts.
        _chunk("chunk_3x1500_capped", 3, (700, 1500), (0, 300), _heads(16, 8, 256, "bf16", 64), window=1024, cap=50.0),
        # Chunked prefill: 2048 new tokens behind 14336 cached ones.
        _chunk("chunk_2048_after_14336", 1, (2048, 2048), (14336, 14336), _heads(32, 8, 128, "mxfp8", 16)),
        # Eight continuations of a short prompt: latency.
        dict(name="shared_8_of_500", kind="shared", groups=1, seqs=8, prefix=500, own_min=1, own_max=60,
             **_heads(32, 8, 128, "bf16", 16)),
        # 64 streams behind one long instruction, some of them just begun.
        dict(name="shared_64_of_8192", kind="shared", groups=1, seqs=64, prefix=8192, own_min=1, own_max=700,
             **_heads(32, 8, 128, "mxfp8", 16)),
        # Three documents of different lengths, 33 questions each.
        dict(name="shared_3x33_of_30000", kind="shared", groups=3, seqs=99, prefix=30000, own_min=5, own_max=200,
             **_heads(16, 4, 128, "bf16", 64)),
        # The decode batch's weights, a step at a time.
        _chunk("weights_64x1_after_4095", 64, (1, 1), (899, 4095), _heads(32, 8, 128, "mxfp8", 16), kind="weights"),
        # A prompt's last 64 tokens say which of its places are kept.
        _chunk("weights_64_after_16320", 1, (64, 64), (16320, 16320), _heads(32, 8, 128, "bf16", 16), kind="weights"),
        # Streams that have outgrown their room go back to it; some have not.
        dict(name="evict_16x4608_to_4096", kind="evict", seqs=16, len_min=3000, len_max=4608, keep=4096, sinks=4,
             recent=512, **_heads(8, 8, 128, "mxfp8", 16)),
        # A long prompt pruned once, before its decoding begins.
        dict(name="evict_1x32768_to_2048", kind="evict", seqs=1, len_min=32768, len_max=32768, keep=2048, sinks=4,
             recent=64, **_heads(8, 8, 128, "bf16", 16)),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["chunk", "chunk", "shared", "weights", "evict"])
    D = rng.choice([64, 96, 128, 192, 256])
    hkv = rng.choice([1, 2, 3, 4, 8])
    hq = hkv * rng.choice([1, 2, 3, 4, 6, 8])
    heads = _heads(hq, hkv, D, rng.choice(["bf16", "mxfp8"]), rng.choice([8, 16, 32, 64, 128]))
    places = 16 * 1024 * 1024 // (hkv * D)             # of all sequences: what the listed ones hold
    if kind == "evict":
        longest = _log(rng, 2, min(65536, places))
        n = max(1, min(_log(rng, 1, 32), places // longest))
        keep = rng.randint(1, longest)
        sinks = min(keep, rng.randint(0, 16))
        return dict(kind=kind, seqs=n, len_min=rng.randint(1, longest), len_max=longest, keep=keep, sinks=sinks,
                    recent=rng.randint(0, (keep - sinks + 1) // 2), **heads)
    if kind == "shared":
        prefix = _log(rng, 1, min(32768, places // 2))
        groups = max(1, min(rng.randint(1, 4), places // 2 // prefix))
        n = max(groups, _log(rng, 2, 128))
        n = max(groups, min(n, 128 * 1024 * 1024 // (hq * prefix)))
        most = _log(rng, 1, max(1, min(2000, places // 2 // n)))
        return dict(kind=kind, groups=groups, seqs=n, prefix=prefix, own_min=rng.randint(0, most), own_max=most, **heads)
    new = _log(rng, 1, 2048) if kind == "chunk" else _log(rng, 1, 128)
    old = rng.choice([0, _log(rng, 1, 16384)])
    old = max(0, min(old, places // 2 - new))
    # The (padded) scores' number, and the products with them, stay below the largest listed case's.
    n = max(1, min(_log(rng, 1, 64), places // 2 // (new + old), 2 ** 30 // (hq * new * (new + old)),
                   2 ** 37 // (hq * new * (new + old) * D)))
    new = max(1, min(new, 2 ** 30 // (hq * (new + old)), 2 ** 37 // (hq * (new + old) * D)))
    case = _chunk("", n, (rng.randint(1, new), new), (rng.randint(0, old), old), heads, kind,
                  window=rng.choice([0, 0, _log(rng, 1, new + old)]), prefix=rng.choice([0, 0, rng.randint(1, new + old)]),
                  doc_len=rng.choice([0, 0, _log(rng, 1, new + old)]), pad=rng.choice([0, 0, rng.randint(0, min(9, new - 1))]),
                  cap=rng.choice([0.0, 0.0, rng.uniform(5.0, 60.0)]), bias=rng.random() < 0.4)
    del case["name"]
    return case


def _spread(n, lo, hi):
    """n whole numbers, evenly from lo to hi (hi alone for one)."""
    return np.array([hi if n == 1 else lo + (hi - lo) * i // (n - 1) for i in range(n)], dtype=np.int64)


def _shape(case):
    """New tokens and lengths of a chunk's or a step's sequences; the longest contexts with the fewest new tokens."""
    new = _spread(case["seqs"], case["new_min"], case["new_max"])
    return new, new + _spread(case["seqs"], case["old_min"], case["old_max"])[::-1]


def _members(case):
    """Sequences of each group, the first one's being the fewest."""
    cuts = [case["seqs"] * i // case["groups"] for i in range(case["groups"] + 1)]
    return np.array(cuts, dtype=np.int64)


# ---------------------------------------------------------------- what is in hand before a call

def _bits(x):
    return x.to(torch.bfloat16).view(torch.int16)


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _int32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _cache(case, g, pages):
    """A filled paged cache: heads of a page side by side, [pages][heads][page_size][head_dim]."""
    shape = (pages, case["kv_heads"], case["page_size"], case["head_dim"])
    c = {"fmt": case["fmt"]}
    for n in ("k", "v"):
        x = _normal(g, *shape)
        if case["fmt"] == "bf16":
            c[n], c[n + "_scales"] = _bits(x), None
        else:
            codes, scales = _to_mx(x.to(torch.bfloat16).float())
            c[n], c[n + "_scales"] = codes.view(torch.uint8), scales
    return c


def _tables(g, case, *lengths):
    """Page tables for lists of lengths, of unrelated pages, unused entries -1; and the number of pages."""
    ps = case["page_size"]
    need = [-(-np.asarray(x) // ps) for x in lengths]
    total = max(1, int(sum(x.sum() for x in need)))
    perm = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    tables, at = [], 0
    for x in need:
        width = max(1, int(x.max()))
        used = torch.from_numpy(np.arange(width)[None] < x[:, None]).cuda()
        t = torch.full((len(x), width), -1, dtype=torch.int32, device="cuda")
        t[used] = perm[at:at + int(x.sum())]
        at += int(x.sum())
        tables.append(t)
    return tables, total


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    kind, D, hq, hkv = case["kind"], case["head_dim"], case["q_heads"], case["kv_heads"]
    s = {"case": case, "handle": None, "workspace": None, "rules": None, "scale": 1.0 / math.sqrt(D)}
    if kind == "evict":
        lens = _spread(case["seqs"], case["len_min"], case["len_max"])
        kept = np.minimum(lens, case["keep"])
        (s["table"], s["to_table"]), pages = _tables(g, case, lens, kept)
        s.update(cache=_cache(case, g, pages), lens=_int32(lens), max_len=int(lens.max()))
        # Weights as attention leaves them: few places with much, equal ones among the rest.
        w = torch.exp(2.0 * _normal(g, case["seqs"], hkv, s["max_len"]) - 6.0)
        s["weights"] = torch.where(w < 5e-4, torch.zeros_like(w), w)
        s["new_lens"] = torch.empty_like(s["lens"])
        s["new_weights"] = torch.empty(case["seqs"], hkv, case["keep"], dtype=torch.float32, device="cuda")
        s["kept"] = torch.empty(case["seqs"], hkv, case["keep"], dtype=torch.int32, device="cuda")
        return s
    n = case["seqs"]
    if kind == "shared":
        lens = _spread(n, case["own_min"], case["own_max"])
        prefixes = _spread(case["groups"], max(1, case["prefix"] // 2), case["prefix"])
        (s["table"], s["prefix_table"]), pages = _tables(g, case, lens, prefixes)
        s.update(lens=_int32(lens), prefix_lens=_int32(prefixes), cu_groups=_int32(_members(case)), T=n,
                 max_len=int(lens.max()), max_prefix=int(prefixes.max()))
    else:
        new, lens = _shape(case)
        cu = np.concatenate([[0], np.cumsum(new)])
        (s["table"],), pages = _tables(g, case, lens)
        s.update(lens=_int32(lens), cu_seqlens=_int32(cu), T=int(cu[-1]), max_len=int(lens.max()),
                 slopes=None, doc_starts=None, prefix_lens=None)
        if case["bias"]:
            s["slopes"] = 2.0 ** (-8.0 * (torch.arange(hq, device="cuda", dtype=torch.float32) + 1) / hq)
        if case["prefix"]:
            s["prefix_lens"] = _int32(np.minimum(lens, case["prefix"]))
        if case["doc_len"] or case["pad"]:
            s["doc_starts"] = _int32(np.concatenate(_doc_starts(case, new, lens)))
    s["cache"] = _cache(case, g, pages)
    # Queries that single out some keys: logits of a spread of about 2.
    s["q"] = _bits(2.0 * _normal(g, s["T"], hq, D))
    if kind == "weights":
        s["lse"] = _chunk_lse(s, case)
        s["weights"] = torch.zeros(n, hkv, s["max_len"], dtype=torch.float32, device="cuda")
        return s
    s["out"] = torch.empty(s["T"], hq, D, dtype=torch.int16, device="cuda")
    s["lse"] = torch.empty(s["T"], hq, dtype=torch.float32, device="cuda")
    return s


def _doc_starts(case, new, lens):
    """For each sequence, where the document of each of its new tokens begins."""
    got = []
    for n, length in zip(new, lens):
        pos = np.arange(length - n, length)
        start = pos // case["doc_len"] * case["doc_len"] if case["doc_len"] else np.zeros_like(pos)
        start[n - min(n, case["pad"]):] = NOTHING
        got.append(start)
    return got


# ---------------------------------------------------------------- the plain forms

def _to_mx(x):
    """e4m3fn codes and e8m0 bytes of x [..., D]: per 32 values the smallest power of two that takes their
    largest magnitude to 448 or below."""
    b = x.unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1, keepdim=True)
    m, e = torch.frexp(amax)                             # amax = m 2^e, m in [1/2, 1)
    e = (e - 9 + (m > 0.875)).clamp(32 - 127, 127)
    e = torch.where(amax > 0, e, torch.zeros_like(e))
    codes = torch.ldexp(b, -e).to(torch.float8_e4m3fn)
    return codes.flatten(-2), (e.squeeze(-1) + 127).to(torch.uint8)


def _float(bits):
    return bits.view(torch.bfloat16).float()


def _places(s, name, table, count):
    """The first `count` places of every row of the table, in 32 bits: [rows, heads, count, D]."""
    c = s["cache"]
    ps = c[name].shape[2]
    at = torch.arange(count, device="cuda")
    page = table.long().clamp(min=0)[:, at // ps]                                # [rows, count]
    x = c[name][page, :, at % ps]                                                # [rows, count, heads, D]
    if c["fmt"] == "bf16":
        x = _float(x)
    else:
        e = c[name + "_scales"][page, :, at % ps].to(torch.int32) - 127
        x = torch.ldexp(x.view(torch.float8_e4m3fn).float().unflatten(-1, (-1, 32)), e[..., None]).flatten(-2)
    return x.transpose(1, 2).contiguous()


def _chunk_scores(s, case):
    """Scores [seqs, kv heads, group, new, places] of the sequences' tokens, -infinity where a place is not seen; and
    which (sequence, token) each token is."""
    n, hkv, D = case["seqs"], case["kv_heads"], case["head_dim"]
    group, lens, L = case["q_heads"] // hkv, s["lens"].long(), s["max_len"]
    first = s["cu_seqlens"].long()
    count = first[1:] - first[:-1]
    i = torch.arange(case["new_max"], device="cuda")
    token = (first[:-1, None] + i).clamp(max=s["T"] - 1)                         # [n, new], past a sequence's end any
    q = _float(s["q"])[token].unflatten(2, (hkv, group)).permute(0, 2, 3, 1, 4)  # [n, hkv, group, new, D]
    k = _places(s, "k", s["table"], L)
    z = (q.flatten(2, 3) @ k.transpose(-1, -2)).unflatten(2, (group, -1)) * s["scale"]
    if case["cap"]:
        z = case["cap"] * torch.tanh(z / case["cap"])
    p = torch.arange(L, device="cuda")
    pos = (lens - count)[:, None, None] + i[None, :, None]                       # [n, new, 1]
    if s["slopes"] is not None:
        z = z - s["slopes"].view(hkv, group, 1, 1) * (pos - p).abs()[:, None, None]
    seen = p <= pos
    if case["window"]:
        seen = seen & (pos - p < case["window"])
    if s["prefix_lens"] is not None:
        seen = seen | (p < s["prefix_lens"].long()[:, None, None])
    seen = seen & (p < lens[:, None, None])
    if s["doc_starts"] is not None:
        seen = seen & (p >= s["doc_starts"].long()[token][..., None])
    which = (i < count[:, None]).nonzero(as_tuple=True)
    return z.masked_fill_(~seen[:, None, None], -math.inf), which


def _softmax(z, v):
    """out and lse of scores [..., rows, places], values [..., places, D]; 0 and -infinity where nothing is seen."""
    top = z.amax(-1, keepdim=True).clamp(min=-3e38)
    p = torch.exp(z - top)
    total = p.sum(-1, keepdim=True)
    return (p @ v) / total.clamp(min=1e-30), (torch.log(total) + top).squeeze(-1)


def _chunk_lse(s, case):
    z, (seq, tok) = _chunk_scores(s, case)
    top = z.amax(-1).clamp(min=-3e38)
    lse = torch.log(torch.exp(z - top[..., None]).sum(-1)) + top                 # [n, hkv, group, new]
    return lse.permute(0, 3, 1, 2)[seq, tok].flatten(1).contiguous()


def _attend_chunk(s, case):
    z, (seq, tok) = _chunk_scores(s, case)
    group, new = z.shape[2], z.shape[3]
    out, lse = _softmax(z.flatten(2, 3), _places(s, "v", s["table"], s["max_len"]))
    out = out.unflatten(2, (group, new)).permute(0, 3, 1, 2, 4)[seq, tok]        # [T, hkv, group, D]
    lse = lse.unflatten(2, (group, new)).permute(0, 3, 1, 2)[seq, tok]
    return {"out": out.flatten(1, 2).to(torch.bfloat16), "lse": lse.flatten(1)}


def _attend_shared(s, case):
    """Every sequence's own places and its group's, side by side."""
    n, hkv, D = case["seqs"], case["kv_heads"], case["head_dim"]
    L, P, group = s["max_len"], s["max_prefix"], case["q_heads"] // hkv
    of = torch.bucketize(torch.arange(n, device="cuda"), s["cu_groups"][1:].long(), right=True)   # a sequence's group
    q = _float(s["q"]).view(n, hkv, group, D)
    if L:
        own_z = (q @ _places(s, "k", s["table"], L).transpose(-1, -2)) * s["scale"]
        unseen = torch.arange(L, device="cuda") >= s["lens"].long()[:, None]
        own_z.masked_fill_(unseen[:, None, None], -math.inf)
    else:
        own_z = q.new_zeros(n, hkv, group, 0)
    k, v = (_places(s, m, s["prefix_table"], P) for m in ("k", "v"))             # [groups, hkv, P, D]
    unseen = torch.arange(P, device="cuda") >= s["prefix_lens"].long()[of, None]
    # The scores against every group's prefix, of which a sequence takes its own group's.
    flat = q.permute(1, 0, 2, 3).flatten(1, 2)                                   # [hkv, n * group, D]
    every = (flat[None] @ k.transpose(-1, -2)).unflatten(2, (n, group)).permute(2, 0, 1, 3, 4)
    shared_z = every[torch.arange(n, device="cuda"), of] * s["scale"]            # [n, hkv, group, P]
    shared_z = shared_z.masked_fill(unseen[:, None, None], -math.inf)
    z = torch.cat([shared_z, own_z], -1)
    top = z.amax(-1, keepdim=True).clamp(min=-3e38)
    p = torch.exp(z - top)
    total = p.sum(-1, keepdim=True)
    weight = p[..., :P].permute(1, 0, 2, 3)                                      # [hkv, n, group, P]
    mine = (of[:, None] == torch.arange(case["groups"], device="cuda")).float().t()          # [groups, n]
    out = (weight[None] * mine[:, None, :, None, None]).flatten(2, 3) @ v        # [groups, hkv, n * group, D]
    out = out.sum(0).unflatten(1, (n, group)).transpose(0, 1)
    if L:
        out = out + p[..., P:] @ _places(s, "v", s["table"], L)
    out = out / total.clamp(min=1e-30)
    lse = (torch.log(total) + top).squeeze(-1)
    return {"out": out.flatten(1, 2).to(torch.bfloat16), "lse": lse.flatten(1)}


def _add_weights(s, case):
    z, (seq, tok) = _chunk_scores(s, case)
    n, hkv, group, new, L = z.shape
    # A padded token's log-sum-exp: +infinity, so that it weighs nothing; so does one that sees nothing.
    lse = torch.full((n, new, hkv * group), math.inf, device="cuda")
    lse[seq, tok] = torch.where(s["lse"] == -math.inf, math.inf, s["lse"])
    lse = lse.unflatten(2, (hkv, group)).permute(0, 2, 3, 1)
    s["weights"] += torch.exp(z - lse[..., None]).sum((2, 3))
    return {"weights": s["weights"]}


def _evict(s, case):
    n, hkv, keep = case["seqs"], case["kv_heads"], case["keep"]
    ps, L = case["page_size"], s["max_len"]
    lens = s["lens"].long()
    p = torch.arange(L, device="cuda")
    # Sinks and recent places above all weights, what is no place below them; ties by the place.
    rank = s["weights"].masked_fill((p < case["sinks"]) | (p >= (lens - case["recent"])[:, None, None]), math.inf)
    rank = rank.masked_fill((p >= lens[:, None])[:, None], -math.inf)
    order = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., :keep]
    count = lens.clamp(max=keep)
    order = order.masked_fill(torch.arange(order.shape[-1], device="cuda") >= count[:, None, None], NOTHING)
    kept = torch.sort(order, -1).values
    kept = torch.cat([kept, kept.new_full((n, hkv, keep - kept.shape[-1]), NOTHING)], -1)
    used = kept != NOTHING
    seq, head, i = used.nonzero(as_tuple=True)
    at = kept[used]
    page, to = s["table"].long()[seq, at // ps], s["to_table"].long()[seq, i // ps]
    c = s["cache"]
    for name in ("k", "v", "k_scales", "v_scales"):
        if c[name] is not None:
            c[name][to, head, i % ps] = c[name][page, head, at % ps]
    s["kept"].copy_(torch.where(used, kept, torch.full_like(kept, -1)))
    s["new_weights"].zero_()
    s["new_weights"][used] = s["weights"][seq, head, at]
    s["new_lens"].copy_(count)
    return _evicted(s)


def _evicted(s):
    got = {"kept": s["kept"], "new_lens": s["new_lens"], "new_weights": s["new_weights"]}
    for name in ("k", "v"):
        if s["cache"]["fmt"] == "bf16":
            got[name] = s["cache"][name].view(torch.bfloat16)
        else:
            got[name] = s["cache"][name].view(torch.float8_e4m3fn)
            got[name + "_scales"] = s["cache"][name + "_scales"].view(torch.float8_e8m0fnu)
    return got


def run(s):
    case = s["case"]
    if own:
        return _run_own(s, case)
    return {"chunk": _attend_chunk, "shared": _attend_shared, "weights": _add_weights, "evict": _evict}[case["kind"]](s, case)


# ---------------------------------------------------------------- the framework's calls

def _handle(s, eg):
    if s["handle"] is None:
        c = s["cache"]
        fmt = eg.ENGRAM_CACHE_BF16 if c["fmt"] == "bf16" else eg.ENGRAM_CACHE_MXFP8
        s["handle"] = eg.KVCache(fmt, c["k"], c["v"], c["k_scales"], c["v_scales"])
    return s["handle"]


def _rules(s, case, eg):
    if s["rules"] is None:
        s["rules"] = eg.AttentionRules(window=case["window"], cap=case["cap"], slopes=s["slopes"],
                                       doc_starts=s["doc_starts"], prefix_lens=s["prefix_lens"])
    return s["rules"]


def _workspace(s, size):
    if s["workspace"] is None:
        s["workspace"] = torch.empty(size(), dtype=torch.uint8, device="cuda")
    return s["workspace"]


def _run_own(s, case):
    import gram_hash_memory_amd as eg
    kind, hq, hkv, D = case["kind"], case["q_heads"], case["kv_heads"], case["head_dim"]
    cache = _handle(s, eg)
    if kind == "evict":
        eg.engram_cache_evict(cache, s["table"], s["lens"], s["max_len"], case["keep"], case["sinks"], case["recent"],
                              s["weights"], s["to_table"], s["new_lens"], s["new_weights"], s["kept"])
        return _evicted(s)
    if kind == "weights":
        eg.engram_cache_weights(cache, s["q"], s["cu_seqlens"], s["table"], s["lens"], s["max_len"], s["scale"],
                                s["lse"], s["weights"], rules=_rules(s, case, eg))
        return {"weights": s["weights"]}
    if kind == "shared":
        ws = _workspace(s, lambda: eg.engram_shared_prefix_attention_workspace_bytes(
            case["seqs"], case["groups"], hq, hkv, D, s["max_prefix"], s["max_len"]))
        eg.engram_shared_prefix_attention(cache, s["q"], s["cu_groups"], s["prefix_table"], s["prefix_lens"],
                                          s["max_prefix"], s["table"], s["lens"], s["max_len"], s["scale"], s["out"],
                                          ws, lse=s["lse"])
    else:
        ws = _workspace(s, lambda: eg.engram_chunk_attention_workspace_bytes(
            s["T"], case["seqs"], hq, hkv, D, s["max_len"]))
        eg.engram_chunk_attention(cache, s["q"], s["cu_seqlens"], s["table"], s["lens"], s["max_len"], s["scale"],
                                  s["out"], ws, rules=_rules(s, case, eg), lse=s["lse"])
    return {"out": s["out"].view(torch.bfloat16), "lse": s["lse"]}


# ---------------------------------------------------------------- what a pass cannot do without

def _seen(case):
    """Of a chunk's or a step's sequences: pairs of a token and a place that it sees, and places that any token sees."""
    pairs = places = 0
    new, lens = _shape(case)
    starts = _doc_starts(case, new, lens)
    for n, length, start in zip(new, lens, starts):
        pos = np.arange(length - n, length)
        lo = np.maximum(start, 0 if not case["window"] else np.maximum(0, pos - case["window"] + 1))
        end = min(length, case["prefix"])
        # Places from lo to pos, and those of the prefix from the document's start on that these leave out.
        mine = np.maximum(0, pos + 1 - lo)
        more = np.maximum(0, np.minimum(end, lo) - np.minimum(start, end)) + np.maximum(0, end - np.maximum(pos + 1, start))
        pairs += int((mine + more).sum())
        some = mine + more > 0
        if some.any():
            low = int(np.where(start < end, start, lo)[some].min())
            places += int(max(pos[some].max() + 1, end) - low)
    return pairs, places


def work(case):
    kind, hq, hkv, D = case["kind"], case["q_heads"], case["kv_heads"], case["head_dim"]
    held = {"bf16": 2 * D, "mxfp8": D + D // 32}[case["fmt"]]                    # of one key or value
    ps = case["page_size"]
    if kind == "evict":
        lens = _spread(case["seqs"], case["len_min"], case["len_max"])
        kept = int(np.minimum(lens, case["keep"]).sum())
        table = 4 * int((-(-lens // ps)).sum())
        return {"bytes": 4 * hkv * int(lens.sum()) + kept * hkv * 4 * held + table + 8 * case["seqs"] * hkv * case["keep"], "flops": 0}
    if kind == "shared":
        prefixes = _spread(case["groups"], max(1, case["prefix"] // 2), case["prefix"])
        own_lens = _spread(case["seqs"], case["own_min"], case["own_max"])
        pairs = int((np.diff(_members(case)) * prefixes).sum() + own_lens.sum())
        places = int(prefixes.sum() + own_lens.sum())
        return {"bytes": places * hkv * 2 * held + 4 * (places // ps) + case["seqs"] * hq * (4 * D + 4), "flops": 4 * D * pairs * hq}
    pairs, places = _seen(case)
    tokens = int(_shape(case)[0].sum())
    if kind == "weights":
        return {"bytes": places * hkv * (held + 8) + 4 * (places // ps) + tokens * hq * (2 * D + 4), "flops": 2 * D * pairs * hq}
    return {"bytes": places * hkv * 2 * held + 4 * (places // ps) + tokens * hq * (4 * D + 4), "flops": 4 * D * pairs * hq}


# ---------------------------------------------------------------- the definition in 64 bits

def _exact_row(s, name, table_row, at):
    """Places `at` of one sequence, float64 [heads, places, D]."""
    c = s["cache"]
    ps = c[name].shape[2]
    page, offset = table_row.long()[at // ps], at % ps
    x = c[name][page, :, offset].contiguous()
    if c["fmt"] == "bf16":
        x = x.view(torch.bfloat16).double()
    else:
        unit = torch.exp2(c[name + "_scales"][page, :, offset].double() - 127)
        x = x.view(torch.float8_e4m3fn).double() * unit.repeat_interleave(32, dim=-1)
    return x.transpose(0, 1).contiguous()


def _exact_logits(s, case, i, h, k):
    """Scores of sequence i's tokens for query head h over keys k [places, D], and which are seen."""
    first, last = (int(x) for x in s["cu_seqlens"][i:i + 2])
    length = int(s["lens"][i])
    z = s["q"][first:last, h].contiguous().view(torch.bfloat16).double() @ k.t().contiguous() * s["scale"]
    if case["cap"]:
        e = torch.exp(2.0 * z / case["cap"])
        z = case["cap"] * (e - 1.0) / (e + 1.0)
    place = torch.arange(length, device="cuda")
    pos = torch.arange(length - (last - first), length, device="cuda")[:, None]
    if s["slopes"] is not None:
        z = z - s["slopes"][h].double() * (place - pos).abs()
    back = pos - place
    seen = (back >= 0) & ((back < case["window"]) if case["window"] else True)
    if s["prefix_lens"] is not None:
        seen = seen | (place < int(s["prefix_lens"][i]))
    if s["doc_starts"] is not None:
        seen = seen & (place >= s["doc_starts"][first:last].long()[:, None])
    return z, seen


def exact(case, seed):
    s = prepare(case, seed)
    kind, hq, hkv, D = case["kind"], case["q_heads"], case["kv_heads"], case["head_dim"]
    group, f64 = hq // hkv, dict(dtype=torch.float64, device="cuda")
    if kind == "evict":
        return _exact_evict(s, case)
    if kind == "weights":
        w = torch.zeros(s["weights"].shape, **f64)
        for i, length in enumerate(s["lens"].tolist()):
            k = _exact_row(s, "k", s["table"][i], torch.arange(length, device="cuda"))
            first, last = (int(x) for x in s["cu_seqlens"][i:i + 2])
            for h in range(hq):
                z, seen = _exact_logits(s, case, i, h, k[h // group])
                e = torch.exp(z - s["lse"][first:last, h, None].double())
                w[i, h // group, :length] += torch.where(seen, e, torch.zeros_like(e)).sum(0)
        return {"weights": w}
    out = torch.zeros(s["T"], hq, D, **f64)
    lse = torch.full((s["T"], hq), -math.inf, **f64)
    if kind == "chunk":
        for i, length in enumerate(s["lens"].tolist()):
            at = torch.arange(length, device="cuda")
            k, v = (_exact_row(s, m, s["table"][i], at) for m in ("k", "v"))
            first, last = (int(x) for x in s["cu_seqlens"][i:i + 2])
            for h in range(hq):
                z, seen = _exact_logits(s, case, i, h, k[h // group])
                z = torch.where(seen, z, torch.full_like(z, -math.inf))
                lse[first:last, h] = torch.logsumexp(z, -1)
                p = torch.softmax(z, -1)
                out[first:last, h] = torch.where(seen.any(-1, keepdim=True), p, torch.zeros_like(p)) @ v[h // group]
        return {"out": out, "lse": lse}
    cuts = s["cu_groups"].tolist()
    for m in range(case["groups"]):
        at = torch.arange(int(s["prefix_lens"][m]), device="cuda")
        shared = [_exact_row(s, name, s["prefix_table"][m], at) for name in ("k", "v")]
        for i in range(cuts[m], cuts[m + 1]):
            mine = [_exact_row(s, name, s["table"][i], torch.arange(int(s["lens"][i]), device="cuda")) for name in ("k", "v")]
            k, v = (torch.cat(x, 1) for x in zip(shared, mine))
            q = s["q"][i].view(torch.bfloat16).double().view(hkv, group, D)
            z = torch.bmm(q, k.transpose(1, 2).contiguous()) * s["scale"]
            lse[i] = torch.logsumexp(z, -1).flatten()
            out[i] = torch.bmm(torch.softmax(z, -1), v).flatten(0, 1)
    return {"out": out, "lse": lse}


def _exact_evict(s, case):
    ps, keep, c = case["page_size"], case["keep"], s["cache"]
    weights = s["weights"].cpu().numpy()
    got = {"kept": None, "new_lens": None}
    moved = np.zeros(s["new_weights"].shape)
    src, dst = [], []                                        # (page, head, place in it)
    table, to_table = s["table"].cpu().numpy(), s["to_table"].cpu().numpy()
    for i, length in enumerate(s["lens"].tolist()):
        for h in range(case["kv_heads"]):
            every = np.arange(length)
            if length > keep:
                middle = every[case["sinks"]:length - case["recent"]]
                best = middle[np.lexsort((middle, -weights[i, h][middle].astype(np.float64)))]
                best = best[:keep - case["sinks"] - case["recent"]]
                every = np.sort(np.concatenate([every[:case["sinks"]], best, every[length - case["recent"]:]]))
            moved[i, h, :len(every)] = weights[i, h][every]
            to = np.arange(len(every))
            src.append(np.stack([table[i][every // ps], np.full_like(every, h), every % ps]))
            dst.append(np.stack([to_table[i][to // ps], np.full_like(to, h), to % ps]))
    got["new_weights"] = torch.from_numpy(moved)
    src, dst = (torch.from_numpy(np.concatenate(x, 1)).long().cuda() for x in (src, dst))
    for name, x in c.items():
        if name == "fmt" or x is None:
            continue
        if name.endswith("_scales"):
            x = torch.exp2(x.double() - 127)
        else:
            x = x.view(torch.bfloat16 if c["fmt"] == "bf16" else torch.float8_e4m3fn).double()
        x[dst[0], dst[1], dst[2]] = x[src[0], src[1], src[2]]
        got[name] = x
    return got
