"""Cases of the decoder layer's attention step that a streaming program runs beside the Engram forward.

Five kinds of pass, over four operators:
  norm_rope  the per-head RMS norm of queries and keys and their rotation, out of one row of the QKV projection;
  chunk      the same for a chunk of a sequence, its keys and values going into the paged cache in the same call,
             and the whole context read back in bf16 (what chunked prefill attends to);
  cache      keys and values written to the paged cache (quantised there) and a context read back;
  attend     attention of one new token per sequence over the paged cache;
  project    the product of few tokens with a 4-bit weight (e2m1 codes, one e8m0 scale per 32 values).

bf16 tensors are held as int16 bit patterns, as everywhere in the package.
"""

import math

import torch

own = False

EPS = 1e-6


# ---------------------------------------------------------------- cases

def _rope(name, kind, T, hq, hkv, D, rot, inter, pad, far, **more):
    return dict(name=name, kind=kind, T=T, q_heads=hq, kv_heads=hkv, head_dim=D, rotary_dim=rot,
                interleaved=inter, pad=pad, far=far, **more)


def listed():
    return [
        # One decode step of 64 streams: the call's latency.
        _rope("norm_rope_decode_64", "norm_rope", 64, 32, 8, 128, 128, False, 0, 32768),
        # A prefill batch of 8192 tokens.
        _rope("norm_rope_prefill_8192", "norm_rope", 8192, 32, 8, 128, 128, False, 0, 32768),
        # A short prompt's tail behind a cached prefix: few tokens, narrow heads, half of each rotated in pairs.
        _rope("chunk_17_after_239", "chunk", 17, 12, 4, 64, 32, True, 8, 1000, prefix=239,
              fmt="mxfp8", page_size=16),
        # Chunked prefill: 2048 new tokens behind 14336 cached ones, in 8 bits.
        _rope("chunk_2048_after_14336", "chunk", 2048, 32, 8, 128, 128, False, 0, 200000,
              prefix=14336, fmt="mxfp8", page_size=16),
        # Odd sizes with an unquantised cache: 333 tokens written, 5000 read.
        dict(name="cache_bf16_333_5000", kind="cache", T=333, read=5000, kv_heads=4, head_dim=96,
             pad=40, fmt="bf16", page_size=32),
        # A prefill's keys and values into an 8-bit cache, and a long context out of it.
        dict(name="cache_mxfp8_8192_32768", kind="cache", T=8192, read=32768, kv_heads=8,
             head_dim=128, pad=0, fmt="mxfp8", page_size=16),
        # One stream with a short context: latency.
        dict(name="attend_1x500_bf16", kind="attend", seqs=1, max_len=500, min_len=500, empty=0,
             q_heads=32, kv_heads=8, head_dim=128, fmt="bf16", page_size=16, window=0),
        # The decode batch: 64 ragged streams over an 8-bit cache, three of them without a context.
        dict(name="attend_64x4096_mxfp8", kind="attend", seqs=64, max_len=4096, min_len=900,
             empty=3, q_heads=32, kv_heads=8, head_dim=128, fmt="mxfp8", page_size=16, window=0),
        # One stream with a very long context.
        dict(name="attend_1x131072_bf16", kind="attend", seqs=1, max_len=131072, min_len=131072,
             empty=0, q_heads=32, kv_heads=8, head_dim=128, fmt="bf16", page_size=64, window=0),
        # One token through a layer's QKV projection: the smallest product.
        dict(name="project_1_4096_6144", kind="project", T=1, K=4096, N=6144),
        # The decode workload's wkv projection at 4 bits.
        dict(name="project_64_6144_20480", kind="project", T=64, K=6144, N=20480),
        # An odd batch through the output projection.
        dict(name="project_101_4096_4096", kind="project", T=101, K=4096, N=4096),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["norm_rope", "chunk", "cache", "attend", "project"])
    if kind == "project":
        return dict(kind=kind, T=_log(rng, 1, 128), K=32 * _log(rng, 4, 192), N=_log(rng, 64, 20480))
    D = rng.choice([64, 96, 128, 192, 256])
    hkv = rng.choice([1, 2, 3, 4, 8])
    fmt = rng.choice(["bf16", "mxfp8"])
    page = rng.choice([8, 16, 32, 64, 128])
    if kind == "attend":
        group = rng.choice([1, 2, 3, 4, 6, 8, 16, 32])
        most = 128 * 1024 * 1024 // (hkv * D)        # tokens, by the largest listed case's bytes
        longest = _log(rng, 1, min(131072, most))
        seqs = max(1, min(_log(rng, 1, 128), most // longest))
        return dict(kind=kind, seqs=seqs, max_len=longest, min_len=rng.randint(1, longest),
                    empty=rng.randint(0, min(2, seqs - 1)), q_heads=group * hkv, kv_heads=hkv,
                    head_dim=D, fmt=fmt, page_size=page,
                    window=rng.choice([0, 0, _log(rng, 1, longest)]))
    most = 64 * 1024 * 1024 // (hkv * D)             # tokens of keys or values
    if kind == "cache":
        return dict(kind=kind, T=min(_log(rng, 1, 8192), most // 4), read=min(_log(rng, 1, 32768), most // 2),
                    kv_heads=hkv, head_dim=D, pad=8 * rng.randint(0, 6), fmt=fmt, page_size=page)
    group = rng.choice([1, 2, 3, 4, 6, 8])
    T = min(_log(rng, 1, 8192 if kind == "norm_rope" else 2048),
            32 * 1024 * 1024 // ((group + 2) * hkv * D))
    case = _rope("", kind, T, group * hkv, hkv, D, rng.choice([D, D // 2]), rng.random() < 0.5,
                 8 * rng.randint(0, 6), _log(rng, 10000, 1000000))
    if kind == "chunk":
        case.update(prefix=min(_log(rng, 1, 16384), most // 4), fmt=fmt, page_size=page)
    del case["name"]
    return case


# ---------------------------------------------------------------- what is in hand before a call

def _bits(x):
    return x.to(torch.bfloat16).view(torch.int16)


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _lengths(case):
    """The sequences' lengths: spread evenly from min_len to max_len, the first `empty` of them 0."""
    n, lo, hi = case["seqs"], case["min_len"], case["max_len"]
    lens = [hi if n == 1 else lo + (hi - lo) * i // (n - 1) for i in range(n)]
    return [0] * case["empty"] + lens[case["empty"]:]


def _cache(case, g, pages, filled=True):
    """An empty or a filled paged cache: heads of a page side by side, [pages][heads][page_size][head_dim]."""
    shape = (pages, case["kv_heads"], case["page_size"], case["head_dim"])
    c = {"fmt": case["fmt"]}
    for n in ("k", "v"):
        if case["fmt"] == "bf16":
            c[n] = _bits(_normal(g, *shape)) if filled else torch.zeros(shape, dtype=torch.int16, device="cuda")
            c[n + "_scales"] = None
        elif filled:
            codes, scales = _to_mx(_normal(g, *shape).to(torch.bfloat16).float())
            c[n], c[n + "_scales"] = codes.view(torch.uint8), scales
        else:
            c[n] = torch.zeros(shape, dtype=torch.uint8, device="cuda")
            c[n + "_scales"] = torch.full(shape[:3] + (shape[3] // 32,), 127, dtype=torch.uint8, device="cuda")
    return c


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    if case["kind"] == "project":
        T, K, N = case["T"], case["K"], case["N"]
        # A trained weight's spread: sigma 1/sqrt(K), rows of differing size.
        w = _normal(g, N, K) * (0.5 + torch.rand(N, 1, generator=g, device="cuda")) / math.sqrt(K)
        s["codes"], s["scales"] = _to_fp4(w)
        s["x"] = _bits(_normal(g, T, K))
        s["out"] = torch.empty(T, N, dtype=torch.int16, device="cuda")
        return s
    D, hkv = case["head_dim"], case["kv_heads"]
    if case["kind"] == "attend":
        n, ps = case["seqs"], case["page_size"]
        order = torch.randperm(n, generator=g, device="cuda").cpu()
        lens = torch.tensor(_lengths(case), dtype=torch.int32)[order]
        need = (lens + ps - 1) // ps
        width, total = max(1, int(need.max())), max(1, int(need.sum()))
        perm = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
        used = torch.arange(width)[None] < need[:, None]
        table = torch.full((n, width), -1, dtype=torch.int32, device="cuda")
        table[used.cuda()] = perm[: int(need.sum())]
        s.update(cache=_cache(case, g, total), table=table, lens=lens.cuda(), scale=1.0 / math.sqrt(D))
        # Queries that single out some keys: logits of a spread of about 2.
        s["q"] = _bits(2.0 * _normal(g, n, case["q_heads"], D))
        s["out"] = torch.empty(n, case["q_heads"], D, dtype=torch.int16, device="cuda")
        s["lse"] = torch.empty(n, case["q_heads"], dtype=torch.float32, device="cuda")
        s["handle"] = s["workspace"] = None
        return s
    T, ps = case["T"], case["page_size"] if "page_size" in case else 1
    width = (case.get("q_heads", 0) + 2 * hkv) * D
    row = _normal(g, T, width + case["pad"]) * (0.5 + 2 * torch.rand(T, 1, generator=g, device="cuda"))
    s["qkv"] = _bits(row)[:, :width]
    if case["kind"] != "cache":
        hq = case["q_heads"]
        s["q_weight"], s["k_weight"] = (_bits(1 + 0.2 * _normal(g, D)) for _ in range(2))
        first = int(torch.randint(0, case["far"], (1,), generator=g, device="cuda"))
        s["positions"] = torch.arange(first, first + T, dtype=torch.int32, device="cuda")
        if case["kind"] == "norm_rope":      # a batch of unrelated streams
            s["positions"] = torch.randint(0, case["far"], (T,), generator=g, device="cuda", dtype=torch.int32)
        half = torch.arange(case["rotary_dim"] // 2, dtype=torch.float64, device="cuda")
        s["inv_freq"] = 10000.0 ** (-2.0 * half / case["rotary_dim"])
        s["q"] = torch.empty(T, hq, D, dtype=torch.int16, device="cuda")
        if case["kind"] == "norm_rope":
            s["k"] = torch.empty(T, hkv, D, dtype=torch.int16, device="cuda")
            return s
    context = case["prefix"] + T if case["kind"] == "chunk" else case["read"]
    tokens = max(context, T)
    pages = -(-tokens // ps) + 3
    perm = torch.randperm(pages, generator=g, device="cuda")
    at = torch.arange(tokens, device="cuda")
    slots = perm[at // ps] * ps + at % ps                # the tokens' places, in the sequence's order
    # The context's last tokens are the new ones (with a context shorter than them, their first ones are read).
    s["write"] = slots[tokens - T:].contiguous()
    s["read"] = slots[:context].contiguous()
    s["cache"] = _cache(case, g, pages)
    s["k_ctx"], s["v_ctx"] = (torch.empty(context, hkv, D, dtype=torch.int16, device="cuda") for _ in range(2))
    s["handle"] = None
    return s


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


def _of_mx(codes, scales):
    b = codes.view(torch.float8_e4m3fn).float().unflatten(-1, (-1, 32))
    return torch.ldexp(b, scales.to(torch.int32)[..., None] - 127).flatten(-2)


def _to_fp4(w):
    """OCP MXFP4 of w [N, K]: e2m1 codes, two a byte (even k low), and e8m0 bytes per 32 values."""
    b = w.to(torch.bfloat16).float().unflatten(-1, (-1, 32))
    _, e = torch.frexp(b.abs().amax(-1, keepdim=True))
    e = (e - 3).clamp(-127, 127)
    x = torch.ldexp(b, -e)
    a = x.abs()
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=w.device)
    code = (a[..., None] > mid).sum(-1)
    # Half-way values go to the even code: 0.75, 1.75 and 3.5 (to 2, 4 and 6) lie above an odd one.
    code = code + ((a == 0.75) | (a == 1.75) | (a == 3.5)).long()
    code = (code + 8 * (x < 0).long()).flatten(-2)
    return (code[:, 0::2] | (code[:, 1::2] << 4)).to(torch.uint8), (e.squeeze(-1) + 127).to(torch.uint8)


def _float(bits):
    return bits.view(torch.bfloat16).float()


def _norm(x, w):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w


def _rotate(x, positions, inv_freq, interleaved):
    rot = 2 * inv_freq.numel()
    angle = positions.double()[:, None, None] * inv_freq
    cos, sin = angle.cos().float(), angle.sin().float()
    r, rest = x[..., :rot], x[..., rot:]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else r.chunk(2, -1)
    y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1 if interleaved else -2)
    return torch.cat([y.flatten(-2), rest], -1)


def _norm_rope(s, case):
    hq, hkv, D = case["q_heads"], case["kv_heads"], case["head_dim"]
    x = _float(s["qkv"]).unflatten(-1, (-1, D))
    q = _rotate(_norm(x[:, :hq], _float(s["q_weight"])), s["positions"], s["inv_freq"], case["interleaved"])
    k = _rotate(_norm(x[:, hq:hq + hkv], _float(s["k_weight"])), s["positions"], s["inv_freq"], case["interleaved"])
    return q.to(torch.bfloat16), k.to(torch.bfloat16), s["qkv"].view(torch.bfloat16).unflatten(-1, (-1, D))[:, hq + hkv:]


def _put(cache, name, slots, x):
    ps = cache[name].shape[2]
    if cache["fmt"] == "bf16":
        cache[name][slots // ps, :, slots % ps] = x.view(torch.int16)
    else:
        codes, scales = _to_mx(x.float())
        cache[name][slots // ps, :, slots % ps] = codes.view(torch.uint8)
        cache[name + "_scales"][slots // ps, :, slots % ps] = scales


def _get(cache, name, slots):
    ps = cache[name].shape[2]
    x = cache[name][slots // ps, :, slots % ps]
    if cache["fmt"] == "bf16":
        return _float(x.contiguous())
    return _of_mx(x.contiguous(), cache[name + "_scales"][slots // ps, :, slots % ps])


def _attend(s, case):
    n, hq, D = s["q"].shape
    ps, hkv = case["page_size"], case["kv_heads"]
    at = torch.arange(int(s["table"].shape[1]) * ps, device="cuda")
    lens = s["lens"].long()[:, None]
    seen = at[None] < lens
    if case["window"]:
        seen = seen & (at[None] >= lens - case["window"])
    slots = s["table"].long().clamp(min=0)[:, at // ps] * ps + at % ps          # [n, L]
    k, v = (_get(s["cache"], name, slots.flatten()).unflatten(0, slots.shape).transpose(1, 2) for name in ("k", "v"))
    q = _float(s["q"]).view(n, hkv, hq // hkv, D)
    logits = (q @ k.transpose(-1, -2)) * s["scale"]                              # [n, hkv, group, L]
    logits = logits.masked_fill(~seen[:, None, None], -math.inf)
    top = logits.amax(-1, keepdim=True).clamp(min=-3e38)                         # finite where nothing is seen
    p = torch.exp(logits - top)
    total = p.sum(-1, keepdim=True)
    out = (p @ v) / total.clamp(min=1e-30)
    return out.view(n, hq, D).to(torch.bfloat16), (torch.log(total) + top).view(n, hq)


def _project(s):
    low, high = s["codes"] & 15, s["codes"] >> 4
    code = torch.stack([low, high], -1).flatten(-2).int()
    value = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], device="cuda")[code]
    w = torch.ldexp(value.unflatten(-1, (-1, 32)), s["scales"].int()[..., None] - 127).flatten(-2)
    return (_float(s["x"]) @ w.t()).to(torch.bfloat16)


def run(s):
    case = s["case"]
    kind = case["kind"]
    if own:
        return _run_own(s, case, kind)
    if kind == "project":
        return {"out": _project(s)}
    if kind == "attend":
        out, lse = _attend(s, case)
        return {"out": out, "lse": lse}
    got = {}
    if kind == "cache":
        k, v = s["qkv"].view(torch.bfloat16).unflatten(-1, (-1, case["head_dim"])).chunk(2, 1)
    else:
        got["q"], k, v = _norm_rope(s, case)
        if kind == "norm_rope":
            return {"q": got["q"], "k": k}
    _put(s["cache"], "k", s["write"], k)
    _put(s["cache"], "v", s["write"], v)
    got["k"], got["v"] = (_get(s["cache"], name, s["read"]).to(torch.bfloat16) for name in ("k", "v"))
    return got


# ---------------------------------------------------------------- the framework's calls

def _handle(s, eg):
    if s["handle"] is None:
        c = s["cache"]
        fmt = eg.ENGRAM_CACHE_BF16 if c["fmt"] == "bf16" else eg.ENGRAM_CACHE_MXFP8
        s["handle"] = eg.KVCache(fmt, c["k"], c["v"], c["k_scales"], c["v_scales"])
    return s["handle"]


def _run_own(s, case, kind):
    import gram_hash_memory_amd as eg
    bf16 = torch.bfloat16
    if kind == "project":
        eg.engram_project_mxfp4(s["x"], s["codes"], s["scales"], s["out"], case["T"], case["K"], case["N"])
        return {"out": s["out"].view(bf16)}
    D, hkv = case["head_dim"], case["kv_heads"]
    if kind == "attend":
        if s["workspace"] is None:
            s["workspace"] = torch.empty(eg.engram_paged_attention_workspace_bytes(
                case["seqs"], case["q_heads"], hkv, D, case["max_len"]), dtype=torch.uint8, device="cuda")
        eg.engram_paged_attention(_handle(s, eg), s["q"], s["table"], s["lens"], case["max_len"], s["scale"],
                                  s["out"], s["workspace"], window=case["window"], lse=s["lse"])
        return {"out": s["out"].view(bf16), "lse": s["lse"]}
    if kind == "cache":
        kv = s["qkv"].unflatten(-1, (-1, D))
        eg.engram_cache_write(_handle(s, eg), kv[:, :hkv], kv[:, hkv:], s["write"])
    else:
        fused = kind == "chunk"
        eg.engram_qk_norm_rope(s["qkv"], case["q_heads"], hkv, D, s["q_weight"], s["k_weight"], EPS, s["positions"],
                               s["inv_freq"], case["interleaved"], s["q"], None if fused else s["k"],
                               cache=_handle(s, eg) if fused else None, slots=s["write"] if fused else None)
        if not fused:
            return {"q": s["q"].view(bf16), "k": s["k"].view(bf16)}
    eg.engram_cache_read(_handle(s, eg), s["read"], s["k_ctx"], s["v_ctx"])
    got = {"k": s["k_ctx"].view(bf16), "v": s["v_ctx"].view(bf16)}
    if kind == "chunk":
        got["q"] = s["q"].view(bf16)
    return got


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    kind = case["kind"]
    if kind == "project":
        T, K, N = case["T"], case["K"], case["N"]
        return {"bytes": N * K / 2 + N * K / 32 + 2 * T * (K + N), "flops": 2 * T * K * N}
    D, hkv = case["head_dim"], case["kv_heads"]
    held = {"bf16": 2 * D, "mxfp8": D + D / 32}.get(case.get("fmt"), 0)          # of one key or value
    if kind == "attend":
        seen = [min(n, case["window"] or n) for n in _lengths(case)]
        pages = sum(-(-n // case["page_size"]) for n in seen)
        rows = case["seqs"] * case["q_heads"]
        return {"bytes": sum(seen) * hkv * 2 * held + 4 * pages + rows * (4 * D + 4), "flops": 4 * D * sum(seen) * case["q_heads"]}
    T = case["T"]
    if kind == "cache":
        return {"bytes": T * (hkv * 2 * (2 * D + held) + 8) + case["read"] * (hkv * 2 * (2 * D + held) + 8), "flops": 0}
    hq = case["q_heads"]
    rows = T * (hq + hkv)
    w = {"bytes": rows * 2 * D + T * (hq * 2 * D + 4) + 4 * D, "flops": rows * (5 * D + 3 * case["rotary_dim"])}
    if kind == "norm_rope":
        w["bytes"] += T * hkv * 2 * D
    else:
        w["bytes"] += T * (hkv * (2 * D + 2 * held) + 8) + (case["prefix"] + T) * (hkv * 2 * (2 * D + held) + 8)
    return w


# ---------------------------------------------------------------- the definition in 64 bits

def _exact_quantised(x):
    """What a cache in 8 bits holds for x (float64, bf16 values)."""
    b = x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    top = b.abs().max(dim=-1, keepdim=True).values
    e = torch.ceil(torch.log2(torch.where(top > 0, top, torch.ones_like(top)) / 448.0))
    # The logarithm's own rounding: one lower where that holds too, one higher where it does not.
    e = torch.where(top <= 448.0 * torch.exp2(e - 1), e - 1, e)
    e = torch.where(top > 448.0 * torch.exp2(e), e + 1, e)
    unit = torch.exp2(torch.where(top > 0, e, torch.zeros_like(e)).clamp(min=-95.0))
    y = b / unit
    lg = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6)))
    quantum = torch.exp2(lg.clamp(min=-6.0) - 3)
    return (torch.round(y / quantum) * quantum * unit).reshape(x.shape)


def _exact_cached(cache, name, page, offset):
    x = cache[name][page, :, offset]
    if cache["fmt"] == "bf16":
        return x.contiguous().view(torch.bfloat16).double()
    unit = torch.exp2(cache[name + "_scales"][page, :, offset].double() - 127)
    return x.contiguous().view(torch.float8_e4m3fn).double() * unit.repeat_interleave(32, dim=-1)


def _exact_norm_rope(s, case, first, heads, weight):
    D, rot = case["head_dim"], case["rotary_dim"]
    x = s["qkv"][:, first * D:(first + heads) * D].contiguous().view(torch.bfloat16).double().view(-1, heads, D)
    y = x / torch.sqrt((x * x).sum(-1, keepdim=True) / D + EPS) * weight.view(torch.bfloat16).double()
    z = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                    s["positions"].double()[:, None] * s["inv_freq"])[:, None]
    i = torch.arange(rot // 2, device="cuda")
    ia, ib = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + rot // 2)
    turned = torch.complex(y[..., ia], y[..., ib]) * z
    y = y.clone()
    y[..., ia], y[..., ib] = turned.real, turned.imag
    return y


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "project":
        lut = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
        T, K = s["x"].shape
        x = s["x"].view(torch.bfloat16).double()
        out = torch.empty(T, case["N"], dtype=torch.float64, device="cuda")
        for i in range(0, case["N"], 4096):
            c = s["codes"][i:i + 4096].long()
            w = torch.empty(c.shape[0], K, dtype=torch.float64, device="cuda")
            for j, nibble in ((0, c % 16), (1, c // 16)):
                w[:, j::2] = lut[nibble % 8] * (1 - 2 * (nibble // 8))
            w *= torch.exp2(s["scales"][i:i + 4096].double() - 127).repeat_interleave(32, dim=1)
            out[:, i:i + 4096] = x @ w.t().contiguous()
        return {"out": out}
    D, hkv = case["head_dim"], case["kv_heads"]
    if kind == "attend":
        group = case["q_heads"] // hkv
        out = torch.zeros(case["seqs"], case["q_heads"], D, dtype=torch.float64, device="cuda")
        lse = torch.full((case["seqs"], case["q_heads"]), -math.inf, dtype=torch.float64, device="cuda")
        q = s["q"].view(torch.bfloat16).double()
        for i, n in enumerate(s["lens"].tolist()):
            t = torch.arange(max(0, n - case["window"]) if case["window"] else 0, n, device="cuda")
            if not len(t):
                continue
            page = s["table"][i].long()[t // case["page_size"]]
            k, v = (_exact_cached(s["cache"], m, page, t % case["page_size"]) for m in ("k", "v"))
            for h in range(hkv):
                rows = slice(h * group, (h + 1) * group)
                z = q[i, rows] @ k[:, h].t().contiguous() * s["scale"]
                lse[i, rows] = torch.logsumexp(z, -1)
                out[i, rows] = torch.softmax(z, -1) @ v[:, h].contiguous()
        return {"out": out, "lse": lse}
    got = {}
    if kind == "cache":
        new = s["qkv"].contiguous().view(torch.bfloat16).double().view(case["T"], 2, hkv, D)
        new = {"k": new[:, 0], "v": new[:, 1]}
    else:
        hq = case["q_heads"]
        got["q"] = _exact_norm_rope(s, case, 0, hq, s["q_weight"])
        k = _exact_norm_rope(s, case, hq, hkv, s["k_weight"])
        if kind == "norm_rope":
            return {"q": got["q"], "k": k}
        new = {"k": k if case["fmt"] == "bf16" else k.float().to(torch.bfloat16).double(),
               "v": s["qkv"][:, (hq + hkv) * D:].contiguous().view(torch.bfloat16).double().view(-1, hkv, D)}
    ps = case["page_size"]
    where = torch.full((int(s["cache"]["k"].shape[0]) * ps,), -1, dtype=torch.long, device="cuda")
    where[s["write"]] = torch.arange(case["T"], device="cuda")      # which new token a slot holds
    which = where[s["read"]]
    for m in ("k", "v"):
        old = _exact_cached(s["cache"], m, s["read"] // ps, s["read"] % ps)
        fresh = new[m] if case["fmt"] == "bf16" else _exact_quantised(new[m])
        got[m] = torch.where((which >= 0)[:, None, None], fresh[which.clamp(min=0)], old)
    return got
