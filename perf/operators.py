"""The operators of the paged key/value cache, as they are measured.

Three operators of a serving step over a paged cache: writing the keys and values of a
chunk of new tokens (kept as bf16, or quantised to FP8 E4M3 with one power-of-two scale per
token and head), reading a cache back into contiguous bf16 tensors, and the attention of a
chunk of new tokens (or of single tokens) over the cache, all keys or a window of the newest
keys beside a few first ones (sinks).

Conventions: a batch of B sequences brings ragged chunks; rows q_start[b] .. q_start[b+1] of
the token tensors belong to sequence b and are its last positions, kv_len[b] counts its keys
with the new ones, and page_table[b, i] is the page that holds positions i * page_size ...
Pages are [page, slot, head, dim].
"""
import math
import random

import torch

own = False

GIB = 1 << 30


def listed():
    return [
        # one decode step of a batch: 16 new rows to quantise, where the launch is what counts
        dict(name="write_step_fp8", op="write", B=16, new=1, ctx=4096, mix=1, singles=0, kv="fp8",
             Hq=32, Hkv=8, D=128, page=64),
        # chunked prefill of four prompts of uneven length into an FP8 cache
        dict(name="write_chunk_fp8", op="write", B=4, new=16384, ctx=32768, mix=2, singles=0, kv="fp8",
             Hq=32, Hkv=8, D=128, page=64),
        # a prompt written as it is, small pages, 64-wide heads
        dict(name="write_chunk_bf16", op="write", B=2, new=8191, ctx=8191, mix=3, singles=0, kv="bf16",
             Hq=16, Hkv=16, D=64, page=16),
        # an FP8 cache of one long context read back for an index build or a selection
        dict(name="read_128k_fp8", op="read", B=1, new=1, ctx=131072, mix=0, singles=0, kv="fp8",
             Hq=32, Hkv=8, D=128, page=64),
        # a ragged batch gathered out of its pages
        dict(name="read_batch_bf16", op="read", B=16, new=1, ctx=8192, mix=4, singles=0, kv="bf16",
             Hq=32, Hkv=8, D=128, page=16),
        # one token of one short conversation: latency
        dict(name="attn_token_2k", op="attn", B=1, new=1, ctx=2048, mix=0, singles=0, kv="bf16",
             Hq=32, Hkv=8, D=128, page=64, sink=0, stream=-1),
        # the decode step of a batch with uneven contexts
        dict(name="attn_tokens_b16_32k", op="attn", B=16, new=1, ctx=32768, mix=5, singles=0, kv="bf16",
             Hq=32, Hkv=8, D=128, page=64, sink=0, stream=-1),
        # one token over a million keys held in FP8
        dict(name="attn_token_1m_fp8", op="attn", B=1, new=1, ctx=1048576, mix=0, singles=0, kv="fp8",
             Hq=32, Hkv=8, D=128, page=64, sink=0, stream=-1),
        # the last chunk of a 128K prompt in chunked prefill
        dict(name="attn_chunk_128k", op="attn", B=1, new=2048, ctx=131072, mix=0, singles=0, kv="bf16",
             Hq=32, Hkv=8, D=128, page=64, sink=0, stream=-1),
        # a mixed step: five prompts in progress and eleven decoding sequences, FP8, small pages
        dict(name="attn_mixed_fp8", op="attn", B=16, new=509, ctx=16384, mix=6, singles=11, kv="fp8",
             Hq=32, Hkv=8, D=128, page=16, sink=0, stream=-1),
        # a layer that sees the newest 1024 keys and 256 first ones, over a whole prompt
        dict(name="attn_window_8k", op="attn", B=1, new=8192, ctx=8192, mix=0, singles=0, kv="bf16",
             Hq=32, Hkv=8, D=128, page=64, sink=256, stream=1024),
        # whole prompts of odd length, one key head for each query head, 64-wide heads
        dict(name="attn_prompt_d64", op="attn", B=2, new=4099, ctx=4099, mix=7, singles=0, kv="bf16",
             Hq=16, Hkv=16, D=64, page=128, sink=0, stream=-1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "read", "attn", "attn", "attn"])
    D = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8, 8])
    Hq = Hkv * rng.choice([1, 2, 4, 4, 6, 8])
    c = dict(op=op, kv=rng.choice(["bf16", "fp8"]), Hq=Hq, Hkv=Hkv, D=D, page=rng.choice([16, 32, 64, 128]),
             mix=rng.randint(8, 1 << 20), singles=0)
    if op == "write":
        B, new = rng.choice([1, 3, 16, 64]), _log(rng, 1, 32768)
        while B * new > 65536:
            B = max(1, B // 2)
        return dict(c, B=B, new=new, ctx=new + _log(rng, 1, 8192))
    if op == "read":
        B, ctx = rng.choice([1, 2, 5, 16]), _log(rng, 17, 131072)
        while B * ctx > 131072:
            B = max(1, B // 2)
        return dict(c, B=B, new=1, ctx=ctx)
    B = rng.choice([1, 1, 2, 5, 16, 33])
    new = rng.choice([1, 1, _log(rng, 2, 17), _log(rng, 18, 2048)])
    ctx = new + _log(rng, 1, 131072)
    # no drawn case is more work than the largest listed ones
    while B > 1 and (B * ctx > 400000 or B * new * ctx * Hq > 2048 * 65536 * 32):
        B //= 2
    while new * ctx * Hq * B > 2048 * 65536 * 32:
        new = (new + 1) // 2
    sink, stream = rng.choice([(0, -1), (0, -1), (rng.randint(0, 300), _log(rng, 1, 4096))])
    return dict(c, B=B, new=new, ctx=ctx, sink=sink, stream=stream,
                singles=rng.choice([0, B // 2]) if new > 1 else 0)


def _lens(c):
    """(new tokens, keys) of each sequence, from the case alone."""
    B, new, ctx = c["B"], c["new"], c["ctx"]
    if c["mix"] == 0:
        return [new] * B, [ctx] * B
    r = random.Random(c["mix"])
    ns, ts = [], []
    for b in range(B):
        n = new if b == 0 else max(1, int(new * r.uniform(0.1, 1.0)))
        if b >= B - c["singles"]:
            n = 1
        t = ctx if b == 0 else max(n, int(ctx * r.uniform(0.05, 1.0)))
        ns.append(n)
        ts.append(t)
    return ns, ts


def _attended(c):
    """Keys attended by all rows of a query head, and the key rows that are read once each."""
    ns, ts = _lens(c)
    sink, stream = c["sink"], c["stream"]
    pairs = rows = 0
    for n, t in zip(ns, ts):
        p0 = t - n
        if stream < 0:
            pairs += n * p0 + n * (n + 1) // 2
            rows += t
        else:
            for p in range(p0, t):
                lo = max(0, p + 1 - stream)
                pairs += p + 1 - lo + min(sink, lo)
            lo = max(0, p0 + 1 - stream)
            rows += t - lo + min(sink, lo)
    return pairs, rows


def work(c):
    ns, ts = _lens(c)
    N, T = sum(ns), sum(ts)
    row = c["Hkv"] * c["D"] * 2                                     # a token's keys (or values) as bf16
    kept = c["Hkv"] * (c["D"] + 1) if c["kv"] == "fp8" else row     # the same as the cache holds them
    if c["op"] == "write":
        return {"bytes": 2 * N * (row + kept), "flops": 0}
    if c["op"] == "read":
        return {"bytes": 2 * T * (row + kept), "flops": 0}
    pairs, rows = _attended(c)
    q = N * c["Hq"] * c["D"] * 2
    return {"bytes": 2 * q + N * c["Hq"] * 4 + 2 * rows * kept, "flops": 4 * c["D"] * c["Hq"] * pairs}


# ------------------------------------------------------------------ what a program holds

def _quantise(x):
    """x [..., D] bf16 -> (E4M3 codes of x / 2^e, scale bytes e + 127), one e per row."""
    x = x.float()
    a = torch.where(torch.isfinite(x), x.abs(), torch.zeros_like(x)).amax(-1)
    m, p = torch.frexp(a)                                     # a = m 2^p, m in [0.5, 1)
    e = p - 9 + (m > 0.875).int()                             # smallest e with a 2^-e <= 448
    e = torch.where(a > 0, e.clamp(-116, 119), torch.zeros_like(e))
    inv = ((127 - e) << 23).view(torch.float32)               # 2^-e
    y = (x * inv[..., None]).clamp(-448.0, 448.0)
    return y.to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def _dequantise(codes, scale):
    return codes.view(torch.float8_e4m3fn).float() * (scale.int() << 23).view(torch.float32)[..., None]


def prepare(c, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32)

    ns, ts = _lens(c)
    N, B, H, D, ps = sum(ns), c["B"], c["Hkv"], c["D"], c["page"]
    need = [-(-t // ps) for t in ts]
    P = sum(need) + 3
    order = torch.randperm(P, generator=g, device=dev).int().cpu()
    table = torch.full((B, max(need)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    # keys with a few strong channels and queries that follow them: scores spread over several
    # units, as after training, while values stay near the unit normal
    gain = 1.0 + 2.0 * (torch.rand(H, D, generator=g, device=dev) < 0.06)
    s = {"op": c["op"], "case": c, "max_new": max(ns), "max_len": max(ts),
         "q_start": torch.tensor([0] + ns).cumsum(0).int().to(dev),
         "kv_len": torch.tensor(ts, dtype=torch.int32, device=dev), "table": table.to(dev)}
    fp8 = c["kv"] == "fp8"
    if c["op"] == "write":
        # keys and values as the fused projection leaves them: slices of one row per token
        qkv = randn(N, c["Hq"] + 2 * H, D)
        qkv[:, c["Hq"]:c["Hq"] + H] *= gain
        qkv = qkv.bfloat16()
        s["k_new"], s["v_new"] = qkv[:, c["Hq"]:c["Hq"] + H], qkv[:, c["Hq"] + H:]
        if fp8:
            for n in ("k", "v"):
                s[n] = torch.zeros(P, ps, H, D, dtype=torch.uint8, device=dev)
                s[n + "_scale"] = torch.full((P, ps, H), 127, dtype=torch.uint8, device=dev)
        else:
            for n in ("k", "v"):
                s[n], s[n + "_scale"] = torch.zeros(P, ps, H, D, dtype=torch.bfloat16, device=dev), None
        return s
    for n in ("k", "v"):
        x = randn(P, ps, H, D)
        if n == "k":
            x *= gain
        x = x.bfloat16()
        if fp8:
            codes, s[n + "_scale"] = _quantise(x)
            s[n] = codes.view(torch.uint8)
        else:
            s[n], s[n + "_scale"] = x, None
        del x
    if c["op"] == "attn":
        q = randn(N, H, c["Hq"] // H, D) * (1.0 + 0.5 * gain[:, None])
        s["q"] = q.reshape(N, c["Hq"], D).bfloat16()
    else:
        s["k_out"] = torch.zeros(B, max(ts), H, D, dtype=torch.bfloat16, device=dev)
        s["v_out"] = torch.zeros_like(s["k_out"])
    return s


# ------------------------------------------------------------------ plain forms

def _write(s):
    ps = s["case"]["page"]
    q_start, kv_len = s["q_start"].long(), s["kv_len"].long()
    n = torch.arange(s["k_new"].shape[0], device=q_start.device)
    b = torch.searchsorted(q_start, n, right=True) - 1
    pos = kv_len[b] - (q_start[b + 1] - n)
    slot = s["table"][b, pos // ps].long() * ps + pos % ps
    for name in ("k", "v"):
        x = s[name + "_new"]
        if s["case"]["kv"] == "fp8":
            codes, scale = _quantise(x)
            s[name].flatten(0, 1)[slot] = codes.view(torch.uint8)
            s[name + "_scale"].flatten(0, 1)[slot] = scale
        else:
            s[name].flatten(0, 1)[slot] = x


def _written(s):
    out = {}
    for name in ("k", "v"):
        if s["case"]["kv"] == "fp8":
            out[name], out[name + "_scale"] = s[name].view(torch.float8_e4m3fn), s[name + "_scale"]
        else:
            out[name] = s[name]
    return out


def _gather(s, name, h=slice(None)):
    """The cache of every sequence as fp32 [B, T, heads, D], zero behind its end."""
    table, T = s["table"].long().clamp(min=0), s["max_len"]
    x = s[name][:, :, h][table].flatten(1, 2)[:, :T]
    if s["case"]["kv"] == "fp8":
        x = _dequantise(x, s[name + "_scale"][:, :, h][table].flatten(1, 2)[:, :T])
    ok = torch.arange(T, device=table.device) < s["kv_len"][:, None]
    return torch.where(ok[:, :, None, None], x.float(), 0.0), ok


def _read(s):
    for name in ("k", "v"):
        x, ok = _gather(s, name)
        o = s[name + "_out"]
        torch.where(ok[:, :, None, None], x.to(o.dtype), o, out=o)
    return {"k": s["k_out"], "v": s["v_out"]}


def _attn(s):
    c, q = s["case"], s["q"]
    N, Hq, D = q.shape
    B, H, G, n, T = c["B"], c["Hkv"], Hq // c["Hkv"], s["max_new"], s["max_len"]
    dev = q.device
    q_start, kv_len = s["q_start"].long(), s["kv_len"].long()
    i = torch.arange(n, device=dev)
    row = q_start[:-1, None] + i                                         # [B, n]
    real = row < q_start[1:, None]
    pos = (kv_len - q_start[1:])[:, None] + row
    j = torch.arange(T, device=dev)
    mask = (j <= pos[..., None]) & (j < kv_len[:, None, None])
    if c["stream"] >= 0:
        mask &= (j > pos[..., None] - c["stream"]) | (j < c["sink"])
    row = row.clamp(max=N - 1)
    out = torch.empty(N, Hq, D, dtype=q.dtype, device=dev)
    lse = torch.empty(N, Hq, dtype=torch.float32, device=dev)
    # key heads together as far as their scores fit: a head's are [B, n G, T] in fp32
    step = max(1, min(H, (3 * GIB) // (B * n * G * T)))
    for h0 in range(0, H, step):
        h = slice(h0, min(H, h0 + step))
        hq = slice(h.start * G, h.stop * G)
        k, v = _gather(s, "k", h)[0], _gather(s, "v", h)[0]
        qb = q[:, hq][row].float().view(B, n, -1, G, D)
        x = torch.einsum("bnhgd,bthd->bhgnt", qb, k) * D ** -0.5
        x.masked_fill_(~mask[:, None, None], -math.inf)
        m = x.amax(-1, keepdim=True)
        m = torch.where(m == -math.inf, 0.0, m)
        x = x.sub_(m).exp_()
        l = x.sum(-1)
        o = torch.einsum("bhgnt,bthd->bnhgd", x, v)
        l = l.permute(0, 3, 1, 2)                                        # [B, n, heads, G]
        o = torch.where(l[..., None] > 0, o / l[..., None], 0.0)
        out[:, hq][row[real]] = o.flatten(2, 3)[real].to(out.dtype)
        lse[:, hq][row[real]] = (m[..., 0].permute(0, 3, 1, 2) + l.log()).flatten(2, 3)[real]
    return {"out": out, "lse": lse}


def _own(s):
    import dynamic_sparse_attention_gb300 as dsa
    c = s["case"]
    cache = dsa.PagedKVCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
    if c["op"] == "write":
        dsa.kv_cache_write(cache, s["k_new"], s["v_new"], s["q_start"], s["kv_len"], s["table"])
        return _written(s)
    if c["op"] == "read":
        k, v = dsa.kv_cache_read(cache, s["kv_len"], s["table"], out=(s["k_out"], s["v_out"]))
        return {"k": k, "v": v}
    out, lse = dsa.paged_attn(s["q"], cache, s["q_start"], s["kv_len"], s["table"], n_sink=c["sink"],
                              n_stream=None if c["stream"] < 0 else c["stream"])
    return {"out": out, "lse": lse}


def run(s):
    if own:
        return _own(s)
    if s["op"] == "write":
        _write(s)
        return _written(s)
    return _read(s) if s["op"] == "read" else _attn(s)


# ------------------------------------------------------------------ in 64 bits

def _e4m3_values(dev):
    """The 127 magnitudes of E4M3 in ascending order of their codes."""
    v = [m * 2.0 ** -9 for m in range(8)]
    v += [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)]
    return torch.tensor(v[:127], dtype=torch.float64, device=dev)


def _exact_rows(x):
    """Rows x [..., D] in float64 -> the E4M3 values they are held as (unscaled)."""
    grid = _e4m3_values(x.device)
    a = x.abs().amax(-1)
    def two(e):                                               # 2^e, exactly
        return ((e.long() + 1023) << 52).view(torch.float64)

    e = torch.ceil(torch.log2(torch.where(a > 0, a, 1.0) / 448.0))
    e = torch.where(a > 448.0 * two(e), e + 1, e)             # the logarithm's own rounding
    e = torch.where(a <= 448.0 * two(e - 1), e - 1, e)
    e = torch.where(a > 0, e, 0.0)
    y = x / two(e)[..., None]
    mid = (grid[1:] + grid[:-1]) / 2
    lo = torch.bucketize(y.abs(), mid)                        # a tie goes to the lower value,
    tie = y.abs() == mid[lo.clamp(max=len(mid) - 1)]
    lo = torch.where(tie & (lo % 2 == 1), lo + 1, lo)         # or to the even code above it
    return grid[lo] * torch.sign(y)


def _value(s, name, page):
    """Pages (an index tensor) of the cache in float64."""
    x = s[name][page]
    if s["case"]["kv"] != "fp8":
        return x.double()
    grid = _e4m3_values(x.device)
    mag = grid[(x & 127).long().clamp(max=126)] * torch.where(x > 127, -1.0, 1.0)
    two = ((s[name + "_scale"][page].long() + 1023 - 127) << 52).view(torch.float64)
    return mag * two[..., None]


def exact(c, seed):
    s = prepare(c, seed)
    ns, ts = _lens(c)
    ps, H, D = c["page"], c["Hkv"], c["D"]
    table = s["table"].tolist()
    if c["op"] == "write":
        out = {}
        for name in ("k", "v"):
            x = s[name + "_new"].double()
            x = _exact_rows(x) if c["kv"] == "fp8" else x
            pages = torch.zeros(s[name].shape, dtype=torch.float64, device=x.device)
            at = 0
            for b, (n, t) in enumerate(zip(ns, ts)):
                p = torch.arange(t - n, t, device=x.device)
                pages[s["table"][b].long()[p // ps], p % ps] = x[at:at + n]
                at += n
            out[name] = pages
            if c["kv"] == "fp8":
                out[name + "_scale"] = None
        return out
    if c["op"] == "read":
        out = {}
        for name in ("k", "v"):
            full = torch.zeros(s[name + "_out"].shape, dtype=torch.float64, device=s["k"].device)
            for b, t in enumerate(ts):
                pages = torch.tensor(table[b][:-(-t // ps)], device=full.device)
                full[b, :t] = _value(s, name, pages).reshape(-1, H, D)[:t]
            out[name] = full
        return out
    q = s["q"].double()
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.zeros(q.shape[:2], dtype=torch.float64, device=q.device)
    G, at = c["Hq"] // H, 0
    for n, t, pages in zip(ns, ts, table):
        page = torch.tensor(pages[:-(-t // ps)], device=q.device)
        key = torch.arange(t, device=q.device)
        k = _value(s, "k", page).reshape(-1, H, D)[:t]
        v = _value(s, "v", page).reshape(-1, H, D)[:t]
        block = max(1, (GIB // 2) // t)
        for i in range(0, n, block):                          # query rows in blocks, head by head
            rows = slice(at + i, at + min(n, i + block))
            p = torch.arange(t - n + i, t - n + min(n, i + block), device=q.device)[:, None]
            seen = key <= p
            if c["stream"] >= 0:
                seen = seen & ((key < c["sink"]) | (key + c["stream"] > p))
            hide = torch.zeros(seen.shape, dtype=torch.float64, device=q.device)
            hide[~seen] = -math.inf
            for h in range(c["Hq"]):
                x = torch.addmm(hide, q[rows, h], k[:, h // G].T, alpha=1.0 / math.sqrt(D))
                z = torch.logsumexp(x, 1)
                lse[rows, h] = z
                out[rows, h] = torch.where(z[:, None] == -math.inf, 0.0, torch.exp(x - z[:, None]).nan_to_num() @ v[:, h // G])
        at += n
    return {"out": out, "lse": lse}
