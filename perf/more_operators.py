"""The operators around the paged key/value cache's sparse path, as they are measured.

Five operators of a serving step: writing a chunk's keys and values into the pages with the
norm of each head and the rotation by position on the way (the queries come back rotated); the
digest of the pages that a chunk touched (per channel the smallest and largest key, in 8 bits);
the choice of pages for each block of queries by a bound on their scores made from the digests;
attention over the chosen pages, a page table for each key head; and copies of pages (a fork's
partly filled pages, a compaction).

Conventions: a batch of B sequences brings ragged chunks; rows q_start[b] .. q_start[b+1] of
the token tensors belong to sequence b and are its last positions, kv_len[b] counts its keys
with the new ones, and page_table[b, i] is the page that holds positions i * page_size ...
Pages are [page, slot, head, dim].
"""
import math
import random

import torch

own = False


def listed():
    return [
        # one decode step of a batch into an FP8 cache: the launch is what counts
        dict(name="rope_step_fp8", op="rope", B=16, new=1, ctx=4096, mix=1, singles=0, kv="fp8",
             Hq=32, Hkv=8, D=128, page=64, norm=True, rot=128, inter=False, theta=1e6),
        # chunked prefill of four prompts of uneven length
        dict(name="rope_chunk_bf16", op="rope", B=4, new=16384, ctx=32768, mix=2, singles=0, kv="bf16",
             Hq=32, Hkv=8, D=128, page=64, norm=True, rot=128, inter=False, theta=1e6),
        # the decode step's sixteen last pages
        dict(name="digest_step", op="digest", B=16, new=1, ctx=32768, mix=5, singles=0, kv="bf16",
             Hq=32, Hkv=8, D=128, page=64),
        # every page of a long prompt
        dict(name="digest_128k", op="digest", B=1, new=131071, ctx=131071, mix=0, singles=0, kv="bf16",
             Hq=32, Hkv=8, D=128, page=64),
        # the decode step of a batch with uneven contexts, each token its own choice
        dict(name="select_tokens_b16_32k", op="select", B=16, new=1, ctx=32768, mix=5, singles=0, kv="bf16",
             Hq=32, Hkv=8, D=128, page=64, q_block=1, keep=60, sink=1, local=2),
        # one token over a million keys
        dict(name="select_token_1m", op="select", B=1, new=1, ctx=1048576, mix=0, singles=0, kv="bf16",
             Hq=32, Hkv=8, D=128, page=64, q_block=1, keep=124, sink=1, local=2),
        # the last chunk of a 128K prompt, one choice for 64 tokens
        dict(name="select_chunk_128k", op="select", B=1, new=2048, ctx=131072, mix=0, singles=0, kv="bf16",
             Hq=32, Hkv=8, D=128, page=64, q_block=64, keep=60, sink=1, local=2),
        # the decode step over 4,096 keys of each long sequence
        dict(name="attend_tokens_b16", op="attend", B=16, new=1, ctx=65536, mix=5, singles=0, kv="bf16",
             Hq=32, Hkv=8, D=128, page=64, q_block=1, keep=60, sink=1, local=2),
        # one token over 8,192 of a million keys held in FP8
        dict(name="attend_token_1m_fp8", op="attend", B=1, new=1, ctx=1048576, mix=0, singles=0, kv="fp8",
             Hq=32, Hkv=8, D=128, page=64, q_block=1, keep=124, sink=1, local=2),
        # the last chunk of a 128K prompt over the pages chosen for each 64 tokens
        dict(name="attend_chunk_128k", op="attend", B=1, new=2048, ctx=131072, mix=0, singles=0, kv="bf16",
             Hq=32, Hkv=8, D=128, page=64, q_block=64, keep=60, sink=1, local=2),
        # 32 sequences forked: the partly filled last page of each
        dict(name="copy_fork", op="copy", pages=32, kv="fp8", Hq=32, Hkv=8, D=128, page=64, digest=True),
        # a compaction that moves half a cache
        dict(name="copy_compact", op="copy", pages=2048, kv="bf16", Hq=32, Hkv=8, D=128, page=64, digest=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "digest", "select", "select", "attend", "attend", "copy"])
    D = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8, 8])
    Hq = Hkv * rng.choice([1, 2, 4, 4, 6, 8])
    c = dict(op=op, kv=rng.choice(["bf16", "fp8"]), Hq=Hq, Hkv=Hkv, D=D, page=rng.choice([16, 32, 64, 128]))
    if op == "copy":
        pages = _log(rng, 1, 4096)
        while pages * c["page"] * Hkv * D > 2048 * 64 * 8 * 128:
            pages //= 2
        return dict(c, pages=max(1, pages), digest=rng.choice([True, False]))
    c.update(mix=rng.randint(8, 1 << 20), singles=0)
    if op in ("rope", "digest"):
        B, new = rng.choice([1, 3, 16, 64]), _log(rng, 1, 32768)
        while B * new > 65536:
            B = max(1, B // 2)
        c.update(B=B, new=new, ctx=new + _log(rng, 1, 8192))
        if op == "digest":
            return c
        return dict(c, norm=rng.choice([True, True, False]), rot=rng.choice([D, D, D // 2]),
                    inter=rng.choice([False, True]), theta=rng.choice([1e4, 5e5, 1e6]))
    B = rng.choice([1, 1, 2, 5, 16, 33])
    new = rng.choice([1, 1, _log(rng, 2, 17), _log(rng, 18, 2048)])
    q_block = 1 if new == 1 else rng.choice([16, 32, 64, 128])
    keep, local = _log(rng, 1, 128), rng.randint(0, 4)
    ctx = new + _log(rng, 64, 131072)
    # no drawn case is more work, or takes more memory in its plain form, than the largest listed ones
    while B > 1 and B * (-(-new // q_block)) * ctx > 32 * 131072 * c["page"] // 64:
        B //= 2
    while (-(-new // q_block)) * ctx > 32 * 131072 * c["page"] // 64 or B * new * Hq > 2048 * 32:
        new = (new + 1) // 2
    while keep > 8 and B * new * Hq * (keep + 3) * c["page"] > 2048 * 32 * 64 * 64:
        keep //= 2
    return dict(c, B=B, new=new, ctx=ctx, q_block=q_block, keep=keep, sink=rng.randint(0, 2), local=local,
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


def _blocks(c):
    """(sequence, position of the first query, queries) of each block of queries."""
    out = []
    for b, (n, t) in enumerate(zip(*_lens(c))):
        for i in range(0, n, c["q_block"]):
            out.append((b, t - n + i, min(c["q_block"], n - i)))
    return out


def _span(c, p0, n):
    """Pages of a block of n queries from position p0 on: (end of the sinks, first page of the
    local ones, first own page, last own page)."""
    own0, own1 = p0 // c["page"], (p0 + n - 1) // c["page"]
    first = max(0, own0 - c["local"])
    return min(c["sink"], first), first, own0, own1


def _max_list(c):
    return c["sink"] + c["keep"] + c["local"] + (c["q_block"] + c["page"] - 2) // c["page"] + 1


def work(c):
    H, Hq, D, ps = c["Hkv"], c["Hq"], c["D"], c["page"]
    row = H * D * 2                                                 # a token's keys (or values) as bf16
    kept = H * (D + 1) if c["kv"] == "fp8" else row                 # the same as the cache holds them
    dig = H * (2 * D + 1)                                           # a page's digest
    if c["op"] == "copy":
        return {"bytes": 2 * c["pages"] * (2 * ps * kept + (dig if c["digest"] else 0)), "flops": 0}
    ns, ts = _lens(c)
    N = sum(ns)
    q = N * Hq * D * 2
    if c["op"] == "rope":
        return {"bytes": 2 * q + 2 * N * (row + kept), "flops": 0}
    if c["op"] == "digest":
        pages = keys = 0
        for n, t in zip(ns, ts):
            first = (t - n) // ps
            pages += -(-t // ps) - first
            keys += t - first * ps
        return {"bytes": keys * kept + pages * dig, "flops": 0}
    if c["op"] == "select":
        pairs = lists = 0
        seen = [0] * c["B"]
        for b, p0, n in _blocks(c):
            s0, first, own0, own1 = _span(c, p0, n)
            pairs += n * Hq * (first - s0)
            seen[b] = max(seen[b], first - s0)
            lists += H * (s0 + min(c["keep"], first - s0) + own1 + 1 - first)
        return {"bytes": q + sum(seen) * dig + 4 * lists, "flops": 2 * D * pairs}
    pairs = 0
    seen = [0] * c["B"]
    for b, p0, n in _blocks(c):
        s0, first, own0, own1 = _span(c, p0, n)
        before = s0 + min(c["keep"], first - s0) + own0 - first
        at = before * ps + p0 % ps
        pairs += n * at + n * (n + 1) // 2
        seen[b] += at + n
    keys = sum(min(s, t) for s, t in zip(seen, ts))
    return {"bytes": 2 * q + N * Hq * 4 + 2 * keys * kept, "flops": 4 * D * Hq * pairs}


# ------------------------------------------------------------------ what a program holds

def _quantise(x):
    """x [..., D] -> (E4M3 codes of x / 2^e, scale bytes e + 127), one e per row."""
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


def _two(e):
    """2^e in fp32, exactly."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _exponent127(a):
    """The least e in [-50, 50] with a 2^-e <= 127; 0 where a is 0."""
    m, p = torch.frexp(a)
    e = p - 7 + (m > 127 / 128).int()
    return torch.where(a > 0, e.clamp(-50, 50), torch.zeros_like(e))


def _digest_of(k, ok):
    """Keys [..., page, heads, D] in fp32, ok [..., page]: int8 bounds [..., heads, 2, D] and exponents."""
    ok = ok[..., None, None]
    real = ok & ~torch.isnan(k)
    a = torch.where(ok & torch.isfinite(k), k.abs(), 0.0).amax((-3, -1))
    e = _exponent127(a)
    lo = torch.where(real, k, math.inf).amin(-3)
    hi = torch.where(real, k, -math.inf).amax(-3)
    some = real.any(-3)
    inv = _two(-e)[..., None]
    lo = torch.where(some, (lo * inv).floor(), 0.0).clamp(-127, 127)
    hi = torch.where(some, (hi * inv).ceil(), 0.0).clamp(-127, 127)
    return torch.stack([lo, hi], -2).to(torch.int8), e.to(torch.int8)


def _query_blocks(s):
    """(sequence, first row, end, real rows [NB, q_block], their token rows) of the blocks of queries;
    blocks behind the last one are empty and stand at the last row's end."""
    c, dev = s["case"], s["q_start"].device
    qb, B, N = c["q_block"], c["B"], s["q"].shape[0]
    q_start = s["q_start"].long()
    per = (q_start[1:] - q_start[:-1] + qb - 1) // qb
    at = torch.cat([per.new_zeros(1), per.cumsum(0)])
    j = torch.arange((N + B * (qb - 1)) // qb, device=dev)
    b = (torch.searchsorted(at, j, right=True) - 1).clamp(max=B - 1)
    lo = torch.minimum(q_start[b] + (j - at[b]) * qb, q_start[b + 1])
    hi = torch.minimum(lo + qb, q_start[b + 1])
    row = lo[:, None] + torch.arange(qb, device=dev)
    return b, lo, hi, row < hi[:, None], row.clamp(max=N - 1)


def _lists(s, score):
    """score [NB, heads, pages] (of every page): the lists as page ids [NB, heads, max], the
    blocks' rows as q_start and the lists' lengths in keys."""
    c, dev = s["case"], score.device
    ps, P = c["page"], score.shape[-1]
    b, lo, hi, _, _ = _query_blocks(s)
    kv_len, q_end = s["kv_len"].long(), s["q_start"].long()[1:]
    n = hi - lo
    p0 = kv_len[b] - (q_end[b] - lo)
    own0, own1 = p0 // ps, (p0 + n - 1) // ps
    first = (own0 - c["local"]).clamp(min=0)
    s0 = first.clamp(max=c["sink"])
    page = torch.arange(P, device=dev)
    cand = (page >= s0[:, None]) & (page < first[:, None])                   # [NB, P]
    score = torch.where(cand[:, None], score, -math.inf)
    best = score.sort(dim=-1, descending=True, stable=True).indices[..., :c["keep"]]
    listed_ = torch.zeros(score.shape, dtype=torch.bool, device=dev).scatter_(-1, best, True) & cand[:, None]
    fixed = (page < s0[:, None]) | ((page >= first[:, None]) & (page <= own1[:, None]))
    listed_ |= (fixed & (n > 0)[:, None])[:, None]
    place = torch.where(listed_, listed_.cumsum(-1) - 1, _max_list(c))
    table = torch.full((*score.shape[:2], _max_list(c) + 1), -1, dtype=torch.int32, device=dev)
    ids = s["table"][b][:, None, :P].expand_as(place)
    table.scatter_(-1, place, ids)
    before = s0 + torch.minimum(first - s0, torch.full_like(s0, c["keep"])) + own0 - first
    length = torch.where(n > 0, before * ps + p0 % ps + n, 0)
    start = torch.cat([lo, hi[-1:]]).int()
    return table[..., :-1].contiguous(), start, length.int()


def prepare(c, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32)

    H, Hq, D, ps = c["Hkv"], c["Hq"], c["D"], c["page"]
    fp8 = c["kv"] == "fp8"
    s = {"op": c["op"], "case": c}
    # keys with a few strong channels and queries that follow them: scores spread over several
    # units, as after training, while values stay near the unit normal
    gain = 1.0 + 2.0 * (torch.rand(H, D, generator=g, device=dev) < 0.06)

    def pages(name, P, group=64):
        x = torch.empty(P, ps, H, D, dtype=torch.bfloat16, device=dev)
        for i in range(0, P, group):                     # keys of one page lie around a point of their own
            j = min(P, i + group)
            y = randn(j - i, ps, H, D)
            x[i:j] = (y * 0.7 + randn(j - i, 1, H, D) * 0.7) * gain if name == "k" else y
        return x

    def cache(P):
        for name in ("k", "v"):
            x = pages(name, P, 1024)
            s[name], s[name + "_scale"] = x, None
            if fp8:
                codes, s[name + "_scale"] = _quantise(x)
                s[name] = codes.view(torch.uint8)

    def digest(P, values=None):
        s["bounds"] = torch.zeros(P, H, 2, D, dtype=torch.int8, device=dev)
        s["exp"] = torch.zeros(P, H, dtype=torch.int8, device=dev)
        if values is not None:
            for i in range(0, P, 1024):
                y = values[i:i + 1024].float()
                s["bounds"][i:i + 1024], s["exp"][i:i + 1024] = _digest_of(y, y.new_ones(y.shape[:2], dtype=torch.bool))

    if c["op"] == "copy":
        n = c["pages"]
        cache(2 * n + 3)
        if c["digest"]:
            digest(2 * n + 3)
            s["bounds"].random_(-127, 128, generator=g)
            s["exp"].random_(-10, 10, generator=g)
        order = torch.randperm(2 * n + 3, generator=g, device=dev).int()
        s["src"], s["dst"] = order[:n].clone(), order[n:2 * n].clone()
        return s

    ns, ts = _lens(c)
    N, B = sum(ns), c["B"]
    need = [-(-t // ps) for t in ts]
    P = sum(need) + 3
    order = torch.randperm(P, generator=g, device=dev).int().cpu()
    table = torch.full((B, max(need)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    s |= {"n_tok": N, "q_start": torch.tensor([0] + ns).cumsum(0).int().to(dev),
          "kv_len": torch.tensor(ts, dtype=torch.int32, device=dev), "table": table.to(dev)}
    if c["op"] == "rope":
        # queries, keys and values as the fused projection leaves them: slices of one row per token
        qkv = randn(N, Hq + 2 * H, D)
        qkv[:, Hq:Hq + H] *= gain
        qkv = qkv.bfloat16()
        s["q"], s["k_new"], s["v_new"] = qkv[:, :Hq], qkv[:, Hq:Hq + H], qkv[:, Hq + H:]
        s["q_weight"] = (1.0 + 0.3 * randn(D)).bfloat16() if c["norm"] else None
        s["k_weight"] = (1.0 + 0.3 * randn(D)).bfloat16() if c["norm"] else None
        s["inv_freq"] = c["theta"] ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64, device=dev) / c["rot"])
        s["eps"], s["q_out"] = 1e-6, torch.zeros(N, Hq, D, dtype=torch.bfloat16, device=dev)
        for n in ("k", "v"):
            s[n] = torch.zeros(P, ps, H, D, dtype=torch.uint8 if fp8 else torch.bfloat16, device=dev)
            s[n + "_scale"] = torch.full((P, ps, H), 127, dtype=torch.uint8, device=dev) if fp8 else None
        return s
    if c["op"] == "digest":
        cache(P)
        digest(P)
        return s
    q = randn(N, H, Hq // H, D) * (1.0 + 0.5 * gain[:, None])
    if c["op"] == "select":
        k = pages("k", P, 1024)
        digest(P, k)
        # each token's queries lean towards the keys of some page of its sequence
        to = torch.randint(0, P, (N,), generator=g, device=dev)
        q = q + k[to, 0].float()[:, :, None]
        s["q"] = q.reshape(N, Hq, D).bfloat16()
        return s
    s["q"] = q.reshape(N, Hq, D).bfloat16()
    cache(P)
    # lists as a selection leaves them: runs of pages that many blocks like, and others
    liked = torch.rand(B, H, max(need), generator=g, device=dev)
    b = _query_blocks(s)[0]
    score = liked[b] + torch.rand(len(b), H, max(need), generator=g, device=dev)
    s["lists"], s["list_start"], s["list_len"] = _lists(s, score)
    return s


# ------------------------------------------------------------------ plain forms

def _tokens(s):
    """Sequence and position of every token row."""
    q_start, kv_len = s["q_start"].long(), s["kv_len"].long()
    n = torch.arange(s["n_tok"], device=q_start.device)
    b = torch.searchsorted(q_start, n, right=True) - 1
    return b, kv_len[b] - (q_start[b + 1] - n)


def _head_norm(s, name, weight):
    x = s[name].float()
    if weight is None:
        return x
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"]) * weight.float()


def _rotate(c, x, cos, sin):
    R = c["rot"]
    y = x.clone()
    a, b = (slice(0, R, 2), slice(1, R, 2)) if c["inter"] else (slice(0, R // 2), slice(R // 2, R))
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., b] * cos + x[..., a] * sin
    return y


def _rope(s):
    c, ps = s["case"], s["case"]["page"]
    b, pos = _tokens(s)
    slot = s["table"][b, pos // ps].long() * ps + pos % ps
    angle = pos.double()[:, None, None] * s["inv_freq"]
    cos, sin = angle.cos().float(), angle.sin().float()
    q = _rotate(c, _head_norm(s, "q", s["q_weight"]), cos, sin)
    s["q_out"].copy_(q)
    rows = {"k": _rotate(c, _head_norm(s, "k_new", s["k_weight"]), cos, sin), "v": s["v_new"]}
    for name, x in rows.items():
        if c["kv"] == "fp8":
            codes, scale = _quantise(x)
            s[name].flatten(0, 1)[slot] = codes.view(torch.uint8)
            s[name + "_scale"].flatten(0, 1)[slot] = scale
        else:
            s[name].flatten(0, 1)[slot] = x.bfloat16()
    return _written(s)


def _written(s):
    out = {"q": s["q_out"]}
    for name in ("k", "v"):
        if s["case"]["kv"] == "fp8":
            out[name] = s[name].view(torch.float8_e4m3fn)
            out[name + "_scale"] = s[name + "_scale"].view(torch.float8_e8m0fnu)
        else:
            out[name] = s[name]
    return out


def _digest(s):
    ps, dev = s["case"]["page"], s["table"].device
    q_start, kv_len = s["q_start"].long(), s["kv_len"].long()
    i = torch.arange(s["table"].shape[1], device=dev)
    n = q_start[1:] - q_start[:-1]
    touched = (i >= ((kv_len - n) // ps)[:, None]) & (i * ps < kv_len[:, None]) & (n > 0)[:, None]
    b, i = touched.nonzero(as_tuple=True)
    page = s["table"][b, i].long()
    k = s["k"][page]
    k = _dequantise(k, s["k_scale"][page]) if s["case"]["kv"] == "fp8" else k.float()
    ok = i[:, None] * ps + torch.arange(ps, device=dev) < kv_len[b][:, None]
    s["bounds"][page], s["exp"][page] = _digest_of(k, ok)
    return {"bounds": s["bounds"], "exp": s["exp"]}


def _select(s):
    c, H, D = s["case"], s["case"]["Hkv"], s["case"]["D"]
    q = s["q"].float()
    a = torch.where(torch.isfinite(q), q.abs(), 0.0).amax(-1, keepdim=True)
    e = _exponent127(a)
    whole = torch.nan_to_num(q * _two(-e), nan=0.0).round().clamp(-127, 127)
    b, _, _, real, row = _query_blocks(s)
    whole = whole[row].view(*row.shape, H, -1, D)                            # [NB, q_block, H, G, D]
    unit = _two(e)[row].view(*row.shape, H, -1)
    page = s["table"][b].long().clamp(min=0)
    lo, hi = s["bounds"][page].float().unbind(-2)                            # [NB, pages, H, D]
    x = torch.einsum("nthgd,nphd->nhtgp", whole.clamp(min=0), hi)
    x += torch.einsum("nthgd,nphd->nhtgp", whole.clamp(max=0), lo)
    x *= torch.where(real[..., None, None], unit, 0.0).permute(0, 2, 1, 3)[..., None]
    x.masked_fill_(~real[:, None, :, None, None], -math.inf)
    score = x.flatten(2, 3).amax(2) * _two(s["exp"][page]).transpose(1, 2)
    table, start, length = _lists(s, score)
    return {"table": table, "q_start": start, "kv_len": length}


def _attend(s):
    c, q = s["case"], s["q"]
    N, Hq, D = q.shape
    H, G, ps = c["Hkv"], Hq // c["Hkv"], c["page"]
    _, lo, hi, real, row = _query_blocks(s)
    NB, n = row.shape
    page = s["lists"].long().clamp(min=0)                                    # [NB, H, pages]
    head = torch.arange(H, device=q.device)[:, None]

    def rows(name):
        x = s[name].transpose(1, 2)[page, head]                              # [NB, H, pages, ps, D]
        if c["kv"] == "fp8":
            x = _dequantise(x, s[name + "_scale"].transpose(1, 2)[page, head])
        return x.flatten(2, 3).float()

    T = page.shape[-1] * ps
    pos = s["list_len"].long()[:, None] - (hi[:, None] - row)                # of the rows, in the lists
    mask = (torch.arange(T, device=q.device) <= pos[..., None])              # [NB, n, T]
    qb = q[row].float().view(NB, n, H, G, D)
    x = torch.einsum("nthgd,nhkd->nhgtk", qb, rows("k")) * D ** -0.5
    x.masked_fill_(~mask[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    x = x.sub_(m).exp_()
    l = x.sum(-1)
    v = torch.where((torch.arange(T, device=q.device) < s["list_len"][:, None])[:, None, :, None], rows("v"), 0.0)
    o = torch.einsum("nhgtk,nhkd->nthgd", x, v)
    l, m = l.permute(0, 3, 1, 2), m[..., 0].permute(0, 3, 1, 2)              # [NB, n, H, G]
    o = torch.where(l[..., None] > 0, o / l[..., None], 0.0)
    out = torch.empty(N, Hq, D, dtype=q.dtype, device=q.device)
    lse = torch.empty(N, Hq, dtype=torch.float32, device=q.device)
    out[row[real]] = o.flatten(2, 3)[real].to(out.dtype)
    lse[row[real]] = (m + l.log()).flatten(2, 3)[real]
    return {"out": out, "lse": lse}


def _copy(s):
    src, dst = s["src"].long(), s["dst"].long()
    for name in _arrays(s):
        s[name][dst] = s[name][src]
    return _copied(s)


def _arrays(s):
    return [n for n in ("k", "v", "k_scale", "v_scale", "bounds", "exp") if s.get(n) is not None]


def _copied(s):
    return {n: s[n].view(torch.float8_e4m3fn) if n in ("k", "v") and s["case"]["kv"] == "fp8" else s[n]
            for n in _arrays(s)}


def _own(s):
    import dynamic_sparse_attention_gb300 as dsa
    c = s["case"]
    if c["op"] == "select":
        digest = dsa.PageDigest(s["bounds"], s["exp"], c["page"])
        sel = dsa.page_select(s["q"], digest, s["q_start"], s["kv_len"], s["table"], keep=c["keep"],
                              n_sink=c["sink"], n_local=c["local"], q_block=c["q_block"])
        return {"table": sel.page_table, "q_start": sel.q_start, "kv_len": sel.kv_len}
    cache = dsa.PagedKVCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
    if c["op"] == "rope":
        dsa.kv_cache_write_rope(cache, s["q"], s["k_new"], s["v_new"], s["q_start"], s["kv_len"], s["table"],
                                s["inv_freq"], interleaved=c["inter"], q_weight=s["q_weight"],
                                k_weight=s["k_weight"], eps=s["eps"], q_out=s["q_out"])
        return _written(s)
    if c["op"] == "digest":
        digest = dsa.PageDigest(s["bounds"], s["exp"], c["page"])
        dsa.page_digest_update(cache, digest, s["n_tok"], s["q_start"], s["kv_len"], s["table"])
        return {"bounds": s["bounds"], "exp": s["exp"]}
    if c["op"] == "attend":
        out, lse = dsa.paged_attn(s["q"], cache, s["list_start"], s["list_len"], s["lists"])
        return {"out": out, "lse": lse}
    digest = dsa.PageDigest(s["bounds"], s["exp"], c["page"]) if c["digest"] else None
    dsa.kv_pages_copy(cache, s["src"], s["dst"], digest=digest)
    return _copied(s)


def run(s):
    if own:
        return _own(s)
    if s["op"] == "rope":
        return _rope(s)
    if s["op"] == "digest":
        return _digest(s)
    if s["op"] == "select":
        return _select(s)
    return _attend(s) if s["op"] == "attend" else _copy(s)


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


def _values(s, name, page, h):
    """One head of pages (an index tensor) of the cache in float64 [keys, D]."""
    x = s[name][page, :, h]
    if s["case"]["kv"] != "fp8":
        return x.double().flatten(0, 1)
    grid = _e4m3_values(x.device)
    mag = grid[(x & 127).long().clamp(max=126)] * torch.where(x > 127, -1.0, 1.0)
    two = ((s[name + "_scale"][page, :, h].long() + 1023 - 127) << 52).view(torch.float64)
    return (mag * two[..., None]).flatten(0, 1)


def _exact_rope(c, s):
    R, ps = c["rot"], c["page"]
    out = {"q": None, "k": torch.zeros(s["k"].shape, dtype=torch.float64, device=s["k"].device)}
    out["v"] = torch.zeros_like(out["k"])
    at, qs = 0, []
    for b, (n, t) in enumerate(zip(*_lens(c))):
        p = torch.arange(t - n, t, device=s["q"].device)
        z = torch.polar(torch.ones((), dtype=torch.float64, device=p.device), p.double()[:, None] * s["inv_freq"])
        turned = {}
        for name, w in (("q", s["q_weight"]), ("k_new", s["k_weight"])):
            x = s[name][at:at + n].double()
            if w is not None:
                x = x / ((x * x).sum(-1, keepdim=True) / c["D"] + s["eps"]).sqrt() * w.double()
            y = x[..., :R].unflatten(-1, (R // 2, 2) if c["inter"] else (2, R // 2))
            y = y if c["inter"] else y.transpose(-1, -2)
            y = torch.view_as_real(torch.view_as_complex(y.contiguous()) * z[:, None])
            y = (y if c["inter"] else y.transpose(-1, -2)).flatten(-2)
            turned[name] = torch.cat([y, x[..., R:]], -1)
        qs.append(turned["q"])
        page = s["table"][b].long()[p // ps]
        for name, x in (("k", turned["k_new"]), ("v", s["v_new"][at:at + n].double())):
            out[name][page, p % ps] = _exact_rows(x) if c["kv"] == "fp8" else x
        at += n
    out["q"] = torch.cat(qs)
    if c["kv"] == "fp8":
        out["k_scale"] = out["v_scale"] = None
    return out


def exact(c, seed):
    if c["op"] not in ("rope", "attend"):     # whole numbers, or copies
        return None
    s = prepare(c, seed)
    if c["op"] == "rope":
        return _exact_rope(c, s)
    q = s["q"].double()
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.zeros(q.shape[:2], dtype=torch.float64, device=q.device)
    G, ps = c["Hq"] // c["Hkv"], c["page"]
    lists, lens, at = s["lists"].long(), s["list_len"].tolist(), 0
    for j, (_, p0, n) in enumerate(_blocks(c)):
        T = lens[j]
        seen = torch.arange(T, device=q.device) <= torch.arange(T - n, T, device=q.device)[:, None]
        hide = torch.zeros(seen.shape, dtype=torch.float64, device=q.device).masked_fill_(~seen, -math.inf)
        for h in range(c["Hkv"]):
            page = lists[j, h, :-(-T // ps)]
            k, v = _values(s, "k", page, h)[:T], _values(s, "v", page, h)[:T]
            x = torch.einsum("tgd,kd->gtk", q[at:at + n, h * G:(h + 1) * G], k) / math.sqrt(c["D"]) + hide
            z = torch.logsumexp(x, -1)
            lse[at:at + n, h * G:(h + 1) * G] = z.T
            out[at:at + n, h * G:(h + 1) * G] = torch.einsum("gtk,kd->tgd", torch.exp(x - z[..., None]), v)
        at += n
    return {"out": out, "lse": lse}
