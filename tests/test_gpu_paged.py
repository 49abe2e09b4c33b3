"""GPU parity of the paged cache (kv_cache_write, kv_cache_read) and of the attention over it
(paged_attn) against the float64 restatement in oracle/paged.py.

Tolerances (set before the first run).  Cache contents are compared bit by bit.  For the
attention, with h = finfo(bf16).eps / 2 = 2^-8 the half step of bf16:
  out  one rounding of the result, h |out|, one of each probability before P V, h * spread with
       spread = sum_j w_j |v_j|, and relative weight errors of twice the score error below
  lse  the score error: an fp32 dot product of D products and its scaling, at most
       2 D * 2^-24 * size with size = scale * sum_d |q_d k_d|; an exponential and a sum, each
       within 2^-20 relative; the rounding of the sum m + log l, 2^-22 |lse|
"""
import numpy as np
import pytest
import torch

import dynamic_sparse_attention_gb300 as dsa
from dynamic_sparse_attention_gb300 import _build
from oracle import paged
from oracle.numerics import to_f64
from parity import from_dev_bits

pytestmark = pytest.mark.gpu

H = 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    _build.build()
    dsa.load()


@pytest.fixture(autouse=True)
def _no_device_errors():
    yield
    torch.cuda.synchronize()
    assert dsa.device_error() == 0


def f64(t):
    return to_f64(from_dev_bits(t), "bf16")


class Batch:
    """Ragged sequences (new, total) over a cache whose pages start as garbage (NaN)."""

    def __init__(self, seqs, H_q, H_kv, D, page, fp8, seed=0, spare=2, max_pages=None):
        self.rng = np.random.default_rng(seed)
        self.seqs, self.H_q, self.H_kv, self.D, self.page, self.fp8 = seqs, H_q, H_kv, D, page, fp8
        need = [-(-t // page) for _, t in seqs]
        n_pages = sum(need) + spare
        self.cache = dsa.PagedKVCache.empty(n_pages, page, H_kv, D, fp8=fp8)
        if fp8:
            for t in (self.cache.k, self.cache.v):
                t.fill_(0x7E)
            for t in (self.cache.k_scale, self.cache.v_scale):
                t.fill_(255)
        else:
            self.cache.k.fill_(float("nan"))
            self.cache.v.fill_(float("inf"))
        order = self.rng.permutation(n_pages)
        width = max(max(need), 1) if max_pages is None else max_pages
        table = np.full((len(seqs), width), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n]
            at += n
        self.table = torch.from_numpy(table).cuda()
        self.N = sum(n for n, _ in seqs)
        self.q_start = torch.tensor(np.cumsum([0] + [n for n, _ in seqs]), dtype=torch.int32).cuda()
        self.kv_len = torch.tensor([t for _, t in seqs], dtype=torch.int32).cuda()
        self.k = [self.rows(t, H_kv) for _, t in seqs]      # every sequence's keys and values
        self.v = [self.rows(t, H_kv) for _, t in seqs]
        self.q = self.rows(self.N, H_q)

    def rows(self, n, heads, gain=1.0):
        x = self.rng.standard_normal((n, heads, self.D), dtype=np.float32) * gain
        return torch.from_numpy(x).bfloat16().cuda()

    def write(self, upto=None):
        """Write every sequence's rows [0, t): what earlier steps wrote, then the chunks."""
        hist = [t - n for n, t in self.seqs]
        for part in ("history", "chunk"):
            lo = [0] * len(hist) if part == "history" else hist
            hi = hist if part == "history" else [t for _, t in self.seqs]
            n = [b - a for a, b in zip(lo, hi)]
            k = torch.cat([x[a:b] for x, a, b in zip(self.k, lo, hi)])
            v = torch.cat([x[a:b] for x, a, b in zip(self.v, lo, hi)])
            qs = torch.tensor(np.cumsum([0] + n), dtype=torch.int32).cuda()
            kl = torch.tensor(hi, dtype=torch.int32).cuda()
            dsa.kv_cache_write(self.cache, k, v, qs, kl, self.table)
        return self

    def held(self, b):
        """Sequence b's keys and values as the cache holds them, in float64."""
        out = []
        for x in (self.k[b], self.v[b]):
            x = f64(x)
            out.append(paged.dequantise(*paged.quantise(x)) if self.fp8 else x)
        return out

    def attn(self, **kw):
        return dsa.paged_attn(self.q, self.cache, self.q_start, self.kv_len, self.table, **kw)

    def check(self, out, lse, n_sink=0, n_stream=None, scale=None, rows=None, lost=None):
        torch.cuda.synchronize()
        scale = self.D ** -0.5 if scale is None else scale
        o, z, q = f64(out), lse.cpu().numpy().astype(np.float64), f64(self.q)
        at = 0
        for b, (n, t) in enumerate(self.seqs):
            if n and (rows is None or b in rows):
                k, v = self.held(b)
                O, L, spread, size = paged.attend(q[at:at + n], k, v, t - n, n_sink, n_stream, scale,
                                                  None if lost is None else lost[b])
                ds = 2 * self.D * 2.0 ** -24 * size
                got, zb = o[at:at + n], z[at:at + n]
                assert np.array_equal(np.isneginf(L), np.isneginf(zb)), f"sequence {b}: empty rows"
                assert np.array_equal(np.isnan(L), np.isnan(zb)), f"sequence {b}: NaN of lse"
                fin = np.isfinite(L)
                with np.errstate(invalid="ignore"):
                    err = np.abs(zb - L)[fin] - (ds + 2.0 ** -19 + 2.0 ** -22 * np.abs(L))[fin]
                assert (err <= 0).all(), f"sequence {b}: lse off by {err.max():.2e} too much"
                tol = H * np.abs(O) + (H + 2 * ds + 2.0 ** -18)[..., None] * spread
                good = np.isfinite(O)
                assert np.array_equal(np.isnan(O), np.isnan(got)), f"sequence {b}: NaN where there is none, or none"
                assert np.array_equal(got[~good], O[~good], equal_nan=True), f"sequence {b}: infinities"
                err = np.abs(got[good] - O[good]) - tol[good]
                assert (err <= 0).all(), f"sequence {b}: out off by {err.max():.2e} too much"
            at += n


# ------------------------------------------------------------ cache

@pytest.mark.parametrize("D,H_kv,page", [(128, 8, 64), (64, 1, 16), (128, 3, 256)])
@pytest.mark.parametrize("fp8", [False, True])
def test_write_and_read_back(D, H_kv, page, fp8):
    b = Batch([(1, 1), (37, 37), (0, 20), (5, 300), (16, 16)], H_kv, H_kv, D, page, fp8, seed=1)
    for x in b.k + b.v:        # magnitudes from the subnormal end of bf16 to its top
        x *= torch.from_numpy(np.exp2(b.rng.integers(-130, 120, (len(x), H_kv, 1))).astype(np.float32)).cuda()
    before = [None if t is None else t.clone() for t in (b.cache.k, b.cache.v, b.cache.k_scale, b.cache.v_scale)]
    b.write()
    k, v = dsa.kv_cache_read(b.cache, b.kv_len, b.table, out=tuple(
        torch.full((len(b.seqs), 310, H_kv, D), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)))
    torch.cuda.synchronize()
    used = np.zeros((b.cache.k.shape[0], page), bool)
    for s, (_, t) in enumerate(b.seqs):
        pos = np.arange(t)
        pages = b.table[s].cpu().numpy()[pos // page]
        used[pages, pos % page] = True
        for got, x, pg, sc in ((k, b.k, b.cache.k, b.cache.k_scale), (v, b.v, b.cache.v, b.cache.v_scale)):
            want = f64(x[s])
            if fp8:
                codes, e = paged.quantise(want)
                assert np.array_equal(pg.cpu().numpy()[pages, pos % page], codes)
                assert np.array_equal(sc.cpu().numpy()[pages, pos % page].astype(int) - 127, e)
                want = paged.dequantise(codes, e)
            assert np.array_equal(f64(got[s, :t]), want)
            assert (got[s, t:] == 7.0).all()          # behind the end: as it was
    # nothing but the sequences' slots was touched
    for t, old in zip((b.cache.k, b.cache.v, b.cache.k_scale, b.cache.v_scale), before):
        if t is not None:
            a, o = (x.cpu().view(torch.uint8 if x.dtype == torch.uint8 else torch.int16).numpy() for x in (t, old))
            assert np.array_equal(a[~used], o[~used])


def test_quantise_special_values():
    D, rows = 64, []
    g = paged.e4m3_grid()
    for e in (-116, -20, -1, 0, 1, 30, 118):
        for base in range(0, 126, 21):           # the grid, its midpoints and both neighbours
            x = np.concatenate([g[base:base + 21], (g[base:base + 21] + g[base + 1:base + 22]) / 2])
            x = np.concatenate([[448.0], x, -x[:21]])
            rows.append(np.ldexp(np.pad(x, (0, D - len(x))), e))
    inf, nan, top = np.inf, np.nan, float(torch.finfo(torch.bfloat16).max)
    for x in ([0.0], [-0.0, 0.0], [nan, 1.0, -2.0], [inf, 1.0], [-inf, 3.0, nan], [inf, -inf], [nan] * D,
              [top, 1e30, -top], [1.75 * 2.0 ** 127], [2.0 ** -133], [2.0 ** -126, 2.0 ** -133], [0.875], [0.879]):
        rows.append(np.pad(np.array(x), (0, D - len(x))))
    x = torch.tensor(np.array(rows), dtype=torch.float64).to(torch.bfloat16)[:, None].cuda()
    n = len(rows)
    cache = dsa.PagedKVCache.empty(-(-n // 16), 16, 1, D, fp8=True)
    table = torch.arange(-(-n // 16), dtype=torch.int32, device="cuda")[None]
    qs, kl = torch.tensor([0, n], dtype=torch.int32).cuda(), torch.tensor([n], dtype=torch.int32).cuda()
    dsa.kv_cache_write(cache, x, x, qs, kl, table)
    k, v = dsa.kv_cache_read(cache, kl, table, T_max=n)
    codes, e = paged.quantise(f64(x))
    got = cache.k.view(-1, 1, D)[:n].cpu().numpy()
    row = e != paged.E_NAN                     # a row with a NaN is known by its scale alone
    assert np.array_equal(got[row], codes[row])
    assert np.array_equal(cache.k_scale.view(-1, 1)[:n].cpu().numpy().astype(int) - 127, e)
    want = paged.dequantise(codes, e)
    assert np.array_equal(f64(k[0]), want, equal_nan=True) and np.array_equal(f64(v[0]), want, equal_nan=True)


# ------------------------------------------------------------ attention

CASES = [
    # (sequences (new, total), H_q, H_kv, D, page)
    ([(1, 1)], 4, 1, 128, 16),
    ([(1, 200)], 8, 2, 128, 64),
    ([(1, 5000)], 8, 2, 128, 64),
    ([(1, 127), (1, 128), (1, 129), (1, 3), (1, 1000)], 16, 4, 128, 32),
    ([(7, 7), (3, 500), (1, 130)], 8, 1, 64, 16),
    ([(32, 32), (33, 33), (64, 64), (65, 300)], 8, 2, 128, 128),
    ([(300, 1000), (1, 900), (0, 50), (129, 129)], 8, 2, 128, 64),
    ([(257, 257)], 2, 2, 64, 128),
    ([(200, 1500)], 6, 1, 128, 16),
    ([(70, 700)], 7, 1, 64, 512),
    ([(40, 41)], 128, 1, 128, 64),
    ([(512, 2048)], 4, 4, 128, 1024),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_attention_over_all_keys(case, fp8):
    seqs, H_q, H_kv, D, page = CASES[case]
    b = Batch(seqs, H_q, H_kv, D, page, fp8, seed=10 + case).write()
    b.check(*b.attn())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n_sink,n_stream", [(0, 0), (5, 0), (0, 1), (0, 128), (1, 100), (130, 257), (300, 64),
                                             (64, 100000)])
def test_attention_window_and_sinks(n_sink, n_stream, fp8):
    b = Batch([(1, 1), (1, 700), (300, 900), (40, 45), (129, 640)], 8, 2, 128, 32, fp8, seed=40).write()
    b.check(*b.attn(n_sink=n_sink, n_stream=n_stream), n_sink=n_sink, n_stream=n_stream)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n_sink,n_stream", [(0, None), (40, 100)])
@pytest.mark.parametrize("seqs", [[(1, 300), (60, 60), (7, 200)], [(300, 900), (150, 150)]])
def test_infinities_and_nan_reach_only_who_sees_them(seqs, n_sink, n_stream, fp8):
    """Value rows (and one key row) of some tokens hold infinities or NaN: rows that do not see
    them -- earlier ones of the chunk, later ones beyond the window -- get their plain result."""
    b = Batch(seqs, 8, 2, 128, 32, fp8, seed=50)
    for s, (n, t) in enumerate(seqs):
        for j, x in ((t - 1, float("nan")), (t - n // 2 - 1, float("inf")), (max(0, t - n - 30), float("-inf")), (5, float("nan"))):
            b.v[s][j, 0, 3 + j % 7] = x
    b.k[-1][seqs[-1][1] - 9, 1, 0] = float("nan")
    b.write()
    if fp8:   # a row with a NaN is NaN throughout; an infinity saturates
        assert np.isnan(b.held(0)[1][5, 0]).all()
    b.check(*b.attn(n_sink=n_sink, n_stream=n_stream), n_sink=n_sink, n_stream=n_stream)


def test_nan_recomputed_across_shares():
    """The same where the launch cuts the item into pieces, and with one query tile."""
    for seqs in ([(3, 9000)], [(40, 9000)]):
        b = Batch(seqs, 4, 1, 64, 64, False, seed=51)
        b.v[0][-1, 0, 7] = float("nan")
        b.v[0][-2, 0, 9] = float("inf")
        b.write()
        b.check(*b.attn())


def test_nan_in_every_item_of_a_long_context():
    """Token 64 m + 40 of a chunk holds a NaN (an infinity) in column m of its value row: rows
    from it on have it, the 40 tokens before it that share its tiles have a finite result, and
    the launch stays far inside the limit of its waits."""
    n, t = 8192, 65536
    b = Batch([(n, t)], 4, 1, 128, 128, False, seed=52)
    for m in range(128):
        b.v[0][t - n + 64 * m + 40, 0, m] = float("nan") if m % 2 else float("inf")
    b.write()
    out, lse = b.attn()
    torch.cuda.synchronize()
    row, col = torch.arange(n, device="cuda")[:, None], torch.arange(128, device="cuda")[None]
    hit = (row >= 64 * col + 40)[:, None].expand(n, 4, 128)
    odd = (col % 2 == 1)[:, None].expand(n, 4, 128)
    assert torch.equal(torch.isnan(out), hit & odd)
    assert torch.equal(torch.isposinf(out), hit & ~odd)
    assert torch.isfinite(lse).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("group", [1, 3, 4, 5, 32, 33])
@pytest.mark.parametrize("n_sink,n_stream", [(0, None), (40, 300)])
def test_few_rows_between_many(group, D, fp8, n_sink, n_stream):
    """Items of at most 32 rows, of one more, and of two tiles, handed out in turn."""
    t = max(32 // group, 1)
    two = 2 * (128 // group)
    seqs = [(t, 700), (two, two + 250), (1, 1), (t + 1, 130), (1, 128), (two + 1, two + 140), (1, 900), (t, t)]
    b = Batch(seqs, 2 * group, 2, D, 16, fp8, seed=20 + group).write()
    b.check(*b.attn(n_sink=n_sink, n_stream=n_stream), n_sink=n_sink, n_stream=n_stream)


@pytest.mark.parametrize("fp8", [False, True])
def test_large_scores_and_moving_references(fp8):
    """Scores of hundreds of units that grow along the keys: the softmax reference moves on
    almost every tile, and early tiles vanish against later ones."""
    b = Batch([(70, 1500), (1, 1500)], 8, 2, 128, 64, fp8, seed=52)
    for s in range(2):
        b.k[s] *= torch.linspace(0.1, 12.0, 1500, device="cuda")[:, None, None].bfloat16()
    b.write()
    b.check(*b.attn())
    b.check(*b.attn(scale=1e-4), scale=1e-4)


def test_values_at_the_top_of_the_range():
    b = Batch([(20, 400)], 4, 2, 128, 16, True, seed=53)
    b.v[0] *= 2.0 ** 100
    b.k[0] *= 2.0 ** -100
    b.write()
    b.check(*b.attn())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("page", [16, 64, 128, 256])
def test_bad_pages_are_skipped(page, fp8):
    b = Batch([(1, 700), (50, 700), (40, 40)], 8, 2, 128, page, fp8, seed=54).write()
    lost, table = [], b.table.cpu().numpy()
    for s, (_, t) in enumerate(b.seqs):
        i = np.arange(-(-t // page))
        table[s, i[1::3]] = [-1, b.cache.k.shape[0], 2 ** 31 - 1][s]
        lost.append(np.isin(np.arange(t) // page, i[1::3]))
    b.table.copy_(torch.from_numpy(table))
    b.check(*b.attn(), lost=lost)
    k, _ = dsa.kv_cache_read(b.cache, b.kv_len, b.table)
    for s, (_, t) in enumerate(b.seqs):
        want = np.where(lost[s][:, None, None], 0.0, b.held(s)[0])
        assert np.array_equal(f64(k[s, :t]), want)


def test_rows_outside_the_chunks_and_short_lengths():
    """Token rows before q_start[0] and behind q_start[B] stay as they were; a chunk longer than
    its kv_len has rows at negative positions, which see nothing and are not written."""
    b = Batch([(40, 100), (300, 300)], 4, 1, 128, 64, False, seed=55)
    q = torch.cat([b.rows(5, 4), b.q, b.rows(130, 4)])
    start = b.q_start + 5
    b.write()
    out, lse = torch.full_like(q, 3.0), torch.full(q.shape[:2], 5.0, device="cuda")
    dsa.paged_attn(q, b.cache, start, b.kv_len, b.table, out=out, lse=lse)
    b.check(out[5:-130], lse[5:-130])
    for t, x in ((out, 3.0), (lse, 5.0)):
        assert (t[:5] == x).all() and (t[-130:] == x).all()
    short = torch.tensor([25, 10], dtype=torch.int32, device="cuda")      # of 40 and 300 rows
    before = b.cache.k.clone()
    dsa.kv_cache_write(b.cache, b.rows(b.N, 1), b.rows(b.N, 1), b.q_start, short, b.table)
    changed = (b.cache.k.view(torch.int16) != before.view(torch.int16)).flatten(2).any(2).sum()
    assert int(changed) == 35
    out, lse = b.attn()
    out, lse = dsa.paged_attn(b.q, b.cache, b.q_start, short, b.table)
    assert (out[:15] == 0).all() and torch.isneginf(lse[:15]).all() and torch.isfinite(lse[15:40]).all()
    assert (out[40:330] == 0).all() and torch.isneginf(lse[40:330]).all() and torch.isfinite(lse[330:]).all()


def test_no_tokens():
    b = Batch([(1, 10)], 4, 1, 64, 16, False, seed=56).write()
    none = torch.zeros(2, dtype=torch.int32, device="cuda")
    q = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    out, lse = dsa.paged_attn(q, b.cache, none, b.kv_len, b.table)
    assert out.shape == q.shape and lse.shape == (0, 4)
    dsa.kv_cache_write(b.cache, q[:, :1], q[:, :1], none, b.kv_len, b.table)
    b.check(*b.attn())


def test_many_sequences():
    rng = np.random.default_rng(57)
    seqs = [(int(rng.integers(0, 4)), int(rng.integers(4, 200))) for _ in range(700)]
    b = Batch(seqs, 4, 2, 64, 16, True, seed=57).write()
    b.check(*b.attn(), rows=range(0, 700, 23))


# ------------------------------------------------------------ as a program calls them

@pytest.mark.parametrize("D,group", [(128, 4), (64, 8), (128, 32)])
@pytest.mark.parametrize("n_sink,n_stream", [(0, None), (30, 90)])
def test_no_more_tokens_than_sequences(D, group, n_sink, n_stream):
    """FP8 launches that look like a decode step, with one token a sequence, and with thirty in
    one (an infinity and a NaN among their values) and none in most others."""
    even = [(1, 37 * i + 1) for i in range(40)]
    uneven = [(0, 33)] * 15 + [(30, 500)] + [(0, 0)] * 15 + [(1, 200 + i) for i in range(8)] + [(0, 70)]
    for seed, seqs in ((60, even), (61, uneven)):
        b = Batch(seqs, 2 * group, 2, D, 16, True, seed=seed)
        if seqs is uneven:
            b.v[15][480, 0, 5] = float("nan")
            b.v[15][490, 1, 6] = float("inf")
        b.write()
        b.check(*b.attn(n_sink=n_sink, n_stream=n_stream), n_sink=n_sink, n_stream=n_stream)


def test_strided_tokens():
    """q, k_new and v_new as slices of one fused projection."""
    b = Batch([(30, 90), (1, 50)], 8, 2, 128, 32, True, seed=60)
    b.write()
    qkv = torch.zeros(b.N, 12 * 128, dtype=torch.bfloat16, device="cuda")
    q, k, v = (x.view(b.N, -1, 128) for x in qkv.split([1024, 256, 256], dim=1))
    q.copy_(b.q)
    k.copy_(torch.cat([x[t - n:] for x, (n, t) in zip(b.k, b.seqs)]))
    v.copy_(torch.cat([x[t - n:] for x, (n, t) in zip(b.v, b.seqs)]))
    before = [t.clone() for t in (b.cache.k, b.cache.v, b.cache.k_scale, b.cache.v_scale)]
    dsa.kv_cache_write(b.cache, k, v, b.q_start, b.kv_len, b.table)
    for t, o in zip((b.cache.k, b.cache.v, b.cache.k_scale, b.cache.v_scale), before):
        assert torch.equal(t, o)
    out, lse = dsa.paged_attn(q, b.cache, b.q_start, b.kv_len, b.table)
    want, wl = b.attn()
    assert torch.equal(out, want) and torch.equal(lse, wl)


@pytest.mark.parametrize("fp8", [False, True])
def test_chunks_one_after_another_equal_the_whole_prompt(fp8):
    """A prompt in chunks, then single tokens: each step writes its rows and attends; every row
    matches the float64 attention of the whole, and the cache read back feeds the selection and
    the sparse decode, which attend the same window and sinks."""
    T, steps = 700, [300, 129, 128, 140, 1, 1, 1]
    b = Batch([(T, T)], 8, 2, 128, 64, fp8, seed=61)
    got, lse, at = [], [], 0
    for n in steps:
        qs = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        kl = torch.tensor([at + n], dtype=torch.int32, device="cuda")
        rows = slice(at, at + n)
        dsa.kv_cache_write(b.cache, b.k[0][rows], b.v[0][rows], qs, kl, b.table)
        o, z = dsa.paged_attn(b.q[rows], b.cache, qs, kl, b.table)
        got.append(o)
        lse.append(z)
        at += n
    b.check(torch.cat(got), torch.cat(lse))
    # the decode step of the contiguous path over the same cache: no selection, sinks and window
    k, v = dsa.kv_cache_read(b.cache, kl, b.table)
    q = b.q[-1:].view(1, 1, 8, 128)
    none, cnt = torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    o1, l1 = dsa.sparse_attn_decode(q, k, v, kl, none, cnt, n_sink=20, n_stream=200)
    o2, l2 = dsa.paged_attn(b.q[-1:], b.cache, qs, kl, b.table, n_sink=20, n_stream=200)
    torch.cuda.synchronize()
    # two roundings of P and of the result each (values are at most a few units)
    assert (o1.float().view(8, 128) - o2.float().view(8, 128)).abs().max() <= 4 * H * float(v.abs().max())
    assert (l1.view(-1) - l2.view(-1)).abs().max() <= 1e-3
    # and the selection runs over what was read back
    sel, n = dsa.hip_select(q, k, kl, dsa.HipConfig((64, 16), (128, 64), 20, 200))
    assert 0 < int(n[0]) <= 64 and int(sel[0, 0]) >= 20


def test_other_streams_graphs_and_repeats():
    b = Batch([(64, 700), (1, 3000), (200, 200)], 8, 2, 128, 64, True, seed=62).write()
    want, wl = b.attn()
    torch.cuda.synchronize()
    for _ in range(3):                                   # the same bits every time
        out, lse = b.attn()
        assert torch.equal(out, want) and torch.equal(lse, wl)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    s1.wait_stream(torch.cuda.current_stream())
    s2.wait_stream(torch.cuda.current_stream())
    o1, l1 = b.attn(stream=s1)                           # two calls at once
    with torch.cuda.stream(s2):
        o2, l2 = b.attn()
    torch.cuda.synchronize()
    for o, z in ((o1, l1), (o2, l2)):
        assert torch.equal(o, want) and torch.equal(z, wl)
    # two graphs with workspaces of their own, replayed side by side, on changed inputs
    graphs = []
    for _ in range(2):
        n = dsa.paged_attn_workspace_bytes(b.q, b.cache, b.table)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        out, lse = torch.empty_like(want), torch.empty_like(wl)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            k = torch.cat([x[t - n:] for x, (n, t) in zip(b.k, b.seqs)])
            v = torch.cat([x[t - n:] for x, (n, t) in zip(b.v, b.seqs)])
            dsa.kv_cache_write(b.cache, k, v, b.q_start, b.kv_len, b.table)
            b.attn(out=out, lse=lse, workspace=ws)
        graphs.append((g, out, lse))
    b.q.copy_(b.rows(b.N, 8))
    new, nl = b.attn()
    torch.cuda.synchronize()
    for (g, _, _), s in zip(graphs, (s1, s2)):
        with torch.cuda.stream(s):
            g.replay()
            g.replay()
    torch.cuda.synchronize()
    for _, out, lse in graphs:
        assert torch.equal(out, new) and torch.equal(lse, nl)
    b.check(new, nl)


def test_offsets_beyond_32_bits():
    """Pages whose first element lies beyond 2^31 elements of the cache."""
    page, heads, D = 64, 8, 128
    n = 2 ** 31 // (page * heads * D) + 40
    b = Batch([(33, 500), (1, 900)], 16, heads, D, page, False, seed=63)
    b.cache = dsa.PagedKVCache(*(torch.empty(n, page, heads, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)))
    t = b.table
    t[t >= 0] += n - 25
    b.write()
    b.check(*b.attn())
    k, _ = dsa.kv_cache_read(b.cache, b.kv_len, b.table)
    assert np.array_equal(f64(k[1, :900]), b.held(1)[0])


def test_waits_that_run_out():
    b = Batch([(100, 2000)], 8, 2, 128, 64, False, seed=64).write()
    want, wl = b.attn()
    torch.cuda.synchronize()
    try:
        dsa.set_wait_limit(1)
        b.attn()
        torch.cuda.synchronize()
        assert dsa.device_error() == 8
    finally:
        dsa.set_wait_limit(0)
    out, lse = b.attn()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, wl)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("fp8,seqs", [(False, [(300, 900), (1, 4000)]), (True, [(300, 900), (1, 4000)]),
                                      (True, [(1, 3000), (1, 500), (1, 9000)])])
def test_every_kernel_gives_up_and_repeats_itself(D, fp8, seqs):
    """Each form of the kernel: the same bits in ten calls in a row, the error word when its waits
    may not last, and the same bits again afterwards."""
    b = Batch(seqs, 8, 2, D, 32, fp8, seed=65).write()
    want, wl = b.attn()
    b.check(want, wl)
    for out, lse in [b.attn() for _ in range(10)]:
        assert torch.equal(out, want) and torch.equal(lse, wl)
    torch.cuda.synchronize()
    try:
        dsa.set_wait_limit(1)
        b.attn()
        torch.cuda.synchronize()
        assert dsa.device_error() == 8
    finally:
        dsa.set_wait_limit(0)
    out, lse = b.attn()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, wl)


def test_items_longer_than_the_wait_limit():
    """A wait is bounded per key tile, not per item: items of 160 tiles on average (some 300 us
    each) under a limit of 100 us."""
    b = Batch([(40960, 40960)], 1, 1, 64, 128, False, seed=31).write()
    try:
        dsa.set_wait_limit(100_000)
        out, lse = b.attn()
        torch.cuda.synchronize()
        assert dsa.device_error() == 0
    finally:
        dsa.set_wait_limit(0)
    want, want_lse = b.attn()
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


def test_arguments_on_the_gpu():
    b = Batch([(4, 40)], 8, 2, 128, 16, True, seed=65).write()
    bad = [dict(n_sink=-1), dict(n_stream=-2), dict(scale=0.0), dict(scale=float("nan"))]
    for kw in bad:
        with pytest.raises((dsa.DsaError, ValueError)):
            b.attn(**kw)
    with pytest.raises(ValueError):
        b.attn(out=torch.empty(4, 8, 128, device="cuda"))
    with pytest.raises(dsa.DsaError):
        b.attn(workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        dsa.paged_attn(b.q.transpose(0, 1), b.cache, b.q_start, b.kv_len, b.table)
    with pytest.raises(TypeError):
        dsa.paged_attn(b.q, b.cache, b.q_start.long(), b.kv_len, b.table)
    with pytest.raises(ValueError):
        dsa.paged_attn(b.q, dsa.PagedKVCache(b.cache.k, b.cache.v), b.q_start, b.kv_len, b.table)
    with pytest.raises(ValueError):
        dsa.kv_cache_read(b.cache, b.kv_len, b.table, out=(b.q, b.q))
    with pytest.raises(dsa.DsaError):                    # 24-token pages
        c = dsa.PagedKVCache.empty(4, 24, 2, 128)
        dsa.kv_cache_read(c, b.kv_len, b.table)
    torch.cuda.synchronize()
    b.check(*b.attn())


# ------------------------------------------------------------ NaN and infinite scores

# items of one token, of one query tile (whole and cut), of two (whole and cut): each with its own epilogue and merge
NAN_SEQS = [[(1, 1)], [(1, 1), (1, 300), (1, 40), (5, 5)], [(20, 20), (3, 3000)], [(60, 60), (64, 100), (40, 41)],
            [(300, 4000)], [(1, 4000)], [(1, 9000 - 31 * i) for i in range(12)]]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n_sink,n_stream", [(0, None), (40, 300)])
@pytest.mark.parametrize("seqs", range(len(NAN_SEQS)))
def test_nan_queries(seqs, n_sink, n_stream, D, fp8):
    """A NaN in a query row (one head of some tokens) comes out as NaN there, and only there."""
    b = Batch(NAN_SEQS[seqs], 8, 2, D, 32, fp8, seed=70 + seqs).write()
    b.q[::3, 1, 5] = float("nan")
    b.q[-1, 6, D - 1] = float("nan")
    b.check(*b.attn(n_sink=n_sink, n_stream=n_stream), n_sink=n_sink, n_stream=n_stream)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("seqs", range(len(NAN_SEQS)))
def test_nan_keys_alone_in_sight(seqs, D, fp8):
    """Rows whose only key is NaN, and keys of NaN that fill whole tiles and pieces of a cut item:
    whoever sees one is NaN, however the launch was cut."""
    b = Batch(NAN_SEQS[seqs], 8, 2, D, 32, fp8, seed=80 + seqs)
    for s, (_, t) in enumerate(b.seqs):
        b.k[s][0, 1, 3] = float("nan")                     # head 1: every row
        b.k[s][t // 4:t // 2, 0, 2] = float("nan")         # head 0: a quarter of the context
    b.write()
    b.check(*b.attn())
    b.check(*b.attn(n_sink=0, n_stream=1), n_sink=0, n_stream=1)
    b.check(*b.attn(n_sink=1, n_stream=0), n_sink=1, n_stream=0)
    b.check(*b.attn(n_sink=0, n_stream=900), n_sink=0, n_stream=900)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("seqs", range(len(NAN_SEQS)))
def test_infinite_scores(seqs, D):
    """Plus infinity among a row's scores makes it NaN, minus infinity is a weight of 0; a row that
    has nothing else is empty."""
    b = Batch(NAN_SEQS[seqs], 8, 2, D, 32, False, seed=90 + seqs)
    b.q.copy_(b.q.abs() + 0.01)
    for s, (_, t) in enumerate(b.seqs):
        b.k[s][t // 4:t // 2 + 1, 0, 2] = float("-inf")
        b.k[s][3 * t // 4, 1, 0] = float("inf")
    b.write()
    b.check(*b.attn())
    b.check(*b.attn(n_sink=0, n_stream=1), n_sink=0, n_stream=1)
    b.check(*b.attn(n_sink=0, n_stream=900), n_sink=0, n_stream=900)


@pytest.mark.parametrize("D", [64, 128])
def test_nan_keys_of_one_piece(D):
    """Two or three tiles of NaN keys at every place of a context: one of them is the whole of a cut
    item's piece, whose other pieces are finite."""
    t = 3000
    b = Batch([(300, t)], 8, 2, D, 32, False, seed=99)
    good = b.k[0].clone()
    for tiles in (2, 3):
        for at in range(0, 2700 // 128 - tiles):
            b.k[0].copy_(good)
            b.k[0][128 * at:128 * (at + tiles), 1, 0] = float("nan")
            out, lse = b.write().attn()
            assert torch.isnan(out[:, 4:]).all() and torch.isnan(lse[:, 4:]).all(), (tiles, at)
            assert torch.isfinite(out[:, :4]).all() and torch.isfinite(lse[:, :4]).all()


# ------------------------------------------------------------ infinities and NaN of little weight

@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("seqs,bad,heavy", [([(1, 200)], 10, 128), ([(1, 300)], 140, 256), ([(1, 250)], 140, 0),
                                            ([(60, 400)], 10, 256), ([(3, 9000)], 10, 8000), ([(1, 9000)], 8500, 0),
                                            ([(300, 4000)], 10, 3600), ([(300, 4000)], 3000, 0),
                                            ([(1, 300), (1, 400), (1, 9000)], 140, 256)])
def test_bad_values_whose_weight_vanishes(seqs, bad, heavy, D, fp8):
    """Key `bad` weighs less than 2^-500 of the keys from `heavy` on (of the 100 first ones), and its
    value row holds a NaN and an infinity: there every row's result is infinite or NaN, however the
    launch was cut, and as without it everywhere else."""
    b = Batch(seqs, 8, 2, D, 32, fp8, seed=100)
    b.q.fill_(1.0)
    for s, (_, t) in enumerate(seqs):
        b.k[s].fill_(0.0)
        b.k[s][heavy:heavy + 100 if heavy == 0 else t] = 64.0      # scores of 64 sqrt(D) and 0
        b.v[s][bad, 0, 7], b.v[s][bad, 0, 9] = float("nan"), float("inf")
    b.write()
    out, lse = b.attn()
    at = 0
    for s, (n, t) in enumerate(seqs):
        k, v = b.held(s)
        O, L, spread, _ = paged.attend(f64(b.q)[at:at + n], k, v, t - n, 0, None, D ** -0.5)
        got, z = f64(out)[at:at + n], lse[at:at + n].cpu().numpy().astype(np.float64)
        assert (np.isfinite(O) == np.isfinite(got)).all()
        assert not np.isfinite(got[:, :4, 7]).any() and np.isfinite(got[:, 4:]).all()
        # dot products are exact: the scale, log2 e, their product, its product with the score, the sum
        # with log2 l, ln 2 and the product with that are seven roundings
        assert (np.abs(z - L) <= 2.0 ** -19 + 7 * 2.0 ** -24 * np.abs(L)).all()
        good = np.isfinite(O)
        assert (np.abs(got - O)[good] <= (H * np.abs(O) + (H + 2.0 ** -18) * spread)[good]).all()
        at += n


def test_rows_without_weight_have_no_bad_values():
    """Every score of a row is minus infinity: it is empty, whatever its value rows hold, in tiles that
    the mask cuts and in others."""
    for n in (1, 5, 70):
        b = Batch([(n, 400), (n, n)], 4, 1, 128, 32, False, seed=101)
        b.q.fill_(1.0)
        for s in range(2):
            b.k[s].fill_(float("-inf"))
            b.v[s][0, 0, 3], b.v[s][-1, 0, 4] = float("inf"), float("nan")
        out, lse = b.write().attn()
        assert (out == 0).all() and torch.isneginf(lse).all()


# ------------------------------------------------------------ scales that the writer never makes

def bf16_of(x):
    """float64 -> the nearest bf16 (ties to even, subnormals and overflow as IEEE) as float64.  x has
    few bits, so that fp32 holds it exactly unless it overflows."""
    with np.errstate(over="ignore"):
        return torch.from_numpy(x.astype(np.float32)).bfloat16().double().numpy()


SCALES = [0, 1, 2, 3, 10, 11, 127, 134, 135, 246, 247, 250, 254]


def hand_made(D):
    """Pages of 16 rows with every scale byte of SCALES and every code but the NaN's."""
    codes = np.array([c for c in range(256) if c & 127 != 127], np.uint8)
    rows = -(-len(codes) // D)
    n = len(SCALES) * rows
    pages = -(-n // 16)
    c = np.zeros((pages * 16, D), np.uint8)
    e = np.zeros(pages * 16, np.uint8)
    for i, s in enumerate(SCALES):
        c[i * rows:(i + 1) * rows].flat[:len(codes)] = codes
        e[i * rows:(i + 1) * rows] = s
    cache = dsa.PagedKVCache(*(torch.from_numpy(c).cuda().view(pages, 16, 1, D).clone() for _ in range(2)),
                             *(torch.from_numpy(e).cuda().view(pages, 16, 1).clone() for _ in range(2)))
    return cache, bf16_of(paged.dequantise(c[:n], e[:n].astype(int) - 127)), n


@pytest.mark.parametrize("D", [64, 128])
def test_every_scale_byte_reads_as_its_power_of_two(D):
    cache, want, n = hand_made(D)
    table = torch.arange(cache.k.shape[0], dtype=torch.int32, device="cuda")[None]
    k, v = dsa.kv_cache_read(cache, torch.tensor([n], dtype=torch.int32, device="cuda"), table, T_max=n)
    for x in (k, v):
        assert np.array_equal(f64(x[0, :, 0]), want)


@pytest.mark.parametrize("D", [64, 128])
def test_every_scale_byte_is_attended_as_it_is_read(D):
    """Rows of one key each: their result is its value, as the cache reads back."""
    cache, want, n = hand_made(D)
    table = torch.arange(cache.k.shape[0], dtype=torch.int32, device="cuda")[None]
    q = torch.zeros(n, 2, D, dtype=torch.bfloat16, device="cuda")
    cache.k.zero_()
    kl = torch.tensor([n], dtype=torch.int32, device="cuda")
    for tokens in (1, n):                                   # decode form, general form
        for at in range(0, n, tokens):
            qs = torch.tensor([0, tokens], dtype=torch.int32, device="cuda")
            out, lse = dsa.paged_attn(q[:tokens], cache, qs, kl * 0 + at + tokens, table, n_stream=1)
            got, w = f64(out), want[at:at + tokens, None]
            normal = (np.abs(w) >= 2.0 ** -126) | (w == 0)  # smaller products may be flushed
            assert np.where(normal, got == w, np.abs(got) <= 2.0 ** -126).all()
            assert (lse == 0).all()


@pytest.mark.parametrize("fp8_few", [True, False])
@pytest.mark.parametrize("D", [64, 128])
def test_large_scales_reach_only_who_sees_them(D, fp8_few):
    """Values that a large scale makes infinite in bf16: rows before them keep a finite result, rows
    that see them get the infinity."""
    n = 8 if fp8_few else 100
    for T, at in ((n, n // 2), (700, 699), (700, 700 - n + 1)):
        b = Batch([(n, T)], 4, 1, D, 32, True, seed=102).write()
        page, slot = int(b.table[0, at // 32]), at % 32
        b.cache.v_scale[page, slot] = 254                  # code * 2^127
        b.cache.v[page, slot, 0] = 0x01                    # 2^-9 * 2^127
        b.cache.v[page, slot, 0, 5] = 0x7E                 # 448 * 2^127
        b.cache.v[page, slot, 0, D - 1] = 0xC0             # -2 * 2^127
        out, lse = b.attn()
        got = f64(out)
        sees = np.arange(T - n, T) >= at
        assert np.isposinf(got[sees][:, :, 5]).all() and np.isneginf(got[sees][:, :, D - 1]).all()
        assert np.isfinite(np.delete(got, (5, D - 1), 2)).all() and np.isfinite(lse.cpu().numpy()).all()
        assert np.isfinite(got[~sees]).all()
        keep = np.flatnonzero(~sees)
        if len(keep):
            k, v = b.held(0)
            O, L, spread, size = paged.attend(f64(b.q)[keep], k, v, T - n, 0, None, D ** -0.5)
            ds = 2 * D * 2.0 ** -24 * size[..., None]
            assert (np.abs(got[keep] - O) <= H * np.abs(O) + (H + 2 * ds + 2.0 ** -18) * spread).all()
