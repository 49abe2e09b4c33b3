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

    def check(self, out, lse, n_sink=0, n_stream=None, scale=None, rows=None):
        torch.cuda.synchronize()
        scale = self.D ** -0.5 if scale is None else scale
        o, z, q = f64(out), lse.cpu().numpy().astype(np.float64), f64(self.q)
        at = 0
        for b, (n, t) in enumerate(self.seqs):
            if n and (rows is None or b in rows):
                k, v = self.held(b)
                O, L, spread, size = paged.attend(q[at:at + n], k, v, t - n, n_sink, n_stream, scale)
                ds = 2 * self.D * 2.0 ** -24 * size
                got, zb = o[at:at + n], z[at:at + n]
                assert np.array_equal(np.isneginf(L), np.isneginf(zb)), f"sequence {b}: empty rows"
                fin = np.isfinite(L)
                with np.errstate(invalid="ignore"):
                    err = np.abs(zb - L)[fin] - (ds + 2.0 ** -19 + 2.0 ** -22 * np.abs(L))[fin]
                assert (err <= 0).all(), f"sequence {b}: lse off by {err.max():.2e} too much"
                tol = H * np.abs(O) + (H + 2 * ds + 2.0 ** -18)[..., None] * spread
                good = np.isfinite(O)
                assert np.array_equal(good, np.isfinite(got)), f"sequence {b}: {np.sum(good != np.isfinite(got))} rows"
                err = np.abs(got - O)[good] - tol[good]
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
