"""GPU parity of the operators around the paged cache's sparse path (kv_cache_write_rope,
page_digest_update, page_select, paged_attn over lists, kv_pages_copy) against the float64
restatements in oracle/pages.py and oracle/paged.py.

Tolerances (set before the first run).  Digests, lists and copies are compared exactly.  Rotated
rows, with h = finfo(t).eps / 2 the half step of the type that holds them (bf16 2^-8, e4m3 2^-4 and
half of its smallest step, 2^-10, times the row's scale) and size = |y_a| + |y_b| for a pair (|y|
for a dimension that is not rotated):
  h |y| for the one rounding, and F * size for fp32 on the way: a mean of D <= 128 squares is off by at
  most D 2^-24 relative and half of that after the root, a reciprocal root and three products by 2^-21,
  cosine and sine by 2^-22 (their own two steps and the angle's 2^-25 of a half turn), two products and a
  sum by 2^-22: together below F = 2^-16.
Attention over lists has the tolerances of test_gpu_paged.py.
"""
import numpy as np
import pytest
import torch

import dynamic_sparse_attention_gb300 as dsa
from dynamic_sparse_attention_gb300 import _build
from oracle import paged, pages
from oracle.numerics import to_f64
from parity import from_dev_bits

pytestmark = pytest.mark.gpu

H, F = 2.0 ** -8, 2.0 ** -16


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
    return to_f64(from_dev_bits(t.contiguous()), "bf16")


def ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32).cuda()


class Batch:
    """Ragged sequences (new, total) over a cache whose pages start with a value of their own."""

    def __init__(self, seqs, H_q, H_kv, D, page, fp8, seed=0, spare=3, max_pages=None, n_pages=None):
        self.rng = np.random.default_rng(seed)
        self.seqs, self.H_q, self.H_kv, self.D, self.page, self.fp8 = seqs, H_q, H_kv, D, page, fp8
        need = [-(-t // page) for _, t in seqs]
        self.n_pages = sum(need) + spare if n_pages is None else n_pages
        self.cache = dsa.PagedKVCache.empty(self.n_pages, page, H_kv, D, fp8=fp8)
        for t in (self.cache.k, self.cache.v, self.cache.k_scale, self.cache.v_scale):
            if t is not None:
                t.fill_(0x5D if fp8 else -3.0)
        order = self.rng.permutation(self.n_pages)
        self.table_np = np.full((len(seqs), max(max(need), 1) if max_pages is None else max_pages), -1, np.int32)
        at = 0
        for b, n in enumerate(need if sum(need) <= self.n_pages else []):
            self.table_np[b, :n] = order[at:at + n]
            at += n
        self.table = ints(self.table_np)
        self.n = [n for n, _ in seqs]
        self.N = sum(self.n)
        self.q_start = ints(np.cumsum([0] + self.n))
        self.kv_len = ints([t for _, t in seqs])
        self.digest = dsa.PageDigest.empty(self.cache)

    def rows(self, n, heads, gain=1.0):
        x = self.rng.standard_normal((n, heads, self.D), dtype=np.float32) * gain
        return torch.from_numpy(x).bfloat16().cuda()

    def fill(self, gain=1.0):
        """Every page's keys and values at random (as pages that nothing else is written to)."""
        P = self.n_pages
        start, lens, table = ints([0, P * self.page]), ints([P * self.page]), ints(np.arange(P)[None])
        k, v = self.rows(P * self.page, self.H_kv, gain), self.rows(P * self.page, self.H_kv)
        dsa.kv_cache_write(self.cache, k, v, start, lens, table)
        return self

    def held(self, page, what="k"):
        """A page's rows [page, H_kv, D] in float64 as the cache holds them."""
        t, s = (self.cache.k, self.cache.k_scale) if what == "k" else (self.cache.v, self.cache.v_scale)
        if not self.fp8:
            return f64(t[page])
        e = s[page].cpu().numpy().astype(int) - 127
        return paged.dequantise(t[page].view(torch.uint8).cpu().numpy(), e)

    def digest_all(self):
        dsa.page_digest_update(self.cache, self.digest, self.n_pages * self.page, ints([0, self.n_pages * self.page]),
                               ints([self.n_pages * self.page]), ints(np.arange(self.n_pages)[None]))
        return self


# ------------------------------------------------------------------ rotation on the way in

def freqs(rot, theta=1e4):
    return theta ** (-np.arange(0, rot, 2) / rot)


def write_rope(b, q, k, v, rot=None, norm=True, wdtype=torch.bfloat16, theta=1e4, eps=1e-6, **kw):
    rot = b.D if rot is None else rot
    w = [torch.from_numpy(1 + 0.3 * b.rng.standard_normal(b.D)).to(wdtype).cuda() if norm else None for _ in range(2)]
    f = torch.from_numpy(freqs(rot, theta)).cuda() if rot else None
    want = {}
    pos = np.concatenate([np.arange(t - n, t) for n, t in b.seqs])
    for name, x, ww in (("q", q, w[0]), ("k", k, w[1])):
        ww = None if ww is None else ww.double().cpu().numpy()
        want[name] = pages.rotate(f64(x), pos, ww, eps, None if f is None else freqs(rot, theta),
                                  kw.get("interleaved", False), kw.get("rope_scale", 1.0))
    out = dsa.kv_cache_write_rope(b.cache, q, k, v, b.q_start, b.kv_len, b.table, f, q_weight=w[0], k_weight=w[1],
                                  eps=eps, **kw)
    return out, want


def check_rows(b, got, want, size, name):
    err = np.abs(got - want)
    assert np.array_equal(np.isnan(got), np.isnan(want)), name
    ok = np.isfinite(want)
    assert (err <= H * np.abs(want) + F * size)[ok].all(), (name, float((err / (np.abs(want) + size + 1e-30))[ok].max()))


def check_cache_rows(b, want_k, size_k, v):
    """Keys within their rounding, values as kv_cache_write leaves them, nothing else touched."""
    twin = dsa.PagedKVCache(*(None if t is None else t.clone().fill_(0x5D if b.fp8 else -3.0)
                              for t in (b.cache.k, b.cache.v, b.cache.k_scale, b.cache.v_scale)))
    dsa.kv_cache_write(twin, v, v, b.q_start, b.kv_len, b.table)
    torch.cuda.synchronize()
    assert torch.equal(b.cache.v.view(torch.uint8), twin.v.view(torch.uint8))
    if b.fp8:
        assert torch.equal(b.cache.v_scale, twin.v_scale)
    touched = np.zeros((b.n_pages, b.page), bool)
    at = 0
    for s, (n, t) in enumerate(b.seqs):
        for i, p in enumerate(range(t - n, t)):
            pg = b.table_np[s, p // b.page] if p >= 0 else -1
            if 0 <= pg < b.n_pages:
                touched[pg, p % b.page] = True
                row = b.cache.k[pg, p % b.page]
                if b.fp8:
                    sb = b.cache.k_scale[pg, p % b.page].cpu().numpy().astype(int)
                    w, z = want_k[at + i], size_k[at + i]
                    a = np.abs(w).max(-1)
                    slack = F * z.max(-1)
                    low, high = paged.quantise((np.maximum(a - slack, 0) / 1.0)[:, None])[1], paged.quantise((a + slack)[:, None])[1]
                    assert ((sb - 127 >= low) & (sb - 127 <= high)).all(), (s, p)
                    got = paged.dequantise(row.view(torch.uint8).cpu().numpy(), sb - 127)
                    tol = 2.0 ** -4 * np.abs(w) + np.exp2(sb - 127.0 - 10)[:, None] + F * z
                    assert (np.abs(got - w) <= tol).all(), (s, p, float((np.abs(got - w) - tol).max()))
                else:
                    check_rows(b, f64(row), want_k[at + i], size_k[at + i], (s, p))
        at += n
    rest = torch.from_numpy(~touched).cuda()
    assert (b.cache.k.view(torch.uint8)[rest] == twin.k.view(torch.uint8)[rest]).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot,H_q,H_kv,page,norm,wdtype", [
    (128, None, 8, 2, 64, True, torch.bfloat16), (128, 64, 4, 4, 16, True, torch.float32), (128, 48, 6, 1, 32, False, None),
    (64, None, 5, 5, 128, True, torch.bfloat16), (64, 32, 12, 2, 16, True, torch.float32), (64, 16, 1, 1, 64, False, None)])
def test_rope_rows(D, rot, H_q, H_kv, page, norm, wdtype, interleaved, fp8):
    b = Batch([(1, 1), (37, 90), (0, 50), (1, 333), (16, 16)], H_q, H_kv, D, page, fp8, seed=D + H_q)
    fused = b.rows(b.N, H_q + 2 * H_kv, 2.0)                # slices of one projection
    q, k, v = fused[:, :H_q], fused[:, H_q:H_q + H_kv], fused[:, H_q + H_kv:]
    out, want = write_rope(b, q, k, v, rot, norm, wdtype, interleaved=interleaved, rope_scale=1.0 if norm else 0.75)
    check_rows(b, f64(out), *want["q"], "q")
    check_cache_rows(b, *want["k"], v)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n", [1, 15, 700, 4999])
def test_without_norm_and_rotation_it_is_the_plain_write(n, fp8):
    b = Batch([(n, n + 77), (3, 3)], 8, 2, 128, 32, fp8)
    q, k, v = b.rows(b.N, 8), b.rows(b.N, 2), b.rows(b.N, 2)
    k[0, 0, 5], v[1, 1, 7], k[2, 1, :3], v[3 % b.N, 0] = float("inf"), float("nan"), float("-inf"), 0.0
    out = dsa.kv_cache_write_rope(b.cache, q, k, v, b.q_start, b.kv_len, b.table, None)
    twin = Batch([(n, n + 77), (3, 3)], 8, 2, 128, 32, fp8)
    dsa.kv_cache_write(twin.cache, k, v, b.q_start, b.kv_len, b.table)
    assert torch.equal(out.view(torch.int16), q.view(torch.int16))
    for x, y in ((b.cache.k, twin.cache.k), (b.cache.v, twin.cache.v), (b.cache.k_scale, twin.cache.k_scale),
                 (b.cache.v_scale, twin.cache.v_scale)):
        assert x is None or torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_rope_in_place_and_far_positions():
    """Rows near position 2^30, rotated where they stand in the projection."""
    page, far = 1024, (1 << 30) - 3
    b = Batch([(5, 5)], 4, 2, 128, page, False, n_pages=4, max_pages=1 << 20)
    b.table_np[:] = -1
    b.table_np[0, -1] = 2
    b.table, b.seqs, b.kv_len = ints(b.table_np), [(5, far)], ints([far])
    fused = b.rows(5, 8)
    q, k, v = fused[:, :4], fused[:, 4:6], fused[:, 6:]
    before = fused.clone()
    out, want = write_rope(b, q, k, v, theta=5e5, q_out=q)
    assert out.data_ptr() == q.data_ptr() and torch.equal(fused[:, 4:], before[:, 4:])
    # (this oracle's angles are products rounded to 2^-53 of 2^30, off by 2^-23; the library's
    # frequencies, held to 2^-52 of themselves, by 2^-22: inside F)
    check_rows(b, f64(out), *want["q"], "q")
    check_rows(b, f64(b.cache.k[2, (far - 5) % page:(far - 5) % page + 5]), *want["k"], "k")


def test_rope_rows_of_bad_numbers_and_bad_pages():
    """A NaN or infinity stays in its row; a token without a page still gets its query; tokens outside
    every chunk are left alone."""
    for fp8 in (False, True):
        b = Batch([(6, 70), (4, 20)], 4, 2, 64, 16, fp8, seed=3)
        q, k, v = b.rows(12, 4), b.rows(12, 2), b.rows(12, 2)
        b.q_start = ints([1, 7, 11])                        # rows 0 and 11 belong to nobody
        clean = dsa.PagedKVCache(*(None if t is None else t.clone() for t in
                                   (b.cache.k, b.cache.v, b.cache.k_scale, b.cache.v_scale)))
        f = torch.from_numpy(freqs(64)).cuda()
        w = torch.ones(64, device="cuda")
        call = lambda c, q, k, table: dsa.kv_cache_write_rope(c, q, k, v, b.q_start, b.kv_len, table, f, q_weight=w,
                                                               k_weight=w, q_out=torch.full_like(q, 9.0))
        plain = call(clean, q, k, b.table)
        q2, k2 = q.clone(), k.clone()
        q2[3, 1, 7], k2[5, 0, 3] = float("nan"), float("inf")
        table = b.table_np.copy()
        table[1, 1] = 99                                    # positions 16 .. of sequence 1
        got = call(b.cache, q2, k2, ints(table))
        assert (got[[0, 11]] == 9.0).all() and torch.isnan(got[3, 1]).all()
        same = torch.ones(12, 4, dtype=torch.bool, device="cuda")
        same[3, 1] = False
        assert torch.equal(got[same], plain[same])
        pg, p = b.table_np[0, 68 // 16], 68 % 16            # row 5: position 64 + 4
        if fp8:
            assert b.cache.k_scale[pg, p, 0] == 255 and b.cache.k_scale[pg, p, 1] != 255
        else:
            assert torch.isnan(b.cache.k[pg, p, 0, [3, 35]]).all() and torch.isfinite(b.cache.k[pg, p, 1]).all()
        lost = b.table_np[1, 1]
        assert (b.cache.k[lost].view(torch.uint8) == (0x5D if fp8 else torch.full((16, 2, 64), -3.0).bfloat16()
                                                      .view(torch.uint8).cuda())).all()
        keep = torch.ones(b.n_pages, 16, 2, dtype=torch.bool, device="cuda")
        keep[lost] = False
        keep[pg, p, 0] = False
        assert torch.equal(b.cache.k[keep].view(torch.uint8), clean.k[keep].view(torch.uint8))


# ------------------------------------------------------------------ digests

def check_digest(b, page, keys, what=None):
    lo, hi, e = zip(*(pages.digest(b.held(page)[:keys, h]) for h in range(b.H_kv)))
    got = b.digest.bounds[page].cpu().numpy().astype(int)
    assert np.array_equal(got[:, 0], lo) and np.array_equal(got[:, 1], hi), (page, keys, what)
    assert b.digest.exp[page].tolist() == list(e), (page, keys, what)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D,H_kv,page,seqs", [
    (128, 8, 64, [(1, 100), (1, 64), (1, 65), (1, 1)]), (64, 1, 16, [(200, 200), (33, 70), (0, 90), (5, 16)]),
    (128, 3, 32, [(700, 1000)]), (64, 5, 128, [(1, 4), (300, 301)]), (128, 2, 1024, [(2500, 3000), (1, 1025)]),
    (128, 4, 16, [(5000, 5003)])])
def test_digests(D, H_kv, page, seqs, fp8):
    b = Batch(seqs, H_kv, H_kv, D, page, fp8, seed=page).fill(3.0)
    b.digest.bounds.fill_(77)
    b.digest.exp.fill_(7)
    dsa.page_digest_update(b.cache, b.digest, b.N, b.q_start, b.kv_len, b.table)
    touched = set()
    for s, (n, t) in enumerate(seqs):
        for i in range((t - n) // page, -(-t // page) if n else 0):
            pg = int(b.table_np[s, i])
            touched.add(pg)
            if len(touched) < 60 or i % 17 == 0:
                check_digest(b, pg, min(page, t - i * page))
    rest = [p for p in range(b.n_pages) if p not in touched]
    assert (b.digest.bounds[rest] == 77).all() and (b.digest.exp[rest] == 7).all()


def test_digests_of_numbers_that_are_none():
    b = Batch([(16 * 8, 16 * 8)], 2, 2, 64, 16, False)
    b.fill(1.0)
    t = b.cache.k
    P = [int(x) for x in b.table_np[0]]
    t[P[0], 3, 0, 5] = float("inf")                       # infinities saturate, the scale is the finite keys'
    t[P[0], 4, 0, 6] = float("-inf")
    t[P[1], 2, 1, 8] = float("nan")                       # one NaN counts as nothing
    t[P[2], :, 0] = float("nan")                          # nothing else there
    t[P[3], :, 1, 9] = float("inf")                       # a channel of infinities
    t[P[4]] = 0.0
    t[P[5], :, 0] *= 2.0 ** 70                            # past the exponent's range, both ways
    t[P[5], :, 1] *= 2.0 ** -70
    t[P[6], :, 0] = float("-inf")
    t[P[7], 0, 0, :4] = torch.tensor([127.0, -127.0, 127.5, 254.0])
    dsa.page_digest_update(b.cache, b.digest, b.N, b.q_start, b.kv_len, b.table)
    for p in P:
        check_digest(b, p, 16)
    q = Batch([(32, 32)], 2, 2, 128, 16, True)            # an FP8 row of NaN
    q.fill(1.0)
    q.cache.k_scale[q.table_np[0, 0], 4, 1] = 255
    dsa.page_digest_update(q.cache, q.digest, q.N, q.q_start, q.kv_len, q.table)
    for p in q.table_np[0]:
        check_digest(q, int(p), 16)


def test_digests_as_tokens_arrive():
    """Token by token and in chunks, the digests are those of the keys so far."""
    b = Batch([(1, 1), (1, 1)], 4, 2, 128, 16, True, n_pages=9, max_pages=4)
    b.table_np[:] = np.arange(8).reshape(2, 4)[::-1]
    b.table = ints(b.table_np)
    done = [0, 0]
    for n in ((1, 15), (1, 1), (13, 2), (1, 30), (20, 1)):
        done = [d + x for d, x in zip(done, n)]
        k = b.rows(sum(n), 2)
        start, lens = ints(np.cumsum([0, *n])), ints(done)
        dsa.kv_cache_write(b.cache, k, k, start, lens, b.table)
        dsa.page_digest_update(b.cache, b.digest, sum(n), start, lens, b.table)
        for s in range(2):
            for i in range(-(-done[s] // 16)):
                check_digest(b, int(b.table_np[s, i]), min(16, done[s] - 16 * i), (n, s))


# ------------------------------------------------------------------ selection

class Scores:
    def __init__(self, b, s):
        self.heads, self.b, self.s = b.H_kv, b, s
        P = -(-max(b.seqs[s][1], 0) // b.page)
        self.pg = b.table_np[s, :P]
        self.good = (self.pg >= 0) & (self.pg < b.n_pages)
        self.lo, self.hi = b.bounds_np[np.where(self.good, self.pg, 0)].transpose(2, 0, 1, 3)
        self.e = b.exp_np[np.where(self.good, self.pg, 0)]

    def __call__(self, rows, h):
        G = self.b.H_q // self.b.H_kv
        s = pages.bound(rows[:, h * G:(h + 1) * G].reshape(-1, self.b.D), self.lo[:, h], self.hi[:, h], self.e[:, h])
        return np.where(self.good, s, -np.inf)


def check_select(b, q, keep, n_sink, n_local, q_block, sel, rows0=0, some=None):
    torch.cuda.synchronize()
    b.bounds_np, b.exp_np = b.digest.bounds.cpu().numpy().astype(int), b.digest.exp.cpu().numpy().astype(int)
    start, lens = sel.q_start.cpu().numpy(), sel.kv_len.cpu().numpy()
    table, index = sel.page_table.cpu().numpy(), None if sel.index is None else sel.index.cpu().numpy()
    qf, at, j = f64(q), rows0, 0
    for s, (n, t) in enumerate(b.seqs):
        for i, rows, lists, keys in pages.select(qf[at:at + n], t - n, b.page, Scores(b, s), keep, n_sink, n_local, q_block):
            assert start[j] == at + i and lens[j] == keys, (s, i, lens[j], keys)
            for h in range(b.H_kv):
                want = np.full(table.shape[2], -1)
                if lists is not None:
                    want[:len(lists[h])] = lists[h]
                if index is not None:
                    assert np.array_equal(index[j, h], want), (s, i, h, index[j, h], want)
                assert np.array_equal(table[j, h], np.where(want < 0, -1, b.table_np[s, want])), (s, i, h)
            j += 1
        at += n
    # blocks behind the last one: no rows, no keys; all pages tie, so the earliest are picked
    assert (start[j:] == at).all() and (lens[j:] == 0).all()
    first = max(0, max(b.seqs[-1][1], 0) // b.page - n_local)
    s0 = min(n_sink, first)
    want = np.full(table.shape[2], -1)
    want[:max(0, min(keep, first) - s0)] = np.arange(s0, max(s0, min(keep, first)))
    assert (table[j:] == np.where(want < 0, -1, b.table_np[-1, want])).all()
    if index is not None:
        assert (index[j:] == want).all()


SELECT = [
    # seqs, H_q, H_kv, D, page, q_block, keep, n_sink, n_local
    ([(1, 3000), (1, 17), (1, 1), (1, 5000)], 8, 2, 128, 16, 1, 20, 1, 2),
    ([(1, 60000)], 8, 8, 64, 16, 1, 100, 2, 0),               # several CTAs an item
    ([(3, 2000), (0, 40), (5, 900)], 16, 1, 128, 32, 1, 7, 0, 1),
    ([(70, 3000)], 4, 4, 64, 16, 16, 9, 1, 3),                # 16 rows: few
    ([(70, 3000), (33, 40), (1, 2000)], 8, 4, 128, 16, 16, 12, 1, 2),   # 32 rows
    ([(200, 4000), (64, 64)], 8, 2, 128, 64, 16, 6, 1, 1),    # 64 rows
    ([(130, 9000)], 12, 2, 64, 64, 16, 11, 0, 0),             # 96 rows
    ([(300, 5000), (100, 1100)], 8, 2, 128, 32, 64, 10, 1, 2),          # 256 rows
    ([(200, 5000)], 32, 1, 128, 64, 128, 5, 1, 1),            # 4,096 rows in pieces
    ([(513, 2000)], 2, 2, 64, 128, 256, 3, 1, 0),
    ([(40, 700)], 8, 2, 128, 16, 8, 0, 2, 1),                 # nothing by score
    ([(40, 700)], 8, 2, 128, 16, 8, 1000, 0, 0),              # everything
]


@pytest.mark.parametrize("seqs,H_q,H_kv,D,page,q_block,keep,n_sink,n_local", SELECT)
def test_select(seqs, H_q, H_kv, D, page, q_block, keep, n_sink, n_local):
    b = Batch(seqs, H_q, H_kv, D, page, False, seed=H_q + D).fill(2.0).digest_all()
    q = b.rows(b.N, H_q + 1, 3.0)[:, :H_q]                    # (strided tokens)
    sel = dsa.page_select(q, b.digest, b.q_start, b.kv_len, b.table, keep=keep, n_sink=n_sink, n_local=n_local,
                          q_block=q_block, want_index=True)
    check_select(b, q, keep, n_sink, n_local, q_block, sel)


@pytest.mark.parametrize("q_block", [1, 8, 32])
def test_select_ties_and_odd_numbers(q_block):
    """Digests of a few values (whole rows of ties), exponents at both ends, queries with NaN, infinities
    and zeros, and pages that are none."""
    b = Batch([(33, 5000), (20, 300)], 8, 2, 128, 16, False, seed=q_block)
    g = torch.Generator(device="cuda").manual_seed(5)
    b.digest.bounds.random_(-1, 2, generator=g)
    b.digest.exp.fill_(3)
    b.digest.exp[::7] = 50
    b.digest.exp[3::11] = -50
    b.digest.bounds[5::9] = 0
    q = b.rows(b.N, 8)
    q[0] = 0.0
    q[1, 3] = float("nan")
    q[2, :, 4] = float("inf")
    q[3, 0, 5] = float("-inf")
    q[4] *= 2.0 ** 90
    q[5] *= 2.0 ** -90
    table = b.table_np.copy()
    table[0, 40:60] = (-1, b.n_pages, 10 ** 9, -5) * 5
    b.table_np, b.table = table, ints(table)
    for keep in (1, 37, 290):
        sel = dsa.page_select(q, b.digest, b.q_start, b.kv_len, b.table, keep=keep, n_local=0, q_block=q_block, want_index=True)
        check_select(b, q, keep, 1, 0, q_block, sel)


@pytest.mark.parametrize("q_block", [1, 4, 32])
def test_select_with_exponents_out_of_range(q_block):
    """Whatever 8 bits a digest holds (arrays that nothing has written yet), every list has its length
    and nothing is written beside the lists; exponents count as the nearest in [-50, 50]."""
    b = Batch([(40, 3000), (7, 90)], 8, 2, 128, 16, False, seed=q_block)
    g = torch.Generator(device="cuda").manual_seed(7)
    q, wide = b.rows(b.N, 8) * 2.0 ** 60, 3
    dims = ((b.N + 2 * (q_block - 1)) // q_block, 2)
    for keep in (1, 20, 100):
        b.digest.bounds.random_(-128, 128, generator=g)
        b.digest.exp.random_(-128, 128, generator=g)
        b.digest.exp[::3] = -128
        b.digest.exp[1::3] = 127
        most = 1 + keep + 1 + (q_block + 14) // 16 + 1
        held = torch.full((dims[0] + 2 * wide, 2, most), 77, dtype=torch.int32, device="cuda")
        index = held.clone()
        out = dsa.PageSelection(torch.empty(dims[0] + 1, dtype=torch.int32, device="cuda"),
                                torch.empty(dims[0], dtype=torch.int32, device="cuda"), held[wide:-wide], index[wide:-wide])
        sel = dsa.page_select(q, b.digest, b.q_start, b.kv_len, b.table, keep=keep, q_block=q_block, out=out)
        torch.cuda.synchronize()
        for x in (held, index):
            assert (x[:wide] == 77).all() and (x[-wide:] == 77).all()
        raw = b.digest.exp.clone()
        b.digest.exp.clamp_(-50, 50)
        check_select(b, q, keep, 1, 1, q_block, sel)
        b.digest.exp.copy_(raw)


def test_select_of_short_sequences_and_loose_rows():
    """Chunks longer than their sequence (rows at negative positions), rows of no chunk, a sequence
    without keys; a table much wider than the sequences."""
    for q_block in (1, 16):
        b = Batch([(40, 25), (3, 0), (10, 400)], 8, 2, 128, 16, False, max_pages=9000).fill().digest_all()
        q = b.rows(b.N + 4, 8)
        b.q_start = ints(np.cumsum([2, 40, 3, 10]))
        sel = dsa.page_select(q, b.digest, b.q_start, b.kv_len, b.table, keep=4, q_block=q_block, want_index=True)
        check_select(b, q, 4, 1, 1, q_block, sel, rows0=2)


# Blocks of many rows whose CTAs take five tiles of 128 pages or more each, however an item is cut over a
# cluster (of 8 CTAs at most at these widths): both buffers of digests and of scores come round several times.
TILES = [
    # seqs (pages of 16), H_q, D, q_block, least tiles
    *(([(n, 16 * pages)], 4, D, n, 5) for D in (128, 64) for n, pages in
      ((16, 4800), (16, 5500), (24, 4800), (32, 5500), (64, 4800), (64, 6300))),   # 64, 96, 128, 256 rows, one set
    *(([(n, 16 * 4800)], 4, D, n, 5) for D in (128, 64) for n in (65, 128, 150)),   # 260, 512 and 600 rows: sets of 256
    ([(130, 16 * 5200), (3, 16 * 4900)], 6, 128, 60, 5),       # 360 rows in two sets, then short blocks
    ([(64, 16 * 57700)], 4, 128, 64, 50),                      # keys so many that sets are of 128 rows
    ([(150, 16 * 57700)], 4, 128, 150, 50),
]


@pytest.mark.parametrize("seqs,H_q,D,q_block,least", TILES)
def test_select_of_many_tiles(seqs, H_q, D, q_block, least):
    b = Batch(seqs, H_q, 1, D, 16, False, n_pages=2000, seed=H_q + D + q_block)
    b.table_np[:] = b.rng.integers(0, b.n_pages, b.table_np.shape)
    b.table = ints(b.table_np)
    b.fill(2.0).digest_all()
    for n, t in seqs:
        first = (t - n) // 16 - 1                           # candidates: pages 1 .. first - 1
        assert all(-(-(-(-(first - 1) // C)) // 128) >= least for C in (1, 2, 4, 8))
    q = b.rows(b.N, H_q, 3.0)
    for keep in (1, 400):
        sel = dsa.page_select(q, b.digest, b.q_start, b.kv_len, b.table, keep=keep, q_block=q_block, want_index=True)
        check_select(b, q, keep, 1, 1, q_block, sel)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("q_block", [16, 32, 64])
def test_select_of_many_tiles_without_clusters(q_block, D):
    """80 blocks and more, so that each is one CTA's: five to seven tiles, odd and even counts."""
    b = Batch([(81 * q_block - 5, 81 * q_block - 5 + 16 * 700)], 4, 1, D, 16, False, seed=q_block).fill(2.0).digest_all()
    q = b.rows(b.N, 4, 3.0)
    sel = dsa.page_select(q, b.digest, b.q_start, b.kv_len, b.table, keep=50, q_block=q_block, want_index=True)
    check_select(b, q, 50, 1, 1, q_block, sel)


@pytest.mark.parametrize("q_block", [1, 3])
def test_select_of_the_largest_batch(q_block):
    """4,096 sequences, which are as many blocks as a call may have, without keys, with one, with a few pages;
    and the attention over their lists."""
    seqs = [(1, t) for t in np.random.default_rng(q_block).integers(0, 200, 4096)]
    seqs[:3], seqs[-1] = [(1, 0), (1, 1), (1, 16)], (1, 199)
    b = Batch(seqs, 2, 1, 64, 16, False, n_pages=3000, max_pages=13)
    b.table_np[:] = b.rng.integers(0, b.n_pages, b.table_np.shape)
    b.table = ints(b.table_np)
    b.fill(2.0).digest_all()
    q = b.rows(b.N, 2)
    sel = dsa.page_select(q, b.digest, b.q_start, b.kv_len, b.table, keep=2, q_block=q_block, want_index=True)
    assert sel.kv_len.shape == (4096,)
    check_select(b, q, 2, 1, 1, q_block, sel)
    out, lse = dsa.paged_attn(q, b.cache, sel.q_start, sel.kv_len, sel.page_table)
    check_lists(b, q, sel.q_start, sel.kv_len, sel.page_table, out, lse, blocks=[0, 1, 2, 3, *range(10, 4096, 97), 4095])


def test_select_of_the_most_rows():
    """256 tokens of 128 heads that share their keys: 32,768 rows in one block."""
    b = Batch([(256, 16 * 700), (1, 16 * 300)], 128, 1, 128, 16, False, seed=5).fill(2.0).digest_all()
    q = b.rows(b.N, 128, 3.0)
    sel = dsa.page_select(q, b.digest, b.q_start, b.kv_len, b.table, keep=40, q_block=256, want_index=True)
    check_select(b, q, 40, 1, 1, 256, sel)


def test_select_over_the_largest_tables():
    """The widest table: 4M keys in pages of 16, a slice of 16,384 pages for each CTA."""
    for q_block, G in ((1, 4), (8, 4)):
        b = Batch([(3, 16 * 262144 - 5)], G, 1, 64, 16, False, n_pages=300)
        b.table_np[:] = b.rng.integers(0, 300, b.table_np.shape)
        b.table = ints(b.table_np)
        b.fill(2.0).digest_all()
        q = b.rows(3, G)
        sel = dsa.page_select(q, b.digest, b.q_start, b.kv_len, b.table, keep=500, q_block=q_block, want_index=True)
        check_select(b, q, 500, 1, 1, q_block, sel)


# ------------------------------------------------------------------ attention over lists

def check_lists(b, q, start, lens, table, out, lse, blocks=None):
    torch.cuda.synchronize()
    o, z, qf = f64(out), lse.cpu().numpy().astype(np.float64), f64(q)
    start, lens, table = (x.cpu().numpy() for x in (start, lens, table))
    G, scale = b.H_q // b.H_kv, b.D ** -0.5
    kv = {}
    for j in range(len(lens)) if blocks is None else blocks:
        rows, t = slice(start[j], start[j + 1]), int(lens[j])
        n = rows.stop - rows.start
        for h in range(b.H_kv if n else 0):
            pg = table[j, h, :-(-t // b.page)]
            lost = np.repeat((pg < 0) | (pg >= b.n_pages), b.page)[:t]
            for p in set(pg[(pg >= 0) & (pg < b.n_pages)].tolist()) - set(kv):
                kv[p] = b.held(p), b.held(p, "v")
            zero = np.zeros((b.page, b.H_kv, b.D))
            k, v = (np.concatenate([kv[p][i][:, h:h + 1] if p in kv else zero[:, :1] for p in pg.tolist()])[:t]
                    if len(pg) else np.zeros((0, 1, b.D)) for i in range(2))
            O, L, spread, size = paged.attend(qf[rows, h * G:(h + 1) * G], k, v, t - n, 0, None, scale, lost)
            ds = 2 * b.D * 2.0 ** -24 * size
            got, zb = o[rows, h * G:(h + 1) * G], z[rows, h * G:(h + 1) * G]
            assert np.array_equal(np.isneginf(L), np.isneginf(zb)), (j, h)
            fin = np.isfinite(L)
            assert (np.abs(zb - L)[fin] <= (ds + 2.0 ** -19 + 2.0 ** -22 * np.abs(L))[fin]).all(), (j, h)
            tol = H * np.abs(O) + (H + 2 * ds[..., None] + 2.0 ** -18) * spread
            assert (np.abs(got - O) <= tol).all(), (j, h, float((np.abs(got - O) - tol).max()))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("seqs,H_q,H_kv,D,page,q_block,keep", [
    ([(1, 3000), (1, 70), (1, 1)], 8, 2, 128, 64, 1, 6), ([(9, 900), (1, 40), (30, 30)], 4, 4, 64, 16, 1, 5),
    ([(200, 3000), (33, 100)], 8, 2, 128, 64, 64, 7), ([(130, 1000), (1, 800)], 12, 2, 64, 16, 16, 9),
    ([(65, 2000)], 16, 1, 128, 128, 32, 3), ([(300, 2100)], 2, 2, 64, 256, 128, 2)])
def test_attention_over_lists(seqs, H_q, H_kv, D, page, q_block, keep, fp8):
    b = Batch(seqs, H_q, H_kv, D, page, fp8, seed=D).fill(1.5).digest_all()
    q = b.rows(b.N, H_q)
    sel = dsa.page_select(q, b.digest, b.q_start, b.kv_len, b.table, keep=keep, q_block=q_block)
    out, lse = dsa.paged_attn(q, b.cache, sel.q_start, sel.kv_len, sel.page_table)
    check_lists(b, q, sel.q_start, sel.kv_len, sel.page_table, out, lse)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kw", [dict(), dict(n_sink=20, n_stream=100)])
def test_equal_lists_are_one_table(fp8, kw):
    """The same pages for every head give, bit by bit, what one table gives."""
    b = Batch([(50, 700), (1, 1500), (0, 30), (5, 64)], 8, 4, 128, 32, fp8, seed=9).fill()
    q = b.rows(b.N, 8)
    one, l1 = dsa.paged_attn(q, b.cache, b.q_start, b.kv_len, b.table, **kw)
    each, l2 = dsa.paged_attn(q, b.cache, b.q_start, b.kv_len, b.table[:, None].repeat(1, 4, 1), **kw)
    assert torch.equal(one, each) and torch.equal(l1, l2)


def test_lists_with_bad_pages_and_values_that_are_none():
    """Entries outside the cache hold no keys; what pages hold behind a list's end reaches nobody;
    an infinity in a value row reaches the rows of the head that lists it."""
    for fp8 in (False, True):
        b = Batch([(40, 500)], 4, 2, 64, 16, fp8, seed=4).fill()
        q = b.rows(40, 4)
        table = np.stack([b.table_np[:, [3, 9, 1, 20, 7]], b.table_np[:, [2, 30, 0, 11, 5]]], 1)
        table[0, 0, 1], table[0, 1, 2] = 10 ** 6, -7
        lens = ints([75])
        last = int(table[0, 0, 4])                          # head 0 sees 11 of its rows
        for t in (b.cache.k, b.cache.v):
            if fp8:
                t[last, 11:, 0] = 0x7F
            else:
                t[last, 11:, 0] = float("nan")
        out, lse = dsa.paged_attn(q, b.cache, ints([0, 40]), lens, ints(table))
        check_lists(b, q, ints([0, 40]), lens, ints(table), out, lse)
        if not fp8:
            b.cache.v[int(table[0, 1, 0]), 3, 1, 17] = float("inf")
            again, _ = dsa.paged_attn(q, b.cache, ints([0, 40]), lens, ints(table))
            assert torch.isinf(again[:, 2:, 17]).all()
            again[:, 2:, 17] = out[:, 2:, 17]
            assert torch.equal(again, out)


# ------------------------------------------------------------------ copies

@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D,H_kv,page,n,digest", [(128, 8, 64, 5, True), (64, 1, 16, 200, True), (64, 3, 16, 7, False),
                                                  (128, 5, 1024, 3, True), (128, 2, 32, 1, False), (64, 7, 128, 33, True)])
def test_copy(D, H_kv, page, n, digest, fp8):
    b = Batch([(1, 1)], H_kv, H_kv, D, page, fp8, n_pages=2 * n + 5).fill()
    b.digest.bounds.random_(-127, 128)
    b.digest.exp.random_(-50, 51)
    every = [t for t in (b.cache.k, b.cache.v, b.cache.k_scale, b.cache.v_scale) if t is not None]
    every += [b.digest.bounds, b.digest.exp]
    old = [t.clone() for t in every]
    order = b.rng.permutation(b.n_pages)
    src, dst = order[:n].copy(), order[n:2 * n].copy()
    if n > 5:
        src[1] = src[0]                                     # one source, two copies
        src[2], dst[3] = -1, b.n_pages                      # no pages: skipped
        dst[4] = src[4]                                     # onto itself
    dsa.kv_pages_copy(b.cache, ints(src), ints(dst), digest=b.digest if digest else None)
    for i, (t, o) in enumerate(zip(every, old)):
        want = o.clone()
        for x, y in zip(src, dst):
            if 0 <= x < b.n_pages and 0 <= y < b.n_pages and (digest or i < len(every) - 2):
                want[y] = o[x]
        assert torch.equal(t.view(torch.uint8), want.view(torch.uint8)), i


def test_copy_past_32_bits():
    """Pages whose offsets pass 2^32 bytes."""
    n = 2 ** 32 // (64 * 2 * 128 * 2) + 3
    cache = dsa.PagedKVCache.empty(n, 64, 2, 128)
    cache.k[1].normal_()
    cache.v[1].normal_()
    dsa.kv_pages_copy(cache, ints([1]), ints([n - 1]))
    assert torch.equal(cache.k[1], cache.k[n - 1]) and torch.equal(cache.v[1], cache.v[n - 1])


# ------------------------------------------------------------------ together

def step(b, q, k, v, f, w, keep=4, q_block=1, out=None):
    """A serving step: rotate and write, digest, select, attend."""
    qr = dsa.kv_cache_write_rope(b.cache, q, k, v, b.q_start, b.kv_len, b.table, f, q_weight=w, k_weight=w)
    dsa.page_digest_update(b.cache, b.digest, q.shape[0], b.q_start, b.kv_len, b.table)
    sel = dsa.page_select(qr, b.digest, b.q_start, b.kv_len, b.table, keep=keep, q_block=q_block)
    o, z = dsa.paged_attn(qr, b.cache, sel.q_start, sel.kv_len, sel.page_table)
    return qr, sel, o, z


@pytest.mark.parametrize("fp8", [False, True])
def test_a_prompt_a_fork_and_decoding(fp8):
    """A prompt in two chunks, a fork of its sequence (shared pages, the last one copied) and tokens
    that differ from there on: every step against the restatements, and the same with nothing
    dropped as attention over the whole cache."""
    page, T = 16, 300
    b = Batch([(150, 150)], 8, 2, 128, page, fp8, seed=1, n_pages=60, max_pages=24)
    order = b.rng.permutation(60)
    b.table_np = order[None, :24].astype(np.int32)
    b.table = ints(b.table_np)
    f, w = torch.from_numpy(freqs(128)).cuda(), torch.ones(128, device="cuda")
    for n, t in ((150, 150), (149, 299)):
        b.seqs, b.q_start, b.kv_len = [(n, t)], ints([0, n]), ints([t])
        qr, sel, o, z = step(b, b.rows(n, 8), b.rows(n, 2), b.rows(n, 2), f, w, q_block=16)
        check_select(b, qr, 4, 1, 1, 16, sel)
        check_lists(b, qr, sel.q_start, sel.kv_len, sel.page_table, o, z)
    fork = b.table_np[0].copy()
    fork[299 // page] = order[30]
    dsa.kv_pages_copy(b.cache, ints([b.table_np[0, 299 // page]]), ints([order[30]]), digest=b.digest)
    fork[299 // page + 1:] = order[31:31 + 24 - 299 // page - 1]
    b.table_np = np.stack([b.table_np[0], fork]).astype(np.int32)
    b.table = ints(b.table_np)
    for t in range(300, 310):
        b.seqs, b.q_start, b.kv_len = [(1, t), (1, t)], ints([0, 1, 2]), ints([t, t])
        qr, sel, o, z = step(b, b.rows(2, 8), b.rows(2, 2), b.rows(2, 2), f, w)
        check_select(b, qr, 4, 1, 1, 1, sel)
        check_lists(b, qr, sel.q_start, sel.kv_len, sel.page_table, o, z)
        every = dsa.page_select(qr, b.digest, b.q_start, b.kv_len, b.table, keep=100)
        o1, z1 = dsa.paged_attn(qr, b.cache, every.q_start, every.kv_len, every.page_table)
        o2, z2 = dsa.paged_attn(qr, b.cache, b.q_start, b.kv_len, b.table)
        assert torch.equal(o1, o2) and torch.equal(z1, z2)


@pytest.mark.parametrize("q_block", [1, 16])
def test_a_captured_step(q_block):
    """A step captured in a graph serves later lengths and inputs, on a stream of its own, beside
    another graph."""
    n = 3 if q_block == 1 else 40
    graphs = []
    f, w = torch.from_numpy(freqs(128)).cuda(), torch.ones(128, device="cuda")
    for seed in (0, 1):
        b = Batch([(n, 900), (n, 700)], 8, 2, 128, 32, seed == 1, seed=seed, max_pages=40, n_pages=90).fill().digest_all()
        b.table_np = b.rng.permutation(90)[:80].reshape(2, 40).astype(np.int32)
        b.table = ints(b.table_np)
        x = [b.rows(2 * n, 8), b.rows(2 * n, 2), b.rows(2 * n, 2)]
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            step(b, *x, f, w, q_block=q_block)
            s.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                out = step(b, *x, f, w, q_block=q_block)
        graphs.append((b, x, s, g, out))
    for t in (901, 1000, 1203):
        for b, x, s, g, out in graphs:
            s.wait_stream(torch.cuda.current_stream())
            b.seqs = [(n, t), (n, t - 200)]
            with torch.cuda.stream(s):
                for y in x:
                    y.copy_(torch.randn_like(y.float()))
                b.kv_len.copy_(ints([t, t - 200]))
                g.replay()
        torch.cuda.synchronize()
        for b, x, s, g, (qr, sel, o, z) in graphs:
            check_select(b, qr, 4, 1, 1, q_block, sel)
            check_lists(b, qr, sel.q_start, sel.kv_len, sel.page_table, o, z)


def test_repeats_bit_by_bit_and_on_another_stream():
    b = Batch([(100, 3000), (7, 900)], 8, 2, 128, 32, False, seed=2).fill().digest_all()
    q = b.rows(b.N, 8)
    runs = []
    for s in (None, torch.cuda.Stream(), torch.cuda.Stream(), None):
        torch.cuda.synchronize()
        sel = dsa.page_select(q, b.digest, b.q_start, b.kv_len, b.table, keep=9, q_block=16, stream=s)
        o, z = dsa.paged_attn(q, b.cache, sel.q_start, sel.kv_len, sel.page_table, stream=s)
        torch.cuda.synchronize()
        runs.append((sel.page_table, o, z))
    for r in runs[1:]:
        assert all(torch.equal(x, y) for x, y in zip(r, runs[0]))


@pytest.mark.parametrize("q_block", [1, 32])
def test_calls_from_threads(q_block):
    """Host threads, each on a stream of its own, over tables of very different width: every call is
    taken and gets the lists that it gets alone.  (The C entry itself: what Python does between two calls
    keeps the threads apart.)"""
    import ctypes
    import threading
    lib, jobs, n = dsa.load(), [], 20 if q_block == 1 else 70
    for width in (24, 32768, 24, 32768):
        b = Batch([(n, 350), (n, 300)], 8, 2, 128, 16, False, seed=width, max_pages=width).fill().digest_all()
        q = b.rows(b.N, 8)
        want = dsa.page_select(q, b.digest, b.q_start, b.kv_len, b.table, keep=6, q_block=q_block)
        got, stream = [torch.zeros_like(t) for t in (want.q_start, want.kv_len, want.page_table)], torch.cuda.Stream()
        shape = dsa.binding.PagedShape(2, b.N, width, b.n_pages, 16, 8, 2, 128, dsa.binding.BF16)
        cfg = dsa.binding.PageSelectCfg(6, 1, 1, q_block)
        args = (q.data_ptr(), 8 * 128, b.digest.bounds.data_ptr(), b.digest.exp.data_ptr(), b.q_start.data_ptr(),
                b.kv_len.data_ptr(), b.table.data_ptr(), ctypes.byref(shape), ctypes.byref(cfg),
                *(t.data_ptr() for t in got), None, stream.cuda_stream)
        jobs.append((b, q, want, got, stream, args, shape, cfg))
    torch.cuda.synchronize()
    refused, go = [0] * len(jobs), threading.Barrier(len(jobs))

    def work(i):
        stream, args = jobs[i][4], jobs[i][5]
        go.wait(timeout=60)
        for k in range(3000):
            refused[i] += lib.page_select(*args) != 0
            if k % 250 == 249:                              # (not too far ahead of the GPU)
                stream.synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join(timeout=300)
    torch.cuda.synchronize()
    assert not any(t.is_alive() for t in threads) and refused == [0] * len(jobs), refused
    for _, _, want, got, *_ in jobs:
        assert all(torch.equal(x, y) for x, y in zip(got, (want.q_start, want.kv_len, want.page_table)))


def test_waits_that_run_out():
    """With a limit of a nanosecond the selection of many rows gives up: the error bit is set, every entry is
    a page of its sequence or -1, and the next call is whole."""
    b = Batch([(100, 8000), (70, 5000)], 8, 2, 128, 16, False, seed=6).fill().digest_all()
    q = b.rows(b.N, 8)
    call = lambda: dsa.page_select(q, b.digest, b.q_start, b.kv_len, b.table, keep=30, q_block=64, want_index=True)
    torch.cuda.synchronize()
    assert dsa.device_error() == 0
    dsa.set_wait_limit(1)
    try:
        sel = call()
        torch.cuda.synchronize()
    finally:
        dsa.set_wait_limit(0)
    assert dsa.device_error() == 16
    owner = torch.tensor([0, 0, 1, 1], device="cuda")
    for j, s in enumerate(owner.tolist()):
        i = sel.index[j]
        assert ((i >= -1) & (i < -(-b.seqs[s][1] // 16))).all()
        assert (sel.page_table[j] == torch.where(i < 0, -1, b.table[s][i.clamp(min=0).long()])).all()
    check_select(b, q, 30, 1, 1, 64, call())


@pytest.mark.parametrize("B", [1, 3])
@pytest.mark.parametrize("kw", [dict(), dict(q_block=1), dict(q_block=64)])
def test_a_step_without_tokens(B, kw):
    """The documented step of a batch that brings nothing, whatever the blocks."""
    b = Batch([(1, 100)] * B, 4, 2, 64, 16, False).fill().digest_all()
    q, start = b.rows(1, 4)[:0], ints([0] * (B + 1))
    old = [t.clone() for t in (b.cache.k, b.cache.v, b.digest.bounds, b.digest.exp)]
    qr = dsa.kv_cache_write_rope(b.cache, q, q[:, :2], q[:, :2], start, b.kv_len, b.table, None)
    dsa.page_digest_update(b.cache, b.digest, 0, start, b.kv_len, b.table)
    sel = dsa.page_select(qr, b.digest, start, b.kv_len, b.table, keep=3, want_index=True, **kw)
    out, lse = dsa.paged_attn(qr, b.cache, sel.q_start, sel.kv_len, sel.page_table)
    assert qr.shape == out.shape == (0, 4, 64) and lse.shape == (0, 4)
    assert not sel.q_start.any() and not sel.kv_len.any() and (sel.page_table == -1).all() and (sel.index == -1).all()
    assert all(torch.equal(x, y) for x, y in zip(old, (b.cache.k, b.cache.v, b.digest.bounds, b.digest.exp)))


@pytest.mark.parametrize("q_block", [1, 16])
def test_no_tokens_at_the_c_entry(q_block):
    """The C entry itself writes the lists of a call without tokens, and nothing beside them."""
    import ctypes
    lib, B = dsa.load(), 2
    b = Batch([(1, 100)] * B, 4, 2, 64, 16, False).fill().digest_all()
    shape = dsa.binding.PagedShape(B, 0, b.table.shape[1], b.n_pages, 16, 4, 2, 64, dsa.binding.BF16)
    cfg, n, m = dsa.binding.PageSelectCfg(3, 1, 1, q_block), ctypes.c_int(), ctypes.c_int()
    assert lib.page_select_sizes(ctypes.byref(shape), ctypes.byref(cfg), ctypes.byref(n), ctypes.byref(m)) == 0
    sizes = [n.value + 1, n.value, n.value * 2 * m.value, n.value * 2 * m.value]
    call = lambda ptrs: lib.page_select(None, 4 * 64, b.digest.bounds.data_ptr(), b.digest.exp.data_ptr(), ints([0, 0, 0]).data_ptr(),
                                        b.kv_len.data_ptr(), b.table.data_ptr(), ctypes.byref(shape), ctypes.byref(cfg), *ptrs, None)
    for index in (True, False):
        outs = [torch.full((size + 2,), 77, dtype=torch.int32, device="cuda") for size in sizes]
        torch.cuda.synchronize()
        assert call([t[1:].data_ptr() for t in outs[:3]] + [outs[3][1:].data_ptr() if index else None]) == 0
        torch.cuda.synchronize()
        for t, want in zip(outs, (0, 0, -1, -1 if index else 77)):
            assert (t[1:-1] == want).all() and t[0] == 77 and t[-1] == 77
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):                              # and as part of a graph
        q, out = b.rows(1, 4)[:0], dsa.page_select(b.rows(1, 4)[:0], b.digest, ints([0, 0, 0]), b.kv_len, b.table, keep=3, q_block=q_block)
        start, g = ints([0, 0, 0]), torch.cuda.CUDAGraph()
        s.synchronize()
        with torch.cuda.graph(g, stream=s):
            dsa.page_select(q, b.digest, start, b.kv_len, b.table, keep=3, q_block=q_block, out=out)
        out.page_table.fill_(5)
        out.q_start.fill_(5)
        g.replay()
    torch.cuda.synchronize()
    assert (out.page_table == -1).all() and not out.q_start.any()


def test_no_tokens():
    """A call without rows: blocks without rows, which attend nothing."""
    b = Batch([(1, 100), (1, 40)], 4, 2, 64, 16, False).fill().digest_all()
    q, zero = b.rows(1, 4)[:0], ints([0, 0, 0])
    sel = dsa.page_select(q, b.digest, zero, b.kv_len, b.table, keep=3, q_block=16, want_index=True)
    assert not sel.q_start.any() and not sel.kv_len.any() and (sel.page_table == -1).all() and (sel.index == -1).all()
    out, lse = dsa.paged_attn(q, b.cache, sel.q_start, sel.kv_len, sel.page_table)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    dsa.page_digest_update(b.cache, b.digest, 0, zero, b.kv_len, b.table)
    dsa.kv_cache_write_rope(b.cache, q, q[:, :2], q[:, :2], zero, b.kv_len, b.table, None)
    dsa.kv_pages_copy(b.cache, zero[:0], zero[:0], digest=b.digest)
