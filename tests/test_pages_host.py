"""The entry points around the paged cache's sparse path validate their arguments on the host (no
GPU needed: every call here fails before any launch, or has nothing to launch), and the float64
restatements that the GPU tests compare with are what they say."""
import ctypes

import numpy as np
import pytest
import torch

import dynamic_sparse_attention_gb300 as dsa
from dynamic_sparse_attention_gb300 import _build, binding
from oracle import pages


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return binding.load()


def _shape(**kw):
    d = dict(B=2, n_tok=8, max_pages=16, n_pages=64, page_size=64, H_q=8, H_kv=2, D=128, dtype=0)
    d.update(kw)
    return binding.PagedShape(**d)


_BUF = (ctypes.c_char * 64)()
OK = ctypes.addressof(_BUF) + (-ctypes.addressof(_BUF) % 16)
FAR = [OK + (i << 32) for i in range(20)]


def _rope(lib, s, q=OK, k=OK, v=OK, qs=1024, ks=256, vs=256, os=1024, start=OK, lens=OK, table=OK, out=OK, kp=OK, vp=OK,
          ksc=OK, vsc=OK, **cfg):
    c = dict(q_weight=OK, k_weight=OK, weight_f32=0, eps=1e-6, inv_freq=OK, rot=128, interleaved=0, rope_scale=1.0)
    c.update(cfg)
    return lib.kv_cache_write_rope(q, qs, k, ks, v, vs, start, lens, table, ctypes.byref(s),
                                   ctypes.byref(binding.RopeCfg(**c)), out, os, kp, vp, ksc, vsc, None)


def _digest(lib, s, k=OK, ks=OK, start=OK, lens=OK, table=OK, bounds=OK, exp=OK):
    return lib.page_digest_update(k, ks, start, lens, table, ctypes.byref(s), bounds, exp, None)


def _select(lib, s, q=OK, stride=1024, bounds=OK, exp=OK, start=OK, lens=OK, table=OK, o=(OK, OK, OK, OK), **cfg):
    c = dict(keep=4, n_sink=1, n_local=1, q_block=4)
    c.update(cfg)
    return lib.page_select(q, stride, bounds, exp, start, lens, table, ctypes.byref(s),
                           ctypes.byref(binding.PageSelectCfg(**c)), *o, None)


def _copy(lib, s, n=3, src=OK, dst=OK, k=OK, v=OK, ks=OK, vs=OK, bounds=OK, exp=OK):
    return lib.kv_pages_copy(src, dst, n, ctypes.byref(s), k, v, ks, vs, bounds, exp, None)


def _lists(lib, s, table=OK, q=OK, out=OK, ws=OK, ws_bytes=1 << 40, scale=0.1, lse=OK):
    return lib.paged_attn_lists(q, 1024, OK, OK, OK, OK, OK, OK, table, ctypes.byref(s), 0, -1, scale, out, lse, ws,
                                ws_bytes, None)


CALLS = (_rope, _digest, _select, _copy, _lists)


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), -1), (dict(B=4097), -2), (dict(n_tok=-1), -1), (dict(n_pages=0), -1), (dict(max_pages=0), -1),
    (dict(page_size=8), -2), (dict(page_size=24), -2), (dict(max_pages=1 << 25), -1),
    (dict(H_q=9), -1), (dict(H_q=256), -2), (dict(D=96), -2), (dict(dtype=1), -2)])
def test_bad_shapes_are_rejected(lib, kw, status):
    for call in CALLS:
        assert call(lib, _shape(**kw)) == status, call
        assert lib.dsa_last_error()


def test_rope_arguments(lib):
    s = _shape()
    for kw in (dict(rot=130), dict(rot=-16), dict(rot=8), dict(rot=144), dict(eps=-1e-6), dict(eps=float("nan")),
               dict(eps=float("inf")), dict(rope_scale=float("nan")), dict(qs=1016), dict(ks=252), dict(vs=260),
               dict(os=1023)):
        assert _rope(lib, s, **kw) == -1, kw
    for kw in (dict(q=None), dict(k=OK + 2), dict(v=None), dict(out=OK + 8), dict(inv_freq=None), dict(inv_freq=OK + 4),
               dict(q_weight=OK + 1), dict(k_weight=OK + 2, weight_f32=1), dict(start=None), dict(lens=OK + 2),
               dict(table=None), dict(kp=OK + 8)):
        assert _rope(lib, s, **kw) == -4, kw
    assert _rope(lib, _shape(dtype=2), ksc=None) == -4
    assert lib.kv_cache_write_rope(OK, 1024, OK, 256, OK, 256, OK, OK, OK, ctypes.byref(s), None, OK, 1024, OK, OK, None,
                                   None, None) == -1


def test_rope_overlaps(lib):
    """The queries may be rotated in place; any other sharing of memory is refused, rows interleaved in one
    projection are not sharing."""
    s = _shape()                                        # a fused row: 8 + 2 + 2 heads of 128
    last = lambda: lib.dsa_last_error().decode()
    f = dict(q=FAR[0], k=FAR[0] + 2048, v=FAR[0] + 2560, qs=1536, ks=1536, vs=1536, os=1024, out=FAR[1], kp=FAR[2],
             vp=FAR[3], start=FAR[4], lens=FAR[5], table=FAR[6], q_weight=FAR[7], k_weight=FAR[8], inv_freq=FAR[9])
    for kw, two in ((dict(out=FAR[0], os=1024), "q_out and q"), (dict(out=FAR[0] + 512, os=1536), "q_out and q"),
                    (dict(out=FAR[0] + 1024, os=1536), "q_out and q"), (dict(out=FAR[0] - 2048, os=1536), "q_out and q"),
                    (dict(out=FAR[4] - 64), "q_out and q_start"), (dict(kp=FAR[0] + 64), "k_pages and q"),
                    (dict(vp=FAR[1] - 16), "v_pages and q_out"), (dict(kp=FAR[9]), "k_pages and inv_freq"),
                    (dict(out=FAR[7]), "q_out and q_weight"), (dict(vp=FAR[2] + 64), "v_pages and k_pages"),
                    # in place, and then something else that is refused
                    (dict(out=FAR[0], os=1536, kp=FAR[3]), "v_pages and k_pages"),
                    (dict(out=FAR[0], os=1536, k=FAR[0], ks=1536), "q_out and k_new")):
        assert _rope(lib, s, **{**f, **kw}) == -1 and last().endswith(two + " overlap"), (kw, last())


def test_digest_and_copy_arguments(lib):
    s, fp8 = _shape(), _shape(dtype=2)
    for kw in (dict(k=None), dict(k=OK + 8), dict(start=None), dict(lens=OK + 1), dict(table=None), dict(bounds=None),
               dict(bounds=OK + 8), dict(exp=None)):
        assert _digest(lib, s, **kw) == -4, kw
    assert _digest(lib, fp8, ks=None) == -4
    last = lambda: lib.dsa_last_error().decode()
    a = dict(k=FAR[0], start=FAR[1], lens=FAR[2], table=FAR[3], bounds=FAR[4], exp=FAR[5], ks=FAR[6])
    for kw, two in ((dict(bounds=FAR[0] + 64), "bounds and k_pages"), (dict(exp=FAR[4] + 5), "exp and bounds"),
                    (dict(exp=FAR[2] + 4), "exp and kv_len")):
        assert _digest(lib, s, **{**a, **kw}) == -1 and last().endswith(two + " overlap"), (kw, last())
    for kw in (dict(k=None), dict(v=OK + 8), dict(src=None), dict(dst=OK + 2), dict(bounds=OK + 4)):
        assert _copy(lib, s, **kw) == -4, kw
    assert _copy(lib, fp8, vs=None) == -4
    assert _copy(lib, s, n=-1) == -1 and _copy(lib, s, n=(1 << 24) + 1) == -1
    assert _copy(lib, s, exp=None) == -1 and _copy(lib, s, bounds=None) == -1
    c = dict(src=FAR[0], dst=FAR[1], k=FAR[2], v=FAR[3], ks=FAR[4], vs=FAR[5], bounds=FAR[6], exp=FAR[7])
    for kw, two in ((dict(v=FAR[2] + 16), "v_pages and k_pages"), (dict(src=FAR[3] + 16), "v_pages and src"),
                    (dict(exp=FAR[6] + 1), "exp and bounds"), (dict(ks=FAR[2] + 1), "k_scale and k_pages")):
        assert _copy(lib, fp8, **{**c, **kw}) == -1 and last().endswith(two + " overlap"), (kw, last())


def test_select_arguments_and_sizes(lib):
    s = _shape()
    for kw in (dict(keep=-1), dict(n_sink=-1), dict(n_local=-5), dict(keep=(1 << 24) + 1), dict(keep=1 << 24)):
        assert _select(lib, s, **kw) == -1, kw
    for kw in (dict(q_block=0), dict(q_block=257)):
        assert _select(lib, s, **kw) == -2, kw
    assert _select(lib, _shape(max_pages=262145)) == -2 and _select(lib, _shape(n_tok=4098), q_block=1) == -2
    for kw in (dict(q=None), dict(q=OK + 8), dict(bounds=OK + 8), dict(exp=None), dict(start=None), dict(lens=None),
               dict(table=OK + 2), dict(o=(None, OK, OK, OK)), dict(o=(OK, OK + 1, OK, OK)), dict(o=(OK, OK, None, OK)),
               dict(o=(OK, OK, OK, OK + 2))):
        assert _select(lib, s, **kw) == -4, kw
    assert _select(lib, s, stride=1016) == -1
    last = lambda: lib.dsa_last_error().decode()
    a = dict(q=FAR[0], bounds=FAR[1], exp=FAR[2], start=FAR[3], lens=FAR[4], table=FAR[5])
    for o, two in (((FAR[6], FAR[7], FAR[0], FAR[9]), "sel_table and q"), ((FAR[6], FAR[6] + 4, FAR[8], None), "sel_kv_len and sel_q_start"),
                   ((FAR[6], FAR[7], FAR[8], FAR[8] + 8), "sel_index and sel_table"), ((FAR[3] + 8, FAR[7], FAR[8], None), "sel_q_start and q_start")):
        assert _select(lib, s, o=o, **a) == -1 and last().endswith(two + " overlap"), (two, last())
    n, m = ctypes.c_int(), ctypes.c_int()

    def sizes(shape, **kw):
        c = dict(keep=4, n_sink=1, n_local=2, q_block=1)
        c.update(kw)
        assert lib.page_select_sizes(ctypes.byref(shape), ctypes.byref(binding.PageSelectCfg(**c)), ctypes.byref(n),
                                     ctypes.byref(m)) == 0
        return n.value, m.value
    assert sizes(_shape(n_tok=8, B=8)) == (8, 8)
    assert sizes(_shape(n_tok=8, B=3), q_block=64) == (3, 9)
    assert sizes(_shape(n_tok=1000, B=1, page_size=16), q_block=64) == (16, 12)
    # never fewer blocks than there are, never a list longer than it can be
    rng = np.random.default_rng(0)
    for _ in range(300):
        B, qb, ps = int(rng.integers(1, 9)), int(rng.integers(1, 100)), int(2 ** rng.integers(4, 8))
        ns = rng.integers(0, 150, B)
        if not ns.sum():
            continue
        got, width = sizes(_shape(n_tok=int(ns.sum()), B=B, page_size=ps), q_block=qb)
        assert got >= sum(-(-x // qb) for x in ns)
        p0 = int(rng.integers(0, 1000))
        s0, first, own0, own1 = pages.span(p0, qb, ps, 1, 2)
        assert s0 + 4 + own1 + 1 - first <= width


@pytest.mark.parametrize("B,q_block", [(1, 1), (3, 1), (1, 64), (3, 64), (4096, 1)])
def test_a_call_without_tokens_has_a_block(lib, B, q_block):
    """So that the attention over its lists, a sequence a block, is a call that is taken."""
    n, m = ctypes.c_int(), ctypes.c_int()
    s = _shape(n_tok=0, B=B)
    cfg = binding.PageSelectCfg(keep=4, n_sink=1, n_local=2, q_block=q_block)
    assert lib.page_select_sizes(ctypes.byref(s), ctypes.byref(cfg), ctypes.byref(n), ctypes.byref(m)) == 0
    assert n.value >= 1 and m.value >= 8
    assert _lists(lib, _shape(n_tok=0, B=n.value, max_pages=m.value), q=None) == 0


def test_lists_arguments(lib):
    s = _shape()
    assert _lists(lib, s, table=None) == -4 and _lists(lib, s, q=None) == -4 and _lists(lib, s, scale=0.0) == -1
    assert _lists(lib, s, ws_bytes=100) == -3
    # the whole table of every head counts: 2 x 2 x 16 entries
    call = lambda table: lib.paged_attn_lists(FAR[0], 1024, FAR[1], FAR[2], None, None, FAR[3], FAR[4], table, ctypes.byref(s),
                                              0, -1, 0.1, FAR[5], FAR[6], FAR[7], 1 << 31, None)
    assert call(FAR[5] - 2 * 2 * 16 * 4 + 4) == -1 and b"out and page_table overlap" in lib.dsa_last_error()


def test_select_without_tokens_checks_its_outputs(lib):
    s = _shape(n_tok=0)
    a = dict(q=None, bounds=FAR[1], exp=FAR[2], start=FAR[3], lens=FAR[4], table=FAR[5])
    for o in ((OK + 1, None, None, None), (None, None, OK + 2, None), (None, None, None, OK + 3)):
        assert _select(lib, s, o=o, **a) == -4, o
    for o in ((None, None, FAR[5] + 4, None), (None, FAR[3], None, None), (None, None, FAR[6], FAR[6] + 4)):
        assert _select(lib, s, o=o, **a) == -1, o


def test_nothing_to_do(lib):
    s = _shape(n_tok=0)
    assert _rope(lib, s, q=None, k=None, v=None, out=None) == 0 and _digest(lib, s) == 0 and _lists(lib, s, q=None) == 0
    assert _select(lib, s, q=None, o=(None,) * 4) == 0 and _copy(lib, s, n=0, src=None, dst=None) == 0
    assert _rope(lib, s, rot=3) == -1 and _select(lib, s, keep=-1) == -1   # still checked


def test_binding_rejects(lib, monkeypatch):
    c = dsa.PagedKVCache.empty(4, 16, 2, 64, device="cpu")
    d = dsa.PageDigest.empty(c)
    one, table = torch.ones(1, dtype=torch.int32), torch.zeros(1, 1, dtype=torch.int32)
    start, q = torch.tensor([0, 1], dtype=torch.int32), torch.zeros(1, 4, 64, dtype=torch.bfloat16)
    calls = (lambda **kw: dsa.kv_cache_write_rope(c, q, q[:, :2], q[:, :2], start, one, table, None, **kw),
             lambda **kw: dsa.page_digest_update(c, d, 1, start, one, table, **kw),
             lambda **kw: dsa.page_select(q, d, start, one, table, keep=3, **kw),
             lambda **kw: dsa.kv_pages_copy(c, one, one, **kw))
    for call in calls:
        with pytest.raises(ValueError, match="CUDA"):
            call()
    # as if on a device: what the checks behind it say
    monkeypatch.setattr(binding, "_cache_args", lambda cache: (OK, OK, None, None, cache.k.shape, 0, -1))
    monkeypatch.setattr(binding, "_digest_args", lambda digest: (OK, OK, *digest.bounds.shape[:2], digest.bounds.shape[3], -1))
    monkeypatch.setattr(binding, "_current_stream", lambda dev: 0)
    write = lambda q=q, k=q[:, :2], f=None, **kw: dsa.kv_cache_write_rope(c, q, k, q[:, :2], start, one, table, f, **kw)
    for kw, e in ((dict(k=q), ValueError), (dict(q=q.float()), ValueError), (dict(q=torch.zeros(2, 4, 64).bfloat16()), ValueError),
                  (dict(f=torch.zeros(16)), TypeError), (dict(f=torch.zeros(2, 8).double()), TypeError),
                  (dict(q_weight=torch.ones(32)), ValueError), (dict(q_weight=torch.ones(64).double()), ValueError),
                  (dict(q_weight=torch.ones(64), k_weight=torch.ones(64).bfloat16()), ValueError),
                  (dict(q_out=torch.zeros(1, 2, 64).bfloat16()), ValueError)):
        with pytest.raises(e):
            write(**kw)
    for kw in (dict(keep=-1), dict(keep=1 << 33), dict(keep=1, n_sink=-2 ** 32), dict(keep=1, n_local=-1),
               dict(keep=1, q_block=2 ** 32 + 1)):
        with pytest.raises(ValueError):
            dsa.page_select(q, d, start, one, table, **kw)
    with pytest.raises(dsa.DsaError):
        dsa.page_select(q, d, start, one, table, keep=1, q_block=0)
    other = dsa.PageDigest(d.bounds[:3], d.exp[:3], 16)
    with pytest.raises(ValueError, match="another cache"):
        dsa.page_digest_update(c, other, 1, start, one, table)
    with pytest.raises(ValueError, match="another cache"):
        dsa.kv_pages_copy(c, one, one, digest=dsa.PageDigest(d.bounds, d.exp, 32))
    with pytest.raises(ValueError, match="same length"):
        dsa.kv_pages_copy(c, one, start)
    with pytest.raises(ValueError, match="each KV head"):
        dsa.paged_attn(q, c, start, one, torch.zeros(1, 3, 1, dtype=torch.int32))
    sel = dsa.PageSelection(start, one, torch.zeros(1, 2, 9, dtype=torch.int32))
    with pytest.raises(ValueError, match="out.page_table"):
        dsa.page_select(q, d, start, one, table, keep=1, out=sel)


def test_numbers_past_32_bits_are_not_cut(lib, monkeypatch):
    """n_tok, and the sizes of tensors, reach the library whole or not at all."""
    c = dsa.PagedKVCache.empty(4, 16, 2, 64, device="cpu")
    d = dsa.PageDigest.empty(c)
    one, table, start = torch.ones(1, dtype=torch.int32), torch.zeros(1, 1, dtype=torch.int32), torch.tensor([0, 1], dtype=torch.int32)
    monkeypatch.setattr(binding, "_cache_args", lambda cache: (OK, OK, None, None, cache.k.shape, 0, -1))
    monkeypatch.setattr(binding, "_digest_args", lambda digest: (OK, OK, *digest.bounds.shape[:2], digest.bounds.shape[3], -1))
    monkeypatch.setattr(binding, "_current_stream", lambda dev: 0)
    for n in (2 ** 32, 2 ** 32 + 5, 2 ** 31, -2 ** 32, -1, 2 ** 30 + 1, 2 ** 64):
        with pytest.raises((ValueError, dsa.DsaError)):
            dsa.page_digest_update(c, d, n, start, one, table)
    dsa.page_digest_update(c, d, 0, start, one, table)   # nothing to do, and taken
    for i in range(9):
        sizes = [1, 0, 1, 4, 16, 2, 2, 64, 0]
        sizes[i] += 2 ** 32
        with pytest.raises(ValueError):
            binding._paged_shape(*sizes)
        with pytest.raises(ValueError):
            binding._select_sizes(3, 1, 1, 1, *sizes)


def test_stream_of_another_device(lib, monkeypatch):
    class Default:
        cuda_stream, device_index = 0, 1
    c = dsa.PagedKVCache.empty(4, 16, 2, 64, device="cpu")
    d = dsa.PageDigest.empty(c)
    monkeypatch.setattr(binding, "_cache_args", lambda cache: (OK, OK, None, None, cache.k.shape, 0, 0))
    monkeypatch.setattr(binding, "_digest_args", lambda digest: (OK, OK, *digest.bounds.shape[:2], digest.bounds.shape[3], 0))
    monkeypatch.setattr(binding, "_current_stream", lambda dev: 0)
    one, table = torch.ones(1, dtype=torch.int32), torch.zeros(1, 1, dtype=torch.int32)
    start, q = torch.tensor([0, 1], dtype=torch.int32), torch.zeros(1, 4, 64, dtype=torch.bfloat16)
    for call in (lambda: dsa.kv_cache_write_rope(c, q, q[:, :2], q[:, :2], start, one, table, None, stream=Default()),
                 lambda: dsa.page_digest_update(c, d, 1, start, one, table, stream=Default()),
                 lambda: dsa.page_select(q, d, start, one, table, keep=1, stream=Default()),
                 lambda: dsa.kv_pages_copy(c, one, one, stream=Default())):
        with pytest.raises(ValueError, match="stream is on device 1"):
            call()


# ------------------------------------------------------------ the restatements

def test_rotation_against_complex_numbers():
    rng = np.random.default_rng(0)
    x, pos = rng.standard_normal((5, 3, 16)), np.array([0, 1, 7, 1000, 10 ** 6])
    f = 100.0 ** (-np.arange(0, 12, 2) / 12)
    y, _ = pages.rotate(x, pos, None, 0, f, interleaved=True, scale=0.5)
    z = (x[..., 0:12:2] + 1j * x[..., 1:12:2]) * 0.5 * np.exp(1j * pos[:, None] * f)[:, None]
    assert np.allclose(y[..., 0:12:2], z.real) and np.allclose(y[..., 1:12:2], z.imag) and np.array_equal(y[..., 12:], x[..., 12:])
    order = [*range(0, 12, 2), *range(1, 12, 2), 12, 13, 14, 15]
    half, _ = pages.rotate(x[..., order], pos, None, 0, f, scale=0.5)
    assert np.allclose(half, y[..., order])
    n, size = pages.rotate(x, pos, np.full(16, 2.0), 0.0, None)
    assert np.allclose((n ** 2).mean(-1), 4.0) and np.array_equal(size, np.abs(n))
    # a rotation keeps scores of the same distance
    a, b = rng.standard_normal((2, 1, 1, 16))
    dot = lambda p, q: (pages.rotate(a, [p], None, 0, f)[0] * pages.rotate(b, [q], None, 0, f)[0]).sum()
    assert np.isclose(dot(5, 3), dot(105, 103))


def test_digests_bound_the_scores():
    """lo 2^e <= k <= hi 2^e, e the least that fits, and the bound is one on whole-number queries."""
    rng = np.random.default_rng(1)
    for scale in (2.0 ** -30, 1.0, 300.0):
        k = rng.standard_normal((40, 32)) * scale
        lo, hi, e = pages.digest(k)
        assert (np.ldexp(lo.astype(float), e) <= k.min(0)).all() and (np.ldexp(hi.astype(float), e) >= k.max(0)).all()
        assert np.abs(k).max() <= 127 * 2.0 ** e and np.abs(k).max() > 127 * 2.0 ** (e - 1)
        q = rng.standard_normal((6, 32)) * 5
        w, eq = pages.whole(q)
        assert np.abs(w).max() <= 127 and np.abs(np.ldexp(w, eq[:, None]) - q).max() <= 0.5 * 2.0 ** eq.max()
        s = pages.bound(q, lo[None], hi[None], np.array([e]))
        assert s[0] >= (np.ldexp(w, eq[:, None]) @ k.T).max() - 1e-9 * abs(s[0])
        brute = max((np.maximum(w[r] * lo, w[r] * hi).sum()) * 2.0 ** (eq[r] + e) for r in range(6))
        assert s[0] == brute and float(np.float32(s[0])) == s[0]   # exact in fp32
    assert pages.digest(np.full((3, 4), np.nan))[0].tolist() == [0] * 4 and pages.digest(np.zeros((2, 4)))[2] == 0
    lo, hi, e = pages.digest(np.array([[np.inf, 1.0], [2.0, np.nan]]))
    assert (lo.tolist(), hi.tolist(), e) == ([64, 32], [127, 32], -5)   # the scale is the finite 2.0's


def test_lists():
    assert pages.choose([5, 1, 5, 7, 5], 0, 5, 3) == [0, 2, 3]   # ties: the earlier
    assert pages.span(100, 1, 16, 1, 2) == (1, 4, 6, 6) and pages.span(3, 1, 16, 1, 2) == (0, 0, 0, 0)
    assert pages.span(30, 5, 16, 9, 0) == (1, 1, 1, 2) and pages.span(-5, 5, 16, 1, 1) is None
    assert pages.span(-5, 6, 16, 1, 1) == (0, 0, 0, 0)

    class S:
        heads = 1

        def __call__(self, rows, h):
            return np.arange(20.0) % 7
    q = np.zeros((1, 1, 4))
    ((i, n, lists, keys),) = pages.select(q, 16 * 18 + 3, 16, S(), 2, 1, 1, 1)
    assert lists == [[0, 6, 13, 17, 18]] and keys == 4 * 16 + 4
