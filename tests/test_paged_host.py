"""The paged-cache entry points validate their arguments on the host (no GPU needed: every call
here fails before any launch, or has nothing to launch), and the float64 restatement that the
GPU tests compare with is what it says."""
import ctypes

import numpy as np
import pytest
import torch

import dynamic_sparse_attention_gb300 as dsa
from dynamic_sparse_attention_gb300 import _build, binding
from oracle import paged


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


def _write(lib, s, k_new=OK, k_stride=1024, v_stride=1024, start=OK, lens=OK, table=OK, k=OK, v=OK, ks=OK, vs=OK):
    return lib.kv_cache_write(k_new, OK, k_stride, v_stride, start, lens, table, ctypes.byref(s), k, v, ks, vs, None)


def _read(lib, s, T=100, k=OK, ks=OK, out=OK):
    return lib.kv_cache_read(k, OK, ks, OK, OK, OK, ctypes.byref(s), T, out, OK, None)


def _attn(lib, s, q=OK, q_stride=1024, start=OK, n_sink=0, n_stream=-1, scale=0.1, ks=OK, out=OK, lse=OK, ws=OK,
          ws_bytes=1 << 40):
    return lib.paged_attn(q, q_stride, OK, OK, ks, OK, start, OK, OK, ctypes.byref(s), n_sink, n_stream, scale, out, lse,
                          ws, ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), -1), (dict(B=4097), -2), (dict(n_tok=-1), -1), (dict(n_pages=0), -1), (dict(max_pages=0), -1),
    (dict(page_size=8), -2), (dict(page_size=24), -2), (dict(page_size=2048), -2), (dict(max_pages=1 << 25), -1),
    (dict(H_q=9), -1), (dict(H_q=256), -2), (dict(D=96), -2), (dict(dtype=1), -2), (dict(dtype=7), -2)])
def test_bad_shapes_are_rejected(lib, kw, status):
    n, s = ctypes.c_size_t(), _shape(**kw)
    assert lib.paged_attn_workspace(ctypes.byref(s), ctypes.byref(n)) == status
    assert lib.dsa_last_error()
    for call in (_write, _read, _attn):
        assert call(lib, s) == status


def test_bad_pointers_and_strides_are_rejected(lib):
    s, fp8 = _shape(), _shape(dtype=2)
    for call in (_write, _read, _attn):
        assert call(lib, fp8, ks=None) == -4
    assert _write(lib, s, k_new=None) == -4 and _write(lib, s, k_new=OK + 2) == -4
    assert _write(lib, s, start=None) == -4 and _write(lib, s, lens=OK + 1) == -4 and _write(lib, s, table=None) == -4
    assert _write(lib, s, k=OK + 8) == -4
    for stride in (255, 252, 260, 0, -1024):            # 2 heads of 128: at least 256, a multiple of 8
        assert _write(lib, s, k_stride=stride) == -1 and _write(lib, s, v_stride=stride) == -1
    assert _read(lib, s, T=0) == -1 and _read(lib, s, out=None) == -4 and _read(lib, s, k=None) == -4
    assert _attn(lib, s, q=OK + 4) == -4 and _attn(lib, s, out=None) == -4 and _attn(lib, s, lse=OK + 2) == -4
    assert _attn(lib, s, q_stride=1016) == -1 and _attn(lib, s, start=None) == -4
    assert _attn(lib, s, n_sink=-1) == -1 and _attn(lib, s, n_stream=-2) == -1
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert _attn(lib, s, scale=scale) == -1
    assert _attn(lib, s, ws_bytes=100) == -3 and _attn(lib, s, ws=None) == -3


def test_overlapping_memory_is_rejected(lib):
    """Ranges that share a byte; the same arguments apart would go on to a launch."""
    s = _shape()                                        # q and out: 8 tokens of 8 heads of 128, 16 KB
    far = [OK + (i << 32) for i in range(8)]
    call = lambda q=far[0], out=far[1], lse=far[2], ws=far[3], k=far[4], v=far[5]: lib.paged_attn(
        q, 1024, k, v, None, None, OK, OK, OK, ctypes.byref(s), 0, -1, 0.1, out, lse, ws, 1 << 31, None)
    names = lambda: lib.dsa_last_error().decode()
    for kw, two in ((dict(out=far[0]), "out and q"), (dict(out=far[0] + 16384 - 16), "out and q"),
                    (dict(lse=far[1] + 64), "lse and out"), (dict(ws=far[4] + 1024), "workspace and k_pages"),
                    (dict(v=far[1] - 64 * 64 * 2 * 256 + 16), "out and v_pages"), (dict(ws=far[2]), "workspace and lse")):
        assert call(**kw) == -1 and two in names(), (kw, names())
    assert lib.kv_cache_write(far[0], far[1], 256, 256, OK, OK, OK, ctypes.byref(s), far[2], far[2] + 4096, None, None,
                              None) == -1 and "v_pages and k_pages" in names()
    assert lib.kv_cache_write(far[0], far[1], 256, 256, OK, OK, OK, ctypes.byref(s), far[2], far[1], None, None,
                              None) == -1 and "v_pages and v_new" in names()
    assert lib.kv_cache_read(far[0], far[1], None, None, OK, OK, ctypes.byref(s), 100, far[2], far[2], None) == -1
    assert "v_out and k_out" in names()


def test_stream_of_another_device():
    class Other:
        cuda_stream, device_index = 7, 3
    with pytest.raises(ValueError, match="device 3"):
        binding._on(0, Other())


def test_nothing_to_do(lib):
    s = _shape(n_tok=0)
    assert _write(lib, s, k_new=None) == 0
    assert _attn(lib, s, q=None, out=None, ws=None, ws_bytes=0) == 0
    assert _write(lib, s, start=None) == -4 and _attn(lib, s, scale=0.0) == -1   # still checked


def test_workspace_covers_every_share(lib):
    n = ctypes.c_size_t()
    s = _shape(n_tok=1)                                 # 4 rows of a KV head
    assert lib.paged_attn_workspace(ctypes.byref(s), ctypes.byref(n)) == 0
    assert n.value >= 2 * 152 * 4 * (128 + 2) * 4
    s = _shape(n_tok=500)                               # two query tiles
    assert lib.paged_attn_workspace(ctypes.byref(s), ctypes.byref(n)) == 0
    assert n.value >= 2 * 152 * 256 * (128 + 2) * 4


def test_binding_rejects_cpu_tensors(lib):
    c = dsa.PagedKVCache.empty(4, 16, 2, 64, device="cpu")
    one, table = torch.ones(1, dtype=torch.int32), torch.zeros(1, 1, dtype=torch.int32)
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        dsa.paged_attn(q, c, torch.tensor([0, 1], dtype=torch.int32), one, table)
    with pytest.raises(ValueError):
        dsa.kv_cache_write(c, q[:, :2], q[:, :2], torch.tensor([0, 1], dtype=torch.int32), one, table)
    with pytest.raises(ValueError):
        dsa.kv_cache_read(c, one, table)


# ------------------------------------------------------------ the restatement

def test_grid_and_rounding_against_torch():
    g = paged.e4m3_grid()
    codes = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(g, codes)
    x = torch.cat([torch.randn(20000) * s for s in (0.003, 1.0, 100.0)] + [torch.tensor(np.concatenate([g, (g[1:] + g[:-1]) / 2]))])
    x = x.clamp(-448, 448).float()
    want = x.to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    got = paged.e4m3_codes(x.double().numpy())
    assert np.array_equal(got & 0x7F, want & 0x7F)


def test_scales_are_the_smallest_that_do_not_saturate():
    rng = np.random.default_rng(0)
    x = torch.from_numpy(rng.standard_normal((3000, 16)) * np.exp2(rng.integers(-40, 40, (3000, 1)))).bfloat16().double().numpy()
    codes, e = paged.quantise(x)
    a = np.abs(x).max(1)
    assert (a <= 448 * np.exp2(e.astype(float))).all() and (a > 448 * np.exp2(e - 1.0)).all()
    back = paged.dequantise(codes, e)
    assert (np.abs(back - x) <= np.maximum(np.abs(x) / 16, np.exp2(e - 10.0)[:, None])).all()
    assert np.array_equal(back, torch.from_numpy(back).bfloat16().double().numpy())   # exactly bf16 values
    assert paged.quantise(np.array([[np.nan, 1.0]]))[1][0] == paged.E_NAN


def test_attend_against_torch_attention():
    rng = np.random.default_rng(1)
    q, k, v = (rng.standard_normal((n, h, 32)) for n, h in ((9, 4), (20, 2), (20, 2)))
    out, lse, _, _ = paged.attend(q, k, v, 11, 0, None, 0.2)
    qt, kt, vt = (torch.from_numpy(x).transpose(0, 1) for x in (q, np.repeat(k, 2, 1), np.repeat(v, 2, 1)))
    mask = torch.arange(20)[None] <= 11 + torch.arange(9)[:, None]
    want = torch.nn.functional.scaled_dot_product_attention(qt, kt, vt, attn_mask=mask, scale=0.2)
    assert np.abs(out - want.transpose(0, 1).numpy()).max() < 1e-12
    # window and sinks, the literal sum over the keys of one row
    out, lse, _, _ = paged.attend(q, k, v, 11, 3, 5, 0.2)
    p, h = 11 + 4, 3
    keys = [0, 1, 2] + list(range(p - 4, p + 1))
    w = np.exp(0.2 * k[keys, h // 2] @ q[4, h])
    assert np.allclose(out[4, h], w @ v[keys, h // 2] / w.sum(), atol=1e-12) and np.isclose(lse[4, h], np.log(w.sum()))
    assert np.isneginf(paged.attend(q, k, v, 11, 0, 0, 0.2)[1]).all()


def test_attend_of_nan_and_infinite_scores():
    """A NaN or plus infinity among a row's scores makes it NaN, minus infinity is a weight of 0,
    and neither touches the other rows."""
    rng = np.random.default_rng(2)
    q, k, v = (rng.standard_normal((n, h, 8)) for n, h in ((4, 2), (9, 1), (9, 1)))
    plain = paged.attend(q, k, v, 5, 0, None, 0.3)[:2]
    q1, k1 = q.copy(), k.copy()
    q1[1, 0, 2] = np.nan                                # row 1 of head 0
    k1[8] = np.inf * np.sign(q[3, 1])                   # seen by row 3 alone: + infinity for its head 1
    out, lse, _, size = paged.attend(q1, k1, v, 5, 0, None, 0.3)
    assert np.isnan(out[1, 0]).all() and np.isnan(lse[1, 0]) and np.isnan(out[3, 1]).all() and np.isnan(lse[3, 1])
    for i, h in ((0, 0), (0, 1), (1, 1), (2, 0), (2, 1)):
        assert np.allclose(out[i, h], plain[0][i, h]) and np.isclose(lse[i, h], plain[1][i, h])
    k1[8] = -k1[8]                                      # - infinity: as if the key were not there
    out, lse, _, _ = paged.attend(q, k1, v, 5, 0, None, 0.3)
    want, wl, _, _ = paged.attend(q[3:], k[:8], v[:8], 7, 0, None, 0.3)
    assert np.allclose(out[3, 1], want[0, 1]) and np.isclose(lse[3, 1], wl[0, 1])
    out, lse, _, _ = paged.attend(np.full((1, 1, 8), np.nan), k[:1], v[:1], 0, 0, None, 0.3)
    assert np.isnan(out).all() and np.isnan(lse).all()
    out, lse, _, _ = paged.attend(np.full((1, 1, 8), np.nan), k[:1], v[:1], 0, 0, 0, 0.3)   # no window, no sinks
    assert (out == 0).all() and np.isneginf(lse).all()  # a row that sees nothing stays empty


def test_overlapping_scales_and_tables_are_rejected(lib):
    """Scale arrays and index tensors count too: as outputs of a write, as inputs of the others.  (Each
    call here overlaps somewhere, so none goes on to a launch.)"""
    s = _shape(dtype=2, B=3)                            # scales of 64 * 64 * 2 bytes, a table of 3 * 16 entries
    far = [OK + (i << 32) for i in range(12)]
    last = lambda: lib.dsa_last_error().decode()

    def write(k=far[2], v=far[3], ks=far[4], vs=far[5], start=far[6], lens=far[7], table=far[8], shape=s):
        return lib.kv_cache_write(far[0], far[1], 256, 256, start, lens, table, ctypes.byref(shape), k, v, ks, vs, None)

    def read(ks=far[2], vs=far[3], lens=far[4], table=far[5], ko=far[6], vo=far[7]):
        return lib.kv_cache_read(far[0], far[1], ks, vs, lens, table, ctypes.byref(s), 100, ko, vo, None)

    def attn(ks=far[2], vs=far[3], start=far[4], lens=far[5], table=far[6], out=far[7], lse=far[8], ws=far[9]):
        return lib.paged_attn(far[11], 1024, far[0], far[1], ks, vs, start, lens, table, ctypes.byref(s), 0, -1, 0.1, out,
                              lse, ws, 1 << 31, None)

    out_bytes = 3 * 100 * 2 * 128 * 2
    for call, kw, two in (
            (write, dict(vs=far[4]), "v_scale and k_scale"), (write, dict(vs=far[4] + 64 * 64 * 2 - 1), "v_scale and k_scale"),
            (write, dict(ks=far[2] + 16), "k_scale and k_pages"), (write, dict(vs=far[0] + 1), "v_scale and k_new"),
            (write, dict(start=far[3] + 64), "v_pages and q_start"), (write, dict(start=far[4] - 12), "k_scale and q_start"),
            (write, dict(lens=far[4] + 8), "k_scale and kv_len"), (write, dict(table=far[5] - 3 * 16 * 4 + 4), "v_scale and page_table"),
            (read, dict(ks=far[6] + 16), "k_out and k_scale"), (read, dict(vs=far[7] - 1), "v_out and v_scale"),
            (read, dict(lens=far[6] + out_bytes - 4), "k_out and kv_len"), (read, dict(table=far[7] + 4), "v_out and page_table"),
            (attn, dict(ks=far[9] + 5), "workspace and k_scale"), (attn, dict(vs=far[7] + 5), "out and v_scale"),
            (attn, dict(start=far[8] - 12), "lse and q_start"), (attn, dict(lens=far[9] - 8), "workspace and kv_len"),
            (attn, dict(table=far[7] + 1024), "out and page_table")):
        assert call(**kw) == -1 and last().endswith(f"{two} overlap"), (kw, last())
    # a bf16 cache has no scales: whatever stands there overlaps nothing (the next pair does)
    assert write(ks=far[2], vs=far[2], lens=far[3], shape=_shape(B=3)) == -1 and "v_pages and kv_len" in last()


def test_default_stream_of_another_device(lib, monkeypatch):
    """Every device's default stream has the handle 0: each entry point tells them apart by the device,
    before it looks at anything else."""
    class Default:
        cuda_stream, device_index = 0, 1
    c = dsa.PagedKVCache.empty(4, 16, 2, 64, device="cpu")
    monkeypatch.setattr(binding, "_cache_args", lambda cache: (OK, OK, None, None, cache.k.shape, 0, 0))
    monkeypatch.setattr(binding, "_current_stream", lambda dev: 0)
    one, table = torch.ones(1, dtype=torch.int32), torch.zeros(1, 1, dtype=torch.int32)
    start, q = torch.tensor([0, 1], dtype=torch.int32), torch.zeros(1, 4, 64, dtype=torch.bfloat16)
    for call in (lambda: dsa.kv_cache_write(c, q[:, :2], q[:, :2], start, one, table, stream=Default()),
                 lambda: dsa.kv_cache_read(c, one, table, stream=Default()),
                 lambda: dsa.paged_attn(q, c, start, one, table, stream=Default())):
        with pytest.raises(ValueError, match="stream is on device 1, the cache on device 0"):
            call()
    Default.device_index = 0                            # the cache's own: on to the next check
    with pytest.raises(ValueError, match="page_table must be contiguous and on the cache's device"):
        dsa.paged_attn(q, c, start, one, table, stream=Default())


@pytest.mark.parametrize("kw", [dict(n_sink=-1), dict(n_sink=-2 ** 32), dict(n_sink=1 - 2 ** 40), dict(n_stream=-1),
                                dict(n_stream=-2 ** 32)])
def test_negative_windows_of_any_size(lib, monkeypatch, kw):
    """-2^32 is 0 in 32 bits.  (Pages of 24 rows: the library would refuse the call as well.)"""
    c = dsa.PagedKVCache.empty(4, 24, 2, 64, device="cpu")
    monkeypatch.setattr(binding, "_cache_args", lambda cache: (OK, OK, None, None, cache.k.shape, 0, -1))
    monkeypatch.setattr(binding, "_current_stream", lambda dev: 0)
    one, table = torch.ones(1, dtype=torch.int32), torch.zeros(1, 1, dtype=torch.int32)
    start, q = torch.tensor([0, 1], dtype=torch.int32), torch.zeros(1, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="must be >= 0"):
        dsa.paged_attn(q, c, start, one, table, **kw)
