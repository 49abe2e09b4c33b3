"""Run by tests/test_gpu_paged_checked.py in its own process with DSA_CHECKED=1: the paged
operators' checked build runs valid inputs without a report, and reports -- while it still
skips or clamps them -- pages outside the cache, lengths beyond the table and chunks longer
than their sequences, all made on the host."""
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

import torch  # noqa: E402

import dynamic_sparse_attention_gb300 as dsa  # noqa: E402
from dynamic_sparse_attention_gb300 import _build  # noqa: E402

CHECK = 4   # device_error bit of the checked build


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def main():
    assert os.environ.get("DSA_CHECKED") == "1"
    dsa.load()
    assert dsa.library_path() == _build.LIB_CHECKED, dsa.library_path()
    assert dsa.device_error() == 0
    for fp8 in (False, True):
        cache = dsa.PagedKVCache.empty(8, 64, 2, 128, fp8=fp8)
        table = ints(3, 1, 4, 0, 6, 2).reshape(2, 3)
        q = torch.randn(40, 8, 128, device="cuda").bfloat16()
        k = torch.randn(40, 2, 128, device="cuda").bfloat16()
        start, lens = ints(0, 39, 40), ints(150, 100)
        hist = torch.randn(210, 2, 128, device="cuda").bfloat16()

        def run(table=table, start=start, lens=lens):
            dsa.kv_cache_write(cache, k, k, start, lens, table)
            written = dsa.device_error()
            out, _ = dsa.paged_attn(q, cache, start, lens, table)
            torch.cuda.synchronize()
            attended = dsa.device_error()
            dsa.kv_cache_read(cache, lens, table)
            torch.cuda.synchronize()
            return out, written, attended, dsa.device_error()

        dsa.kv_cache_write(cache, hist, hist, ints(0, 111, 210), ints(111, 99), table)
        out, *codes = run()
        assert codes == [0, 0, 0], codes
        assert torch.isfinite(out.float()).all()
        dsa.kv_cache_read(cache, lens, table, T_max=70)   # shorter than the sequences: no error
        torch.cuda.synchronize()
        assert dsa.device_error() == 0
        bad = table.clone()
        bad[0, 2] = 8                      # past the cache: the chunk's own page and keys
        bad[1, 1] = -1
        out, *codes = run(table=bad)
        assert all(c & CHECK for c in codes), codes
        assert torch.isfinite(out.float()).all()
        out, *codes = run(lens=ints(150, 193))   # longer than the table
        assert all(c & CHECK for c in codes), codes
        out, written, attended, _ = run(lens=ints(20, 100))   # shorter than its chunk
        assert written & CHECK and attended & CHECK
        _, written, attended, _ = run(start=ints(0, 39, 41))   # a chunk past the token rows
        assert written & CHECK and attended & CHECK
        assert dsa.device_error() == 0     # read and cleared
    print("paged checked-build ok")


if __name__ == "__main__":
    main()
