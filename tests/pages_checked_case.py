"""Run by tests/test_gpu_pages_checked.py in its own process with DSA_CHECKED=1: the checked build of
the operators around the paged cache's sparse path runs valid inputs without a report, and reports --
while it still skips or clamps them -- pages outside the cache, lengths beyond the table, chunks
longer than their sequences and copies of pages that are none, all made on the host."""
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

import torch  # noqa: E402

import dynamic_sparse_attention_gb300 as dsa  # noqa: E402

CHECK = 4   # device_error bit of the checked build


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def main():
    assert os.environ.get("DSA_CHECKED") == "1"
    dsa.load()
    assert dsa.device_error() == 0
    for fp8 in (False, True):
        cache = dsa.PagedKVCache.empty(40, 16, 2, 128, fp8=fp8)
        k = torch.randn(640, 2, 128, device="cuda").bfloat16()
        dsa.kv_cache_write(cache, k, k, ints(0, 640), ints(640), torch.arange(40, device="cuda").int()[None])
        digest = dsa.PageDigest.empty(cache)
        dsa.page_digest_update(cache, digest, 640, ints(0, 640), ints(640), torch.arange(40, device="cuda").int()[None])
        table = torch.randperm(40, device="cuda").int().reshape(2, 20)
        q = torch.randn(40, 8, 128, device="cuda").bfloat16()
        start, lens = ints(0, 39, 40), ints(300, 310)
        f = 1e4 ** (-torch.arange(0, 128, 2, device="cuda").double() / 128)

        def run(table=table, start=start, lens=lens):
            """What each call met, and the lists."""
            codes = []
            dsa.kv_cache_write_rope(cache, q, k[:40], k[:40], start, lens, table, f)
            codes.append(dsa.device_error())
            dsa.page_digest_update(cache, digest, 40, start, lens, table)
            codes.append(dsa.device_error())
            for q_block in (1, 16):
                sel = dsa.page_select(q, digest, start, lens, table, keep=4, q_block=q_block)
                codes.append(dsa.device_error())
                out, _ = dsa.paged_attn(q, cache, sel.q_start, sel.kv_len, sel.page_table)
                codes.append(dsa.device_error())
                assert torch.isfinite(out.float()).all()
            return codes

        assert run() == [0] * 6
        bad = table.clone()
        bad[0, 3] = 40                     # a candidate
        bad[0, 18] = -1                    # the chunk's own
        got = run(table=bad)
        assert all(c & CHECK for c in (got[0], got[1], got[2], got[4])), got
        got = run(lens=ints(300, 321))     # longer than the table
        assert all(c & CHECK for c in (got[0], got[1], got[2], got[4])), got
        got = run(lens=ints(20, 310))      # shorter than its chunk
        assert got[0] & CHECK and got[2] & CHECK and got[4] & CHECK, got
        got = run(start=ints(0, 39, 41))   # a chunk past the token rows
        assert got[0] & CHECK and got[1] & CHECK, got
        dsa.kv_pages_copy(cache, ints(1, 2), ints(5, 6), digest=digest)
        assert dsa.device_error() == 0
        dsa.kv_pages_copy(cache, ints(1, 2), ints(5, 40), digest=digest)
        assert dsa.device_error() & CHECK
        dsa.kv_pages_copy(cache, ints(-1, 2), ints(5, 6))
        assert dsa.device_error() & CHECK
        assert dsa.device_error() == 0     # read and cleared
    print("pages checked-build ok")


if __name__ == "__main__":
    main()
