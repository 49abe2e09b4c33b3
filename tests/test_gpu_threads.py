"""Calls from several host threads at once: a kernel's dynamic shared memory limit is one for all of them, so a
call over small tensors must not lower it under another thread's over large ones."""
import ctypes
import threading

import pytest
import torch

import dynamic_sparse_attention_gb300 as dsa
from dynamic_sparse_attention_gb300 import _build, binding

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    _build.build()
    dsa.load()


def test_block_sparse_lists_of_short_and_long_prompts():
    """Four threads, each on a stream and a workspace of its own: every call is taken and leaves the lists that
    it leaves alone.  (The C entry itself: what Python does between two calls keeps the threads apart.)"""
    lib, jobs, k_b, block = dsa.load(), [], 4, 64
    for S in (1024, 16384, 1024, 16384):
        g = torch.Generator(device="cuda").manual_seed(S)
        q, k = (torch.randn(1, S, h, 64, generator=g, device="cuda").bfloat16() for h in (2, 1))
        names = ("blk_cnt", "blk_idx", "col_cnt")
        want = dsa.block_sparse_index_build(q, k, k_b=k_b)
        for n in names:                                     # (entries behind a list's end are not written)
            want[n].zero_()
        want = dsa.block_sparse_index_build(q, k, k_b=k_b, out=want)
        got = {n: torch.zeros_like(want[n]) for n in names}
        ws = torch.empty(dsa.block_sparse_index_build_workspace_bytes(q, k), dtype=torch.uint8, device="cuda")
        shape, stream = binding.prefill_shape(q, k), torch.cuda.Stream()
        args = (q.data_ptr(), k.data_ptr(), ctypes.byref(shape), block, k_b, want["blk_idx"].shape[-1],
                *(got[n].data_ptr() for n in names), None, ws.data_ptr(),
                ctypes.c_size_t(ws.numel()), stream.cuda_stream)
        jobs.append((q, k, want, got, ws, shape, stream, args))
    torch.cuda.synchronize()
    refused, go = [0] * len(jobs), threading.Barrier(len(jobs))

    def work(i):
        stream, args = jobs[i][-2:]
        go.wait(timeout=60)
        for n in range(2000):
            refused[i] += lib.block_sparse_index_build(*args) != 0
            if n % 100 == 99:                               # (not too far ahead of the GPU)
                stream.synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join(timeout=300)
    torch.cuda.synchronize()
    assert not any(t.is_alive() for t in threads) and refused == [0] * len(jobs), refused
    for _, _, want, got, *_ in jobs:
        assert all(torch.equal(got[n], want[n]) for n in got)
