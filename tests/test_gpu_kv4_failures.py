"""Waits of the attention kernels that run out, without a GPU fault: a warp that waits for what nothing
brings, and launches of the index-checking build in which every fetching warp leaves out one copy while its
readers wait for it. The call ends after the wait limit with W4A16_ERR_DEVICE_TIMEOUT; with the workspace
zeroed the next call gives what it always gave."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

from gpu_util import lib
from test_gpu_kv4 import Batch, cuda

pytestmark = pytest.mark.gpu

TIMEOUT = 5  # W4A16_ERR_DEVICE_TIMEOUT


@pytest.fixture(scope="module")
def W():
    return lib()


@pytest.mark.parametrize("mode", [0, 1])
def test_a_wait_that_nothing_ends_is_reported(W, mode):
    assert W.w4a16_device_status() == W.OK
    assert W.w4a16_set_wait_timeout_ns(1_000_000) == W.OK
    try:
        assert W.w4a16_kv4_selftest_wait_timeout(mode) == W.OK
        assert W.w4a16_device_status() == TIMEOUT
        assert W.w4a16_device_status() == W.OK
    finally:
        assert W.w4a16_set_wait_timeout_ns(2_000_000_000) == W.OK


CASES = {
    # lens, q_lens, H, KV, D, table for longer sequences, copy left out
    "chunks-first": ([60000], [1], 20, 4, 256, False, 0),
    "chunks-second": ([60000], [1], 20, 4, 256, False, 1),
    "runs-first": ([1000] * 40, [1] * 40, 40, 8, 128, False, 0),
    "runs-later": ([1000] * 40, [1] * 40, 40, 8, 128, False, 3),
    "runs-heads-of-64": ([300, 2000, 0, 7] * 12, [1, 2, 1, 1] * 12, 16, 16, 64, False, 2),
    "one-cta-first": ([5000, 90], [20, 20], 20, 4, 256, True, 0),
    "one-cta-later": ([5000, 90], [20, 20], 20, 4, 256, True, 3),
    "one-cta-heads-of-64": ([4000, 900], [30, 5], 8, 2, 64, True, 5),
    "pair-first": ([5000, 300], [60, 60], 20, 4, 256, True, 0),
    "pair-later": ([5000, 300], [60, 60], 20, 4, 256, True, 4),
    "pair-heads-of-128": ([3000], [60], 8, 2, 128, True, 1),
}


@pytest.mark.parametrize("case", CASES)
def test_a_copy_that_never_comes_ends_the_call_and_not_the_next(W, case):
    lens, q_lens, H, KV, D, wide, copy = CASES[case]
    debug = W.load_debug_bounds()
    b = Batch(W, 30, lens, q_lens, H, KV, D, 64)
    q, args = cuda(b.q), b.args(wide)
    want = W.kv4_attention(q, b.cache, **args)
    torch.cuda.synchronize()
    s = torch.cuda.current_stream().cuda_stream

    def call():
        out = torch.zeros_like(q)
        assert debug.w4a16_kv4_attention(
            q.data_ptr(), q.stride(0), H, ctypes.byref(b.cache.desc), args["block_table"].data_ptr(),
            args["block_table"].shape[1], args["kv_len"].data_ptr(), args["q_start"].data_ptr(), len(lens), sum(q_lens),
            args["max_q_len"], 1, D ** -0.5, out.data_ptr(), None, b.work.data_ptr(), b.work.numel(), s) == W.OK
        torch.cuda.synchronize()
        return out

    assert debug.w4a16_device_status(s) == W.OK
    assert debug.w4a16_set_wait_timeout_ns(1_000_000) == W.OK
    assert debug.w4a16_kv4_selftest_withhold(copy) == W.OK
    try:
        call()
        assert debug.w4a16_device_status(s) == TIMEOUT
        assert debug.w4a16_device_status(s) == W.OK
    finally:
        assert debug.w4a16_kv4_selftest_withhold(-1) == W.OK
        assert debug.w4a16_set_wait_timeout_ns(2_000_000_000) == W.OK
    b.work.zero_()
    for _ in range(2):
        out = call()
        assert debug.w4a16_device_status(s) == W.OK
        assert torch.equal(out.view(torch.int16), want.view(torch.int16))
    assert np.isfinite(out.float().cpu().numpy()).all()
