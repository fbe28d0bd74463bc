"""Failure detection on the device: a bounded wait of the attention kernels that
runs out is reported, and the device stays usable.

As for the GEMM, a wait runs out on purpose without any fault: with the test hook
on (nvfp4_set_test_stall) the barrier of every CTA's first copy of codes never
completes, so that what waits for it gives up after the nvfp4_set_wait_limit bound.  The kernel must
record NVFP4_ERR_TIMEOUT, wait for the copies and products it issued, meet the
other CTAs of its cluster, free its tensor memory and return; the next call with
the same workspace gives the right result with no error recorded."""
import pytest
import torch

import nvfp4_block_scaled_20_b200 as nv
from nvfp4_block_scaled_20_b200 import capi
from gpu_helpers import DEV, require_gpu
from test_gpu_attention_ops import check_sequence, filled, gen, i32

pytestmark = pytest.mark.gpu

NVFP4_ERR_TIMEOUT = 6


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("nq,n,hq,hk,d", [
    (1, 50, 4, 2, 128),       # 8 rows, one step
    (3, 40, 4, 1, 64),        # 16 rows, one step
    (1, 1500, 24, 24, 128),   # runs joined in a cluster
    (5, 1400, 12, 4, 64),
    (1, 20000, 4, 2, 128),    # runs joined by a second kernel
    (2, 30000, 16, 2, 64),
    (100, 90, 1, 1, 128),     # one half of a tile of 256 rows, one step
    (100, 9000, 3, 1, 64),    # both halves, split along the keys
    (600, 3000, 4, 2, 128)])
def test_attention_wait_that_runs_out_is_reported_and_the_device_stays_usable(nq, n, hq, hk, d):
    pages = -(-n // 64)
    c = filled(pages, hk, 64, d, 141)
    t = torch.arange(pages, device=DEV, dtype=torch.int32)[None].contiguous()
    q = (torch.randn((nq, hq, d), generator=gen(142), device=DEV) * 0.1).bfloat16()
    lens, starts = i32([n]), i32([0, nq])
    ws = nv.kv8_attention_workspace(c, t, starts, hq, nq)
    out = torch.full_like(q, 9.0)
    try:
        assert capi.nvfp4_set_wait_limit(2_000_000) == 0  # 2 ms
        assert capi.nvfp4_set_test_stall(1) == 0
        nv.kv8_attention(q, c, t, lens, starts, causal=True, out=out, ws=ws)
        torch.cuda.synchronize()
    finally:
        capi.nvfp4_set_test_stall(0)
        capi.nvfp4_set_wait_limit(0)
    assert nv.device_error(ws) == NVFP4_ERR_TIMEOUT
    assert nv.device_error(ws) == 0  # read back once, then cleared
    lse = torch.empty((nq, hq), device=DEV)
    nv.kv8_attention(q, c, t, lens, starts, causal=True, out=out, lse=lse, ws=ws)
    assert nv.device_error(ws) == 0
    check_sequence(out, lse, q, c, t[0], n, causal=True)
