"""The bounded waits of the products on 4-bit activations, driven to run out.

The testing switch makes the copying warp stop behind the first stage, so a stage's products are
under way when the next wait runs out.  The kernel must report NVFP4_ERR_TIMEOUT and end; with the
switch off the next call on the workspace must be right."""
import pytest
import torch

from nvfp4_weight_only_gb300 import ffi
from test_gpu_w4a4 import draw, draw_weight, starts

pytestmark = pytest.mark.gpu

TIMEOUT = 7
WAIT_NS = 2_000_000


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ffi.load(build_if_missing=True)
    return torch.device("cuda:0")


@pytest.mark.parametrize("lens", [None, [30, 0, 250]])
@pytest.mark.parametrize("M,K,N", [(280, 8192, 512), (280, 512, 6000), (30, 5120, 300),
                                   (30, 1024, 30000), (1000, 8192, 5000), (280, 512, 7000)])
def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right(dev, M, K, N, lens):
    if lens and M < sum(lens):
        lens = [10, 0, 20]
    elif lens and M > 2 * sum(lens):
        lens = [500, 0, 500]
    start = starts(lens, 0, dev) if lens else None
    x, w = draw(M, K, 1, dev), draw_weight(N, K, 2, dev, len(lens) if lens else None)
    rows, packed = ffi.w4a4_quantize(x, start=start), ffi.w4a4_repack(*w[:2])
    ws = ffi.workspace(ffi.w4a4_gemm_workspace_bytes(M, N, K, rows.experts), dev)
    want = ffi.w4a4_gemm(rows, packed, w[2], N, ws=ws)
    L = ffi.load()
    for _ in range(2):
        assert L.nvfp4_testing_inject_stall(1, WAIT_NS) == 0
        try:
            ffi.w4a4_gemm(rows, packed, w[2], N, ws=ws)
            assert ffi.nvfp4_workspace_status(ws) == TIMEOUT
        finally:
            assert L.nvfp4_testing_inject_stall(0, 0) == 0
        assert torch.equal(ffi.w4a4_gemm(rows, packed, w[2], N, ws=ws), want)
        assert ffi.nvfp4_workspace_status(ws) == 0
