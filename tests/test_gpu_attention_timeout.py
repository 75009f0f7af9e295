"""The bounded waits of attention with many rows, driven to run out.

The testing switch makes the copying warp stop behind half of a block's tiles, so the first tiles'
products are under way when the converting warps' wait runs out.  The kernel must report
NVFP4_ERR_TIMEOUT and end; with the switch off the next call on the workspace must be right."""
import pytest
import torch

from nvfp4_weight_only_gb300 import ffi
from test_gpu_kv8 import Setup, draw_q

pytestmark = pytest.mark.gpu

TIMEOUT = 7
WAIT_NS = 2_000_000


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ffi.load(build_if_missing=True)
    return torch.device("cuda:0")


@pytest.mark.parametrize("q_lens,kv_lens,heads,kv_heads,dim", [
    ([64], [3000], 16, 2, 128),            # both row tiles, a unit cut into parts
    ([64], [3000], 16, 2, 64),
    ([40], [300], 2, 2, 128),              # one row tile
    ([300] * 8, [900] * 8, 16, 4, 128),    # several segments per block
    ([300] * 8, [900] * 8, 16, 4, 64),
    ([33], [33], 1, 1, 64)])               # one tile in all: no copy is made
def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right(dev, q_lens, kv_lens, heads,
                                                                      kv_heads, dim):
    s = Setup(dev, q_lens, kv_lens, kv_heads, dim, 64, seed=37)
    q = draw_q(s.tokens, heads, dim, 2).to(dev)
    want = ffi.kv8_attention(q, s.cache, s.batch, 0.1)
    ws = ffi.workspace(ffi.kv8_attention_workspace_bytes(s.cache, s.batch, s.tokens, heads), dev)
    L = ffi.load()
    for _ in range(2):
        assert L.nvfp4_testing_inject_stall(1, WAIT_NS) == 0
        try:
            ffi.kv8_attention(q, s.cache, s.batch, 0.1, ws=ws)
            assert ffi.nvfp4_workspace_status(ws) == TIMEOUT
        finally:
            assert L.nvfp4_testing_inject_stall(0, 0) == 0
        assert torch.equal(ffi.kv8_attention(q, s.cache, s.batch, 0.1, ws=ws), want)
        assert ffi.nvfp4_workspace_status(ws) == 0
    assert ffi.kv8_batch_status(s.batch) == 0
