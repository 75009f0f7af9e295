"""A decoder layer's buffers are its constructor's."""
import pytest
import torch

from nvfp4_weight_only_gb300 import ffi
from nvfp4_weight_only_gb300.decode_layer import DecodeLayer

pytestmark = pytest.mark.gpu

H, I, PAGE = 512, 1024, 16


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ffi.load(build_if_missing=True)
    return torch.device("cuda:0")


@pytest.mark.parametrize("heads,kv_heads,dim", [(8, 2, 64), (40, 1, 128), (4, 2, 256)])
def test_a_step_allocates_nothing(dev, heads, kv_heads, dim):
    """So a first step inside a graph's capture leaves no workspace behind whose zero-fill is part of
    the graph only.  Workspaces are as large as each batch's call asks for."""
    rope = ffi.rope_table(100, dim, 10000.0, dev)
    layer = DecodeLayer.synthetic(H, I, heads, kv_heads, dim, dev, layer=1, rope=rope)
    cache = ffi.Kv8Cache.empty(16, kv_heads, PAGE, dim, dev)
    x = torch.zeros((64, H), dtype=torch.bfloat16, device=dev)
    for q_lens in ([1], [1, 1, 1, 1], [40], [2, 2], [1, 0, 0, 0]):
        starts = [sum(q_lens[:b]) for b in range(len(q_lens) + 1)]
        batch = ffi.Kv8Batch(torch.tensor(starts, dtype=torch.int32, device=dev),
                             torch.full((len(q_lens),), 50, dtype=torch.int32, device=dev),
                             torch.arange(16, dtype=torch.int32, device=dev).view(-1, 4)[
                                 :len(q_lens)].contiguous())
        before = torch.cuda.memory_allocated(dev)
        layer.step(x[:starts[-1]], x[:starts[-1]], cache, batch)
        assert torch.cuda.memory_allocated(dev) == before
    torch.cuda.synchronize()
