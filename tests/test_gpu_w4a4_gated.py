"""act(g) * u where the sigmoid of g is below fp32's normal numbers: a product with a large u is not."""
import math

import pytest
import torch

import w4a4_reference as ref
from nvfp4_weight_only_gb300 import ffi

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
H, I = 256, 64


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ffi.load(build_if_missing=True)
    return torch.device("cuda:0")


@pytest.mark.parametrize("M", [5, 300, 20000])  # single blocks, few and many rows; pairs
@pytest.mark.parametrize("u", [1.0, -2.0 ** 40, 2.0 ** 100])
@pytest.mark.parametrize("kind,low", [(0, -190.0), (1, -13.0)])
def test_gates_far_below_zero(dev, kind, low, u, M):
    # feature i: weight 1 at element i, so g is x's value there; up has weight 1 at element 64 + i
    codes = torch.zeros((2, I, H // 2), dtype=torch.uint8)
    for i in range(I):
        for which, at in enumerate((i, 64 + i)):
            codes[which, i, at // 2] = 2 << 4 * (at % 2)
    scales = torch.full((I, H // 16), 0x38, dtype=torch.uint8, device=dev)
    codes = codes.to(dev)
    packed = ffi.w4a4_repack_gate_up(codes[0], scales, codes[1], scales)
    # each value one that its block's scale (1) and the codes hold: -6 .. -0.5, times the row's r
    x = torch.zeros((M, H), dtype=torch.float64, device=dev)
    grid = torch.tensor([6, 4, 3, 2, 1.5, 1, 0.5, 6], dtype=torch.float64, device=dev)
    x[:, :64] = -grid.repeat(8)
    x[:, 64:128] = 6.0
    rows = ffi.w4a4_quantize(x.to(BF))
    assert torch.equal(ffi.w4a4_dequantize(rows).double(), x)
    # (M rows alike: what differs is the gate's scale, over the calls)
    for top in torch.linspace(low, low / 4, 24, dtype=torch.float64).tolist():
        scale = float(torch.tensor(-top / 6).to(torch.float32))
        g = (x[0, :64] * scale).to(torch.float32).to(BF).double()  # one fp32 product, then bf16
        h = ffi.w4a4_gate_up(rows, packed, scale, u / 6, I, kind).double()
        want = ref.act(kind, g) * u
        # a rounding to bf16 (2^-134 below its normal numbers), and an exponential whose argument, up
        # to 256, is off by 2^-24 of it at most 8 times: 5 products and sums of GeLU's, 3 of a
        # power of 2's
        far = (h - want).abs() - (2.0 ** -8 + 2.0 ** -13) * want.abs() - 2.0 ** -134
        assert bool((far <= 0).all()), (top, h[0], want)
