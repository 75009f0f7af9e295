"""Calls on 4-bit activations directly behind what writes their inputs, the weight among them, and
decode products behind them."""
import pytest
import torch

from nvfp4_weight_only_gb300 import ffi
from test_gpu_w4a4 import draw, draw_weight

pytestmark = pytest.mark.gpu

# few rows, tiles of 128 x 128 in one turn, pairs of blocks with cut tiles
SIZES = [(7, 5120, 1024), (300, 1024, 1000), (1000, 8192, 5000)]
TIMES = 12


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ffi.load(build_if_missing=True)
    return torch.device("cuda:0")


def alternate(step, outs, wants, captured):
    """step(i) leaves outs as wants[i % 2] has them, every time."""
    step(0)
    graphs = []
    for i in range(2):
        if captured:
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[i]):
                step(i)
    got = []
    for i in range(TIMES):
        graphs[i % 2].replay() if captured else step(i % 2)
        got.append([t.clone() for t in outs])
    for i, mine in enumerate(got):
        for a, b in zip(mine, wants[i % 2]):
            assert torch.equal(a, b), i


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("between", ["nothing", "norm", "product"])
@pytest.mark.parametrize("M,K,N", SIZES)
def test_a_weight_written_by_the_kernel_in_front(dev, M, K, N, between, captured):
    x, w = draw(M, K, 1, dev), [draw_weight(N, K, s, dev) for s in (2, 3)]
    rows, packs = ffi.w4a4_quantize(x), [ffi.w4a4_repack(*v[:2]) for v in w]
    ws = ffi.workspace(ffi.w4a4_gemm_workspace_bytes(M, N, K), dev)
    wants = [[ffi.w4a4_gemm(rows, p, w[0][2], N)] for p in packs]
    assert not torch.equal(wants[0][0], wants[1][0])
    packed, out, other = packs[0].clone(), torch.empty_like(wants[0][0]), torch.empty_like(wants[0][0])
    a, g = draw(4, 256, 5, dev), torch.ones(256, dtype=torch.bfloat16, device=dev)

    def step(i):
        packed.copy_(packs[i])
        if between == "norm":
            ffi.add_rmsnorm_bf16(a, g, 1e-6)
        if between == "product":
            ffi.w4a4_gemm(rows, packs[0], w[0][2], N, ws=ws, out=other)
        ffi.w4a4_gemm(rows, packed, w[0][2], N, ws=ws, out=out)

    alternate(step, [out], wants, captured)


@pytest.mark.parametrize("M,K,N", SIZES)
def test_a_weight_repacked_in_place(dev, M, K, N):
    L, x = ffi.load(), draw(M, K, 1, dev)
    w = [draw_weight(N, K, s, dev) for s in (2, 3)]
    rows = ffi.w4a4_quantize(x)
    ws = ffi.workspace(ffi.w4a4_gemm_workspace_bytes(M, N, K), dev)
    wants = [[ffi.w4a4_gemm(rows, ffi.w4a4_repack(*v[:2]), v[2], N)] for v in w]
    packed, out = ffi.w4a4_repack(*w[0][:2]), torch.empty_like(wants[0][0])

    def step(i):
        assert L.w4a4_repack(w[i][0].data_ptr(), w[i][1].data_ptr(), 1, N, K, packed.data_ptr(),
                             torch.cuda.current_stream(dev).cuda_stream) == 0
        ffi.w4a4_gemm(rows, packed, w[i][2], N, ws=ws, out=out)

    alternate(step, [out], wants, False)


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("M,H,I", [(7, 5120, 1024), (300, 1024, 1040), (1000, 5120, 2496)])
def test_an_ffn_whose_weights_the_kernels_in_front_write(dev, M, H, I, captured):
    x = draw(M, H, 1, dev)
    parts = [[draw_weight(n, k, 10 * s + j, dev) for j, (n, k) in enumerate(((I, H), (I, H), (H, I)))]
             for s in (1, 2)]
    gus = [ffi.w4a4_repack_gate_up(*g[:2], *u[:2]) for g, u, _ in parts]
    dns = [ffi.w4a4_repack(*d[:2]) for _, _, d in parts]
    ws = ffi.workspace(ffi.ffn_swiglu_w4a4_workspace_bytes(M, H, I), dev)
    wants = [[ffi.ffn_swiglu_w4a4(x, a, 1e-5, 1e-5, b, 1e-3, I, ws=ws)] for a, b in zip(gus, dns)]
    gu, dn, out = gus[0].clone(), dns[0].clone(), torch.empty_like(x)

    def step(i):
        dn.copy_(dns[i])
        gu.copy_(gus[i])
        ffi.ffn_swiglu_w4a4(x, gu, 1e-5, 1e-5, dn, 1e-3, I, ws=ws, out=out)

    alternate(step, [out], wants, captured)


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("call", ["product", "quantise", "sum"])
def test_a_decode_product_whose_weight_was_written_two_kernels_before(dev, call, captured):
    N, K = 5120, 2048
    q = [ffi.nvfp4_quantize(draw(N, K, s, dev).float()) for s in (1, 2)]
    packs = [ffi.nvfp4_repack(*v[:2], N, K) for v in q]
    x, scale = draw(1, K, 3, dev), q[0][2]
    ws = ffi.workspace(ffi.nvfp4_gemv_workspace_bytes(1, N, K), dev)
    wants = [[ffi.nvfp4_gemv(x, p, scale, N, ws=ws)] for p in packs]
    packed, out = packs[0].clone(), torch.empty_like(wants[0][0])
    rows, w = ffi.W4a4Rows.empty(5, 256, dev), draw_weight(64, 256, 4, dev)
    a, other = draw(5, 256, 5, dev), ffi.w4a4_repack(*w[:2])
    ws4, y = ffi.workspace(ffi.w4a4_gemm_workspace_bytes(5, 64, 256), dev), draw(5, 64, 6, dev)
    place, one = torch.arange(5, dtype=torch.int32, device=dev).view(5, 1), torch.ones((5, 1), device=dev)
    ffi.w4a4_quantize(a, out=rows)

    def step(i):
        packed.copy_(packs[i])
        if call == "product":
            ffi.w4a4_gemm(rows, other, w[2], 64, ws=ws4, out=y)
        elif call == "quantise":
            ffi.w4a4_quantize(a, out=rows)
        else:
            ffi.experts_sum(a, place, one)
        ffi.nvfp4_gemv(x, packed, scale, N, ws=ws, out=out)

    alternate(step, [out], wants, captured)
