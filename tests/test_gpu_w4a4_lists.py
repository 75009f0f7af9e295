"""Products by expert on lists that do not fit their rows: what the header says of each, row by row,
through both kernels (few rows per expert, many)."""
import math

import pytest
import torch

import w4a4_reference as ref
from nvfp4_weight_only_gb300 import ffi
from test_gpu_w4a4 import check, check_gated, draw, draw_weight, of_expert

pytestmark = pytest.mark.gpu

FAR = 2 ** 31 - 1
LISTS = [[0, 50, 20, 90], [0, 20, 5000, 90], [-3, 20, 40, 90], [0, 20, 40, 91], [90, 0, 0, 0],
         [0, FAR, 40, 90], [0, 30, 60, 90], [-5, -5, 0, 90], [5, 5, 70, 70], [90, 90, 90, 95],
         [0, 90, 91, 100], [-FAR - 1, -FAR, 0, 40], [40, 80, FAR, FAR], [-20, 100, 120, 130],
         [10, 10, 10, 9]]


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ffi.load(build_if_missing=True)
    return torch.device("cuda:0")


def computed(list_, M):
    """The experts that take part: none where the list decreases, else those with all of their rows
    inside."""
    if any(a > b for a, b in zip(list_, list_[1:])):
        return []
    return [e for e in range(len(list_) - 1) if 0 <= list_[e] < list_[e + 1] <= M]


def test_the_rule():
    assert [computed(v, 90) for v in LISTS] == [
        [], [], [1, 2], [0, 1], [], [], [0, 1, 2], [2], [1], [], [0], [2], [0], [], []]


@pytest.mark.parametrize("size", [1, 13])  # rows of 3 experts: 90, then 1170 (more than 128 each)
@pytest.mark.parametrize("list_", LISTS)
def test_lists_that_do_not_fit_row_by_row(dev, list_, size):
    M, K, N = 90 * size, 272, 80
    at = [v if abs(v) > 10000 else v * size for v in list_]
    x, w, up = draw(M, K, 1, dev), draw_weight(N, K, 2, dev, 3), draw_weight(N, K, 3, dev, 3)
    rows = ffi.w4a4_quantize(x, start=torch.tensor(at, dtype=torch.int32, device=dev))
    s = torch.full((3,), 1e-3 / math.sqrt(K), device=dev)
    buffers = [torch.full((M + 2, N), -7.0, dtype=torch.bfloat16, device=dev) for _ in range(2)]
    y, h = [b[1:M + 1] for b in buffers]
    ws = ffi.workspace(ffi.w4a4_gemm_workspace_bytes(M, N, K, 3), dev)
    ffi.w4a4_gemm(rows, ffi.w4a4_repack(*w[:2]), w[2], N, ws=ws, out=y)
    ffi.w4a4_gate_up(rows, ffi.w4a4_repack_gate_up(*w[:2], *up[:2]), s, s, N, ws=ws, h=h)
    assert ffi.nvfp4_workspace_status(ws) == 0
    untouched = torch.ones(M, dtype=torch.bool, device=dev)
    for e in computed(at, M):
        mine = slice(at[e], at[e + 1])
        untouched[mine] = False
        v = ref.values(x[mine])
        check(y[mine], *ref.product(v, of_expert(w, e)))
        check_gated(h[mine], 0, v, of_expert((w[0], w[1], s), e), of_expert((up[0], up[1], s), e))
    for b, t in zip(buffers, (y, h)):
        assert bool((b[0] == -7).all()) and bool((b[M + 1] == -7).all())
        assert bool((t[untouched] == -7).all())
