"""The norm with the residual's addition against 64 bits.  fp32 inside: the sum of squares is off
by at most (H/8 + 16) 2^-24 of itself, so y by half of that and 6 roundings, before the output's own
rounding.  A group's scale carries y's error; a code may be the neighbouring one
where y / scale lies that near to a tie."""
import pytest
import torch

import kv8_reference as ref
from nvfp4_weight_only_gb300 import ffi

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ffi.load(build_if_missing=True)
    return torch.device("cuda:0")


def inputs(M, H, seed=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((M, H), generator=g).bfloat16()
    r = (torch.randn((M, H), generator=g) * 5).bfloat16()
    w = (1 + torch.randn(H, generator=g) * 0.3).bfloat16()
    return x, r, w


def relative(H):
    return (H / 8 + 16) * 2.0 ** -25 + 6 * 2.0 ** -24


SHAPES = [(1, 16), (3, 112), (2, 128), (1, 5120), (64, 5376), (5, 272), (2, 8208), (3, 17408),
          (2, 32768), (300, 4096)]


@pytest.mark.parametrize("M,H", SHAPES)
@pytest.mark.parametrize("with_residual", [True, False])
def test_bf16(dev, M, H, with_residual):
    x, r, w = inputs(M, H, M + H)
    r = r if with_residual else None
    total = torch.empty((M, H), dtype=torch.bfloat16, device=dev)
    out = ffi.add_rmsnorm_bf16(x.to(dev), w.to(dev), 1e-6, sum_out=total,
                               residual=r.to(dev) if with_residual else None, weight_bias=0.25)
    want_r, want = ref.norm(x, r, w, 1e-6, 0.25)
    assert torch.equal(total.cpu(), want_r.float().bfloat16())
    assert bool(ref.rounds_to(out, want, relative(H) * want.abs()).all())


@pytest.mark.parametrize("M,H", SHAPES)
def test_e4m3(dev, M, H):
    x, r, w = inputs(M, H, M + 2 * H)
    total = torch.empty((M, H), dtype=torch.bfloat16, device=dev)
    codes, scales = ffi.add_rmsnorm_e4m3(x.to(dev), w.to(dev), 1e-5, residual=r.to(dev),
                                         sum_out=total)
    want_r, y = ref.norm(x, r, w, 1e-5)
    assert torch.equal(total.cpu(), want_r.float().bfloat16())
    e = relative(H) + 2.0 ** -22
    for g in range(0, H, 128):
        part, scale = y[:, g:g + 128], scales[:, g // 128].cpu().double()
        top = part.abs().amax(1)
        assert bool(((scale - top / 448).abs() <= e * top / 448).all())
        v = part / scale[:, None]
        got = ref.e4m3_value(codes[:, g:g + 128].cpu())
        step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(2.0 ** -6, 448.0))) - 3)
        assert bool(((got - v).abs() <= 0.5 * step + e * v.abs()).all())


def test_zero_rows_and_groups(dev):
    x = torch.zeros((2, 256), dtype=torch.bfloat16)
    x[1, :128] = 1.0
    w = torch.ones(256, dtype=torch.bfloat16)
    out = ffi.add_rmsnorm_bf16(x.to(dev), w.to(dev), 1e-6)
    assert bool((out[0] == 0).all()) and bool((out[1, 128:] == 0).all())
    codes, scales = ffi.add_rmsnorm_e4m3(x.to(dev), w.to(dev), 1e-6)
    assert scales[0].tolist() == [1.0, 1.0] and float(scales[1, 1]) == 1.0
    assert int(codes[0].max()) == 0 and bool((codes[1, :128].view(ref.E4M3).float() == 448).all())
    # zero rows without eps: 0 * inf
    assert bool(torch.isnan(ffi.add_rmsnorm_bf16(x.to(dev), w.to(dev), 0.0)[0].float()).all())


def test_in_place(dev):
    x, r, w = inputs(4, 512)
    out = ffi.add_rmsnorm_bf16(x.to(dev), w.to(dev), 1e-6, residual=r.to(dev))
    a, b = x.to(dev), r.to(dev)
    ffi.add_rmsnorm_bf16(a, w.to(dev), 1e-6, residual=b, sum_out=b, out=a)
    assert torch.equal(a, out) and torch.equal(b.cpu(), (x.float() + r.float()).bfloat16())


def test_rows_are_independent_of_the_batch(dev):
    x, r, w = inputs(17, 1040)
    every = ffi.add_rmsnorm_bf16(x.to(dev), w.to(dev), 1e-6, residual=r.to(dev))
    for i in (0, 9, 16):
        one = ffi.add_rmsnorm_bf16(x[i:i + 1].to(dev), w.to(dev), 1e-6, residual=r[i:i + 1].to(dev))
        assert torch.equal(one[0], every[i])
