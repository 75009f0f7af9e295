"""The 8-bit norm's codes are those of the fp32 quotient y / scale, rounded once, near ties too.

Rows of +-1 with eps 0 have the norm 1 exactly, so y is the weight, any bf16 value, and the scale is
fl(amax / 448): every quotient is known without an error."""
import numpy as np
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


def ties():
    """Groups of 128 bf16 weights, the largest first, whose quotients by fl(largest / 448) lie at
    or beside a midpoint of two E4M3 values."""
    values = (torch.arange(0x3000, 0x4380, dtype=torch.int32) << 16).view(torch.float32).numpy()
    groups = []
    for top in values[values >= 1][::7]:
        scale = np.float32(top) / np.float32(448)
        below = values[values <= top]
        q = below / scale
        step = np.exp2(np.floor(np.log2(np.maximum(q, 2.0 ** -6))) - 3).astype(np.float32)
        # distance from the midpoint, in fp32 units of the quotient
        off = np.abs(np.mod(q.astype(np.float64) / step, 1) - 0.5) * step / np.spacing(q)
        near = below[off <= 3]
        if near.size:
            row = np.full(128, top, dtype=np.float32)
            row[1:1 + min(127, near.size)] = near[:127]
            groups.append(row)
    return torch.from_numpy(np.concatenate(groups))


@pytest.mark.parametrize("M", [1, 300])  # few rows and many: one and two vectors per thread
def test_codes_are_those_of_the_exact_quotient(dev, M):
    w = ties()
    H = min(w.numel(), 8192) // 128 * 128
    assert H >= 1024
    for at in range(0, w.numel() - H + 1, H):
        part = w[at:at + H].bfloat16()
        assert torch.equal(part.float(), w[at:at + H])
        g = torch.Generator().manual_seed(at)
        sign = torch.randint(0, 2, (M, H), generator=g) * 2 - 1
        codes, scales = ffi.add_rmsnorm_e4m3(sign.bfloat16().to(dev), part.to(dev), 0.0)
        top = part.float().view(-1, 128).amax(1)
        want_scales = torch.from_numpy(top.numpy() / np.float32(448))
        assert torch.equal(scales.cpu(), want_scales.expand(M, -1))
        q = torch.from_numpy((part.float().view(-1, 128).numpy() / want_scales.numpy()[:, None]))
        want = ref.round_e4m3(q.flatten()).expand(M, -1) | (sign < 0).to(torch.uint8) * 128
        assert torch.equal(codes.cpu(), want)


def test_zeros_keep_their_signs_and_infinities_take_the_scale(dev):
    tops = torch.linspace(1, 2, 16)[:, None].expand(16, 128)  # scales of many mantissas
    w = tops.clone()
    w[:, 1:64] = 0.0
    w[3, 100], w[5, 101] = float("inf"), float("nan")
    part = w.flatten().bfloat16()
    sign = torch.randint(0, 2, (1, 2048), generator=torch.Generator().manual_seed(2)) * 2 - 1
    codes, scales = ffi.add_rmsnorm_e4m3(sign.bfloat16().to(dev), part.to(dev), 0.0)
    codes, scales = codes.cpu(), scales.cpu()[0]
    minus = (sign < 0).to(torch.uint8) * 128
    groups = part.float().view(16, 128)
    known = groups.masked_fill(torch.isnan(groups), 0)
    assert torch.equal(scales, torch.from_numpy(known.amax(1).numpy() / np.float32(448)))
    with np.errstate(invalid="ignore"):  # inf / inf
        q = torch.from_numpy(groups.numpy() / scales.numpy()[:, None])
    want = ref.round_e4m3(q.flatten()) | minus[0]
    nan = torch.isnan(q.flatten())
    assert torch.equal(codes[0][~nan], want[~nan])
    assert nan.sum() == 2 and bool(((codes[0][nan] & 127) == 127).all())
