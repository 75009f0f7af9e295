"""Value scales at both ends of fp32 in the attention over the cache.  kv8_attention takes v_scales
from 2^-80 to 2^126 and counts others as the nearest of these.

Bounds as in test_gpu_kv8.py.  A weight below the least that f16 holds is lost from the output (not
from the sum): at most 2^-25 of a unit each, where the largest weight is 2^6 or more, so keys * 448 *
2^-31 of the largest v_scale in all."""
import math

import pytest
import torch

import kv8_reference as ref
from nvfp4_weight_only_gb300 import ffi
from test_gpu_kv8 import Setup, draw_q, run_attention

pytestmark = pytest.mark.gpu

LEAST, MOST = 2.0 ** -80, 2.0 ** 126


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ffi.load(build_if_missing=True)
    return torch.device("cuda:0")


def check(s, q, scale):
    out, lse = run_attention(s, q, scale)
    v_scales = s.scales["v"].double().clamp(LEAST, MOST)
    v = ref.e4m3_value(s.codes["v"]) * v_scales[..., None, None]
    want, want_lse, weight, reach = ref.attention(q, s.values("k"), v, s.page, s.table, s.q_lens,
                                                  s.kv_lens, scale)
    d = (s.dim + 8) * 2.0 ** -24 * reach
    used = v_scales[s.table.long()[0, :-(-s.kv_lens[0] // s.page)]]
    lost = s.kv_lens[0] * 448 * 2.0 ** -31 * float(used.max())
    # t = log2(e) s + log2(v_scale), up to 128 in size, is rounded once
    d = d + 2.0 ** -17
    assert bool(ref.rounds_to(out, want, (2 * d[..., None] + 2.0 ** -10) * weight + lost).all())
    off = (lse.cpu().double() - want_lse).abs()
    assert bool((off <= d + 2.0 ** -17 + s.kv_lens[0] * 2.0 ** -24
                 + 2.0 ** -22 * want_lse.abs()).all())


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("kind", ["least", "zeros", "most", "tiny", "apart"])
def test_value_scales_at_both_ends(dev, n, dim, kind):
    """Pages of 128 tokens, so that a warp, a row's first tile or a block sees one page only."""
    s = Setup(dev, [n], [300], 1, dim, 128, seed=31)
    first, second, third = (int(p) for p in s.table[0])
    if kind == "least":  # zeros under the least normal scale, as a quantiser with that floor writes
        s.codes["v"][first] = 0
        s.scales["v"][first] = 2.0 ** -126
    elif kind == "zeros":  # a denormal scale
        s.codes["v"][first] = 0
        s.scales["v"][first] = 2.0 ** -140
    elif kind == "most":  # above 2^126: small codes, so that the values are finite
        s.codes["v"][second] = 0x08 | (s.codes["v"][second] & 0x87)
        s.scales["v"][second] = 1.5 * 2.0 ** 126
        for p in (first, third):
            s.scales["v"][p] = 2.0 ** 100
    elif kind == "tiny":
        for p in (first, second, third):
            s.scales["v"][p] = 2.0 ** -110
    else:  # 2^40 apart, and the larger page zero in half of the columns
        s.codes["v"][second, :, :, dim // 2:] = 0
        s.scales["v"][second] = 1.0
        for p in (first, third):
            s.scales["v"][p] = 2.0 ** -40
    s.upload()
    check(s, draw_q(n, 8, dim, 12), 1.0 / math.sqrt(dim))
