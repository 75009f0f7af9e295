"""Products on 4-bit activations against their definitions in 64 bits: quantisation code by code,
dense and grouped products, the FFN, a routed batch's lists and sums, the experts' FFN."""
import math

import pytest
import torch

import w4a4_reference as ref
from nvfp4_weight_only_gb300 import ffi

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
HALF = 2.0 ** -8  # a rounding to bf16, of the value


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ffi.load(build_if_missing=True)
    return torch.device("cuda:0")


def draw(M, K, seed, dev):
    """Rows of unequal size with outliers."""
    g = torch.Generator(device=dev).manual_seed(seed)
    x = torch.randn((M, K), generator=g, device=dev)
    x *= torch.exp(torch.randn((M, 1), generator=g, device=dev))
    big = torch.rand((M, K), generator=g, device=dev) < 0.01
    return torch.where(big, 20 * x, x).to(BF)


def draw_weight(N, K, seed, dev, experts=None):
    """(codes, scales, scale2) with every code and scales over their range."""
    g = torch.Generator(device=dev).manual_seed(seed)
    front = () if experts is None else (experts,)
    codes = torch.randint(0, 256, (*front, N, K // 2), generator=g, device=dev).to(torch.uint8)
    scales = torch.randint(0, 0x7f, (*front, N, K // 16), generator=g, device=dev).to(torch.uint8)
    if experts is None:
        return codes, scales, 0.0007
    return codes, scales, torch.rand(experts, generator=g, device=dev) * 1e-3 + 1e-4


def of_expert(w, e):
    return ref.weight(w[0][e], w[1][e], float(w[2][e]))


def check(got, want, off):
    """got bf16 within a rounding of want, where fp32 sums may be `off` from it."""
    bound = HALF * want.abs() + (1 + HALF) * off + 1e-37
    far = (got.double() - want).abs() - bound
    assert bool((far <= 0).all()), f"{int((far > 0).sum())} values off, worst by {float(far.max())}"


def check_gated(got, kind, x, gate, up):
    """got = bf16(act(bf16(g)) * bf16(u)).  |act'| is at most 1.13, and bf16(g) is within HALF |g|
    of g, or of a sum that is off by its bound."""
    (g, g_off), (u, u_off) = ref.product(x, gate), ref.product(x, up)
    dg, du = HALF * g.abs() + (1 + HALF) * g_off, HALF * u.abs() + (1 + HALF) * u_off
    a = ref.act(kind, g)
    check(got, a * u, 1.13 * dg * (u.abs() + du) + a.abs() * du)


# ------------------------------------------------------------------ quantisation

@pytest.mark.parametrize("M,K", [(1, 16), (1, 256), (3, 272), (127, 48), (130, 5376), (300, 1024),
                                 (5, 17408), (2, 65536), (257, 2064)])
def test_quantize_is_exact(dev, M, K):
    x = draw(M, K, M + K, dev)
    got = ffi.w4a4_dequantize(ffi.w4a4_quantize(x))
    assert torch.equal(got.double(), ref.values(x))


@pytest.mark.parametrize("lo,hi", [(0, 0x7f00), (0x3f00, 0x4080), (0x3f80, 0x3f90), (0x3d00, 0x4400)])
def test_quantize_every_magnitude(dev, lo, hi):
    """Rows of arbitrary bit patterns: ties of both roundings, subnormal blocks, both ends of r."""
    g = torch.Generator(device=dev).manual_seed(lo + hi)
    bits = torch.randint(lo, hi, (20000, 256), generator=g, device=dev)
    sign = torch.randint(0, 2, (20000, 256), generator=g, device=dev) << 15
    x = (bits | sign).to(torch.int32).to(torch.int16).view(BF)
    assert torch.equal(ffi.w4a4_dequantize(ffi.w4a4_quantize(x)).double(), ref.values(x))


@pytest.mark.parametrize("M,K", [(1, 16), (37, 528), (160, 4112), (3, 17408)])
def test_quantize_rows_that_begin_on_16_bytes(dev, M, K):
    x = draw(M * K + 8, 1, K, dev).flatten()[8:].view(M, K)
    assert x.data_ptr() % 32 == 16
    assert torch.equal(ffi.w4a4_dequantize(ffi.w4a4_quantize(x)).double(), ref.values(x))


@pytest.mark.parametrize("K", [16, 512, 528, 1040, 2048, 2064, 4096, 4112, 5120])
@pytest.mark.parametrize("M", [152, 153, 155, 156])
def test_quantize_short_and_long_rows_few_and_many(dev, M, K):
    """Both sides of each rule on rows per block and warps per row, dense and by expert."""
    x = draw(M, K, M + K, dev)
    want = ref.values(x)
    assert torch.equal(ffi.w4a4_dequantize(ffi.w4a4_quantize(x)).double(), want)
    lens = [0, 1, 0, 0, 63, 0, 70, 5]  # rows behind the last expert's
    start = starts(lens, 2, dev)
    rows = ffi.w4a4_quantize(x, start=start)
    out = torch.full((M, K), 7.0, dtype=BF, device=dev)
    ffi.w4a4_dequantize(rows, out=out)
    assert torch.equal(out[2:141].double(), want[2:141])
    assert bool((out[:2] == 7.0).all()) and bool((out[141:] == 7.0).all())


@pytest.mark.parametrize("at", [0, 15, 16, 511, 512, 1037])
@pytest.mark.parametrize("bad", [0x7f80, 0xff80, 0x7fc0, 0xffc0, 0x7f81, 0xffff])
def test_quantize_rows_with_any_value_that_is_not_finite(dev, at, bad):
    """Infinities and NaN of both signs and any payload, in every place of a lane's values."""
    x = draw(3, 1040, at, dev)
    x[1].view(torch.int16)[at] = bad - 65536 if bad > 32767 else bad
    got = ffi.w4a4_dequantize(ffi.w4a4_quantize(x))
    assert bool(torch.isnan(got[1]).all())
    assert torch.equal(got[[0, 2]].double(), ref.values(x[[0, 2]]))


def test_quantize_every_tie(dev):
    """x = tie * s for every scale s that a block can get, beside a value that gives it."""
    s = torch.tensor(ref.E4M3[1:], dtype=torch.float64)
    ties = torch.tensor((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0), dtype=torch.float64)
    x = torch.zeros((s.numel(), 32), dtype=torch.float64)
    x[:, 0] = 6 * s                                # the block's largest
    x[:, 1:8] = ties * s[:, None]
    x[:, 8:15] = -ties * s[:, None]
    x[:, 16] = 2688                                # the row's: r = 1
    assert torch.equal(x, x.to(BF).double())
    got = ffi.w4a4_dequantize(ffi.w4a4_quantize(x.to(BF).to(dev)))
    even = torch.tensor((0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0), dtype=torch.float64)
    assert torch.equal(got[:, 1:8].cpu().double(), even * s[:, None])
    assert torch.equal(got.double(), ref.values(x.to(BF).to(dev)))


def test_zero_rows_and_rows_that_are_not_finite(dev):
    x = draw(10000, 512, 3, dev)
    x[5] = 0
    x[7, 100], x[20, 0], x[139, 511] = math.inf, -math.inf, math.nan
    w = draw_weight(64, 512, 4, dev)
    packed = ffi.w4a4_repack(*w[:2])
    for M in (40, 140, 10000):  # both kernels
        rows = ffi.w4a4_quantize(x[:M].contiguous())
        y = ffi.w4a4_gemm(rows, packed, w[2], 64)
        bad = [r for r in (7, 20, 139) if r < M]
        fine = [r for r in range(M) if r not in bad]
        assert bool(torch.isnan(y[bad]).all()) and bool((y[5] == 0).all())
        want, off = ref.product(ref.values(x[:M][fine]), ref.weight(*w))
        check(y[fine], want, off)


def test_extreme_rows(dev):
    """Rows near both ends of bf16, beside each other."""
    x = draw(300, 256, 5, dev).double()
    x *= torch.exp2(torch.linspace(-118, 112, 300, device=dev, dtype=torch.float64).round())[:, None]
    x = x.to(BF)
    assert bool(torch.isfinite(x).all())
    assert torch.equal(ffi.w4a4_dequantize(ffi.w4a4_quantize(x)).double(), ref.values(x))
    w = draw_weight(128, 256, 6, dev)
    want, off = ref.product(ref.values(x), ref.weight(*w))
    for M in (100, 300):
        y = ffi.w4a4_gemm(ffi.w4a4_quantize(x[:M].contiguous()), ffi.w4a4_repack(*w[:2]), w[2], 128)
        # sums times scale2 times r: fp32's subnormals start at 2^-126
        keep = (want[:M].abs() < 1e38) & ((want[:M].abs() > 2.0 ** -120) | (want[:M] == 0))
        check(torch.where(keep, y.double(), 0.0), torch.where(keep, want[:M], 0.0), off[:M])


# ------------------------------------------------------------------ weights

@pytest.mark.parametrize("N,K,experts", [(1, 16, None), (128, 256, None), (300, 272, None),
                                         (5, 48, 3), (257, 528, 2)])
def test_repack_keeps_every_byte(dev, N, K, experts):
    codes, scales, _ = draw_weight(N, K, N, dev, experts)
    got = ffi.w4a4_unpack(ffi.w4a4_repack(codes, scales), N, K, experts)
    assert torch.equal(got[0], codes) and torch.equal(got[1], scales)


def test_a_weight_of_the_library_s_quantiser(dev):
    g = torch.Generator(device=dev).manual_seed(8)
    w = ffi.nvfp4_quantize(torch.randn((200, 512), generator=g, device=dev) * 0.02)
    x = draw(33, 512, 9, dev)
    want, off = ref.product(ref.values(x), ref.weight(*w))
    check(ffi.w4a4_gemm(ffi.w4a4_quantize(x), ffi.w4a4_repack(*w[:2]), w[2], 200), want, off)


# ------------------------------------------------------------------ products

SIZES = [(1, 256, 128), (1, 16, 1), (2, 272, 77), (15, 512, 128), (16, 512, 130), (17, 1024, 300),
         (31, 48, 257), (33, 4096, 64), (64, 1040, 128), (100, 5376, 513), (127, 256, 2000),
         (128, 2048, 20000), (8, 768, 40000), (128, 5120, 5120),
         # more than one tile of tokens, whole and partial ones, cut ones
         (129, 256, 16), (130, 16, 1), (144, 512, 256), (255, 272, 300), (256, 4096, 256),
         (257, 8192, 130), (300, 8208, 264), (333, 5376, 5376), (700, 10240, 1111),
         (1000, 1024, 1000), (2048, 2048, 2056), (1025, 16384, 3000), (513, 8992, 2432)]


SIZES += [(5, 17408, 130), (128, 8192, 264), (77, 65536, 48), (300, 65536, 48), (40, 21504, 5376)]
# pairs of blocks, from 129 rows and 153 tiles of 128 x 128 on: whole and partial tiles, and those
# of the last turn cut in 9, 4, 3 and 2 parts
PAIRS = [(300, 272, 13000), (257, 48, 13100), (1301, 1040, 1801), (2600, 528, 1030), (20000, 64, 130),
         (129, 256, 20000), (384, 5120, 6656), (1000, 8192, 5000), (1280, 16384, 5120),
         (4864, 18432, 1040), (1024, 18432, 5376), (1500, 16384, 4864)]
SIZES += PAIRS


@pytest.mark.parametrize("M,K,N", SIZES)
def test_gemm(dev, M, K, N):
    x, w = draw(M, K, M, dev), draw_weight(N, K, N, dev)
    ws = ffi.workspace(ffi.w4a4_gemm_workspace_bytes(M, N, K), dev)
    rows, packed = ffi.w4a4_quantize(x), ffi.w4a4_repack(*w[:2])
    y = ffi.w4a4_gemm(rows, packed, w[2], N, ws=ws)
    want, off = ref.product(ref.values(x), ref.weight(*w))
    check(y, want, off)
    assert ffi.nvfp4_workspace_status(ws) == 0
    # the workspace is left as it has to be, and the same call gives the same bits
    assert int(ws[256:256 + (128 << 10)].count_nonzero()) == 0
    assert torch.equal(ffi.w4a4_gemm(rows, packed, w[2], N, ws=ws), y)


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("M,H,I", [(1, 16, 16), (1, 5120, 512), (20, 272, 208), (48, 4096, 1024),
                                   (128, 512, 4000), (129, 256, 64), (200, 1040, 336),
                                   (600, 8192, 1040), (2000, 512, 1024), (128, 12288, 272),
                                   (300, 16384, 528), (1000, 8192, 2496), (700, 272, 2064),
                                   (10000, 256, 48), (1280, 16384, 2560)])
def test_gate_up(dev, M, H, I, kind):
    x, gate, up = draw(M, H, M, dev), draw_weight(I, H, 1, dev), draw_weight(I, H, 2, dev)
    packed = ffi.w4a4_repack_gate_up(*gate[:2], *up[:2])
    scale = 1e-3 / math.sqrt(H)  # values on both sides of the activation's bend
    h = ffi.w4a4_gate_up(ffi.w4a4_quantize(x), packed, scale, 2 * scale, I, kind)
    check_gated(h, kind, ref.values(x), ref.weight(*gate[:2], scale), ref.weight(*up[:2], 2 * scale))


def test_gated_products_that_are_ties_of_bf16(dev):
    """Large g: the sigmoid's loss decides a product that lies between two bf16 values, as long as
    64 bits have it; else the tie goes to even."""
    I, H = 16, 256
    codes = torch.zeros((I, H // 2), dtype=torch.uint8, device=dev)
    codes[:, 0] = 2  # weight 1 at element 0
    scales = torch.full((I, H // 16), 0x38, dtype=torch.uint8, device=dev)  # 1
    packed = ffi.w4a4_repack_gate_up(codes, scales, codes, scales)
    x = torch.zeros((10000, H), device=dev)
    x[:, 0] = 6.0
    few, many, pairs = [ffi.w4a4_quantize(x[:n].to(BF)) for n in (20, 300, 10000)]
    # g * u = 8 * 315, 16 * 323, 64 * 323, 128 * 315, 128 * 325: half a step from both neighbours
    for g, u, silu, gelu in ((20, 126, 2512, 2528), (34, 152, 5152, 5184), (34, -152, -5152, -5184),
                             (136, 152, 20736, 20736), (168, 240, 40448, 40448),
                             (200, 208, 41472, 41472)):
        for kind, want in ((0, silu), (1, gelu)):
            for rows in few, many, pairs:
                got = ffi.w4a4_gate_up(rows, packed, g / 6, u / 6, I, kind)
                assert bool((got == want).all()), (g, u, kind)


def test_wide_and_narrow_agree(dev):
    """The same rows through both kernels within the bound of either."""
    x, w = draw(6000, 1024, 1, dev), draw_weight(512, 1024, 2, dev)
    packed = ffi.w4a4_repack(*w[:2])
    many = ffi.w4a4_gemm(ffi.w4a4_quantize(x), packed, w[2], 512)
    few = ffi.w4a4_gemm(ffi.w4a4_quantize(x[:100].contiguous()), packed, w[2], 512)
    want, off = ref.product(ref.values(x), ref.weight(*w))
    check(many, want, off)
    check(few, want[:100], off[:100])


@pytest.mark.parametrize("M", [40, 300, 10000])
@pytest.mark.parametrize("N,shift", [(48, 0), (48, 8), (40, 0), (40, 8), (50, 0), (33, 8)])
def test_outputs_of_every_alignment(dev, M, N, shift):
    """Rows of 32-, 16- and 2-byte alignment, of a buffer that begins on 16 bytes; nothing beside
    the output is written."""
    x, w = draw(M, 256, 1, dev), draw_weight(N, 256, 2, dev)
    buf = torch.full((M * N + 64,), -7.0, dtype=BF, device=dev)
    out = buf[shift:shift + M * N].view(M, N)
    ffi.w4a4_gemm(ffi.w4a4_quantize(x), ffi.w4a4_repack(*w[:2]), w[2], N, out=out)
    want, off = ref.product(ref.values(x), ref.weight(*w))
    check(out, want, off)
    assert bool((buf[:shift] == -7).all()) and bool((buf[shift + M * N:] == -7).all())


# ------------------------------------------------------------------ the FFN

@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("M,H,I", [(1, 256, 512), (7, 16, 16), (65, 528, 1040), (128, 1024, 256),
                                   (300, 512, 2048), (1100, 256, 528), (5000, 528, 528),
                                   (1000, 5120, 2496)])
def test_ffn_is_its_parts(dev, M, H, I, kind):
    x = draw(M, H, M, dev)
    gate, up, down = draw_weight(I, H, 1, dev), draw_weight(I, H, 2, dev), draw_weight(H, I, 3, dev)
    gu, dn = ffi.w4a4_repack_gate_up(*gate[:2], *up[:2]), ffi.w4a4_repack(*down[:2])
    s = 1e-3 / math.sqrt(H)
    ws = ffi.workspace(ffi.ffn_swiglu_w4a4_workspace_bytes(M, H, I), dev)
    out = ffi.ffn_swiglu_w4a4(x, gu, s, s, dn, down[2], I, kind, ws=ws)
    h = ffi.w4a4_gate_up(ffi.w4a4_quantize(x), gu, s, s, I, kind)
    want = ffi.w4a4_gemm(ffi.w4a4_quantize(h), dn, down[2], H)
    assert torch.equal(out, want)
    exact, off = ref.product(ref.values(h), ref.weight(*down))
    check(out, exact, off)
    check_gated(h, kind, ref.values(x), ref.weight(*gate[:2], s), ref.weight(*up[:2], s))
    assert ffi.nvfp4_workspace_status(ws) == 0


# ------------------------------------------------------------------ by expert

def starts(lens, first, dev):
    at = [first]
    for n in lens:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32, device=dev)


LENS = [[3], [0, 5, 0], [1, 1, 1, 1], [128, 0, 129, 1], [300, 0, 0, 17, 256, 257], [0, 0, 700],
        [40] * 40, [1] * 130 + [500], [513, 255]]


@pytest.mark.parametrize("first,behind", [(0, 0), (3, 5)])
@pytest.mark.parametrize("lens", LENS)
def test_grouped_rows(dev, lens, first, behind):
    """Ragged shares, empty experts, rows of no expert in front and behind."""
    E, M, K, N = len(lens), first + sum(lens) + behind, 528, 272
    x, start = draw(M, K, M, dev), starts(lens, first, dev)
    rows = ffi.w4a4_quantize(x, start=start)
    end = first + sum(lens)
    got = ffi.w4a4_dequantize(rows)
    assert torch.equal(got[first:end].double(), ref.values(x[first:end]))
    assert bool((got[:first] == 0).all()) and bool((got[end:] == 0).all())
    w = draw_weight(N, K, 1, dev, E)
    y = torch.full((M, N), -7.0, dtype=BF, device=dev)
    ffi.w4a4_gemm(rows, ffi.w4a4_repack(*w[:2]), w[2], N, out=y)
    up = draw_weight(N, K, 2, dev, E)
    h = torch.full((M, N), -7.0, dtype=BF, device=dev)
    s = torch.full((E,), 1e-3 / math.sqrt(K), device=dev)
    ffi.w4a4_gate_up(rows, ffi.w4a4_repack_gate_up(*w[:2], *up[:2]), s, s, N, h=h)
    at = start.tolist()
    for e in range(E):
        mine = slice(at[e], at[e + 1])
        if lens[e]:
            v = ref.values(x[mine])
            check(y[mine], *ref.product(v, of_expert(w, e)))
            check_gated(h[mine], 0, v, of_expert((w[0], w[1], s), e), of_expert((up[0], up[1], s), e))
    for t in (y, h):  # rows of no expert are left as they were
        assert bool((t[:first] == -7).all()) and bool((t[end:] == -7).all())


@pytest.mark.parametrize("list_", [[0, 50, 20, 90], [0, 20, 5000, 90], [-3, 20, 40, 90],
                                   [0, 20, 40, 91], [90, 0, 0, 0], [0, 2 ** 31 - 1, 40, 90]])
def test_lists_that_do_not_fit(dev, list_):
    """Experts whose rows are not all inside take no part; what fits is right."""
    M, K, N = 90, 256, 64
    x, w = draw(M, K, 1, dev), draw_weight(N, K, 2, dev, 3)
    start = torch.tensor(list_, dtype=torch.int32, device=dev)
    rows = ffi.w4a4_quantize(x, start=start)
    y = torch.full((M + 2, N), -7.0, dtype=BF, device=dev)
    ffi.w4a4_gemm(rows, ffi.w4a4_repack(*w[:2]), w[2], N, out=y[1:M + 1])
    torch.cuda.synchronize()
    assert bool((y[0] == -7).all()) and bool((y[M + 1] == -7).all())
    ordered = all(0 <= a <= b <= M for a, b in zip(list_, list_[1:]))
    fit = [e for e in range(3) if 0 <= list_[e] < list_[e + 1] <= M]
    if ordered:
        assert fit
    if list_ == [0, 20, 40, 91]:
        for e in (0, 1):
            mine = slice(list_[e], list_[e + 1])
            check(y[1:M + 1][mine], *ref.product(ref.values(x[mine]), of_expert(w, e)))
        assert bool((y[41:M + 1] == -7).all())


def test_a_thousand_experts(dev):
    E, K, N = 1024, 256, 48
    g = torch.Generator().manual_seed(1)
    lens = torch.randint(0, 4, (E,), generator=g).tolist()
    lens[700] = 300
    M, start = sum(lens), starts(lens, 0, dev)
    x, w = draw(M, K, 1, dev), draw_weight(N, K, 2, dev, E)
    y = ffi.w4a4_gemm(ffi.w4a4_quantize(x, start=start), ffi.w4a4_repack(*w[:2]), w[2], N)
    v, at = ref.values(x), start.tolist()
    for e in range(E):
        if lens[e]:
            mine = slice(at[e], at[e + 1])
            check(y[mine], *ref.product(v[mine], of_expert(w, e)))


def test_rows_that_are_not_finite_by_expert(dev):
    x, E, I, H = draw(200, 256, 1, dev), 2, 64, 256
    x[3, 5], x[150, 7] = math.nan, math.inf
    gate, up = draw_weight(I, H, 2, dev, E), draw_weight(I, H, 3, dev, E)
    s = torch.full((E,), 1e-4, device=dev)
    rows = ffi.w4a4_quantize(x, start=starts([100, 100], 0, dev))
    h = ffi.w4a4_gate_up(rows, ffi.w4a4_repack_gate_up(*gate[:2], *up[:2]), s, s, I)
    assert bool(torch.isnan(h[[3, 150]]).all())
    fine = [r for r in range(200) if r not in (3, 150)]
    assert bool(torch.isfinite(h[fine]).all())


def test_offsets_beyond_32_bits(dev):
    """An output, an experts' weight and quantised rows of more than 2^32 bytes: their last rows."""
    M, K, N = 65600, 16, 33000
    x, w = draw(M, K, 1, dev), draw_weight(N, K, 2, dev)
    y = ffi.w4a4_gemm(ffi.w4a4_quantize(x), ffi.w4a4_repack(*w[:2]), w[2], N)
    for rows in (slice(0, 3), slice(M - 300, M)):
        check(y[rows], *ref.product(ref.values(x[rows]), ref.weight(*w)))
    del y
    E, K, N = 300, 16384, 2048
    codes = torch.zeros((E, N, K // 2), dtype=torch.uint8, device=dev)
    scales = torch.zeros((E, N, K // 16), dtype=torch.uint8, device=dev)
    last = draw_weight(N, K, 3, dev)
    codes[E - 1], scales[E - 1] = last[0], last[1]
    packed = ffi.w4a4_repack(codes, scales)
    assert packed.numel() > 2 ** 32
    del codes, scales
    x = draw(70, K, 4, dev)
    s = torch.full((E,), last[2], device=dev)
    start = torch.zeros(E + 1, dtype=torch.int32, device=dev)
    start[E] = 70  # all rows are the last expert's
    for n in (70, 70 * 600):  # both kernels
        x = draw(n, K, 4, dev)
        start[E] = n
        y = ffi.w4a4_gemm(ffi.w4a4_quantize(x, start=start), packed, s, N)
        check(y[-70:], *ref.product(ref.values(x[-70:]), ref.weight(*last)))
    del packed, y
    M, K = 150000, 65536  # 5.5 GB of tiles, 19.7 GB of x
    x = torch.zeros((M, K), dtype=BF, device=dev)
    x[-200:] = draw(200, K, 5, dev)
    rows = ffi.w4a4_quantize(x)
    assert rows.data.numel() > 2 ** 32
    w = draw_weight(32, K, 6, dev)
    y = ffi.w4a4_gemm(rows, ffi.w4a4_repack(*w[:2]), w[2], 32)
    check(y[-200:], *ref.product(ref.values(x[-200:]), ref.weight(*w)))
    assert bool((y[:-200] == 0).all())


@pytest.mark.parametrize("M", [100, 9000])
def test_a_list_that_decreases_leaves_every_row_out(dev, M):
    E, K, N = 64, 256, 64
    x, w = draw(M, K, 1, dev), draw_weight(N, K, 2, dev, E)
    start = torch.tensor([0, M] * (E // 2) + [0], dtype=torch.int32, device=dev)
    rows = ffi.w4a4_quantize(x, start=start)
    y = torch.full((M, N), -7.0, dtype=BF, device=dev)
    ffi.w4a4_gemm(rows, ffi.w4a4_repack(*w[:2]), w[2], N, out=y)
    assert bool((y == -7).all())


# ------------------------------------------------------------------ routing

def draw_ids(T, k, E, seed, dev, outside=True):
    g = torch.Generator(device=dev).manual_seed(seed)
    ids = torch.randint(-1 if outside else 0, E + (1 if outside else 0), (T, k), generator=g,
                        device=dev)
    return ids.int()


@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 8, 64), (3, 2, 5), (61, 8, 64), (333, 7, 33),
                                   (1, 64, 1024), (1000, 3, 1024), (4096, 1, 2), (24576, 1, 43),
                                   (3077, 8, 43), (4097, 6, 1024), (9001, 8, 200), (30000, 1, 1000)])
def test_order(dev, T, k, E):
    ids = draw_ids(T, k, E, T + k, dev)
    got = ffi.experts_order(ids, E)
    for a, b in zip(got, ref.order(ids.cpu(), E)):
        assert torch.equal(a.cpu(), b)


@pytest.mark.parametrize("T,k,E,value", [(50, 4, 8, -1), (50, 4, 8, 7), (5000, 8, 40, -1),
                                         (5000, 8, 40, 0), (5000, 8, 40, 39), (5000, 8, 40, 40)])
def test_order_of_one_value(dev, T, k, E, value):
    ids = torch.full((T, k), value, dtype=torch.int32, device=dev)
    for a, b in zip(ffi.experts_order(ids, E), ref.order(ids.cpu(), E)):
        assert torch.equal(a.cpu(), b)


def test_order_of_lists_that_begin_anywhere(dev):
    base = draw_ids(500, 3, 9, 1, dev).flatten()
    for shift in (1, 2, 3):
        ids = base[shift:shift + 300].view(100, 3)
        for a, b in zip(ffi.experts_order(ids, 9), ref.order(ids.cpu(), 9)):
            assert torch.equal(a.cpu(), b)


@pytest.mark.parametrize("T,k,H", [(1, 1, 16), (5, 8, 272), (64, 3, 4096), (700, 17, 528), (3, 64, 32)])
def test_sum(dev, T, k, H):
    rows = T * k
    y = draw(rows, H, T, dev)
    g = torch.Generator(device=dev).manual_seed(k)
    place = torch.randperm(rows, generator=g, device=dev).view(T, k).int()
    place[0, 0], place[T - 1, k - 1] = -1, rows  # outside
    w = torch.rand((T, k), generator=g, device=dev)
    w[0, 0] = math.nan  # whatever a weight of none is
    got = ffi.experts_sum(y, place, w)
    live = (place >= 0) & (place < rows)
    v = y.double()[place.clamp(0, rows - 1).long()] * torch.where(live, w.double(), 0.0)[..., None]
    # k products added in fp32, a fused one each
    check(got, v.sum(1), k * 2.0 ** -24 * v.abs().sum(1))


@pytest.mark.parametrize("k", [1, 4, 5, 9])
@pytest.mark.parametrize("T,H", [(9, 16), (40, 48), (17, 240), (5, 272), (3, 2000), (2, 2064),
                                 (2, 5376), (1, 65536)])
def test_sum_of_rows_of_any_length(dev, T, H, k):
    y = draw(T * k, H, T + k, dev)
    g = torch.Generator(device=dev).manual_seed(H)
    place = torch.randperm(T * k, generator=g, device=dev).view(T, k).int()
    w = torch.rand((T, k), generator=g, device=dev) - 0.5
    buf = torch.full((T * H + 64,), 7.0, dtype=BF, device=dev)
    ffi.experts_sum(y, place, w, out=buf[:T * H].view(T, H))
    v = y.double()[place.long()] * w.double()[..., None]
    check(buf[:T * H].view(T, H), v.sum(1), k * 2.0 ** -24 * v.abs().sum(1))
    assert bool((buf[T * H:] == 7.0).all())


def test_sum_with_the_same_row_twice(dev):
    y = draw(4, 64, 1, dev)
    place = torch.tensor([[2, 2], [0, 3]], dtype=torch.int32, device=dev)
    w = torch.tensor([[0.5, 0.25], [1.0, 0.0]], device=dev)
    got = ffi.experts_sum(y, place, w).double()
    check(got, torch.stack((0.75 * y[2].double(), y[0].double())), 0.0 * got)


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("T,k,E,H,I", [(1, 2, 4, 256, 128), (1, 8, 64, 512, 256), (33, 3, 5, 272, 144),
                                       (64, 8, 16, 1024, 512), (600, 4, 6, 512, 256),
                                       (1500, 2, 3, 256, 1040)])
def test_experts_ffn(dev, T, k, E, H, I, kind):
    x = draw(T, H, T, dev)
    ids = draw_ids(T, k, E, 2, dev)
    if T > 1:
        ids[T - 1] = -1  # a spare row of the batch
    weights = torch.rand((T, k), generator=torch.Generator(device=dev).manual_seed(3), device=dev)
    gate, up, down = [draw_weight(*s, i, dev, E) for i, s in enumerate(((I, H), (I, H), (H, I)))]
    gu, dn = ffi.w4a4_repack_gate_up(*gate[:2], *up[:2]), ffi.w4a4_repack(*down[:2])
    s = torch.full((E,), 1e-3 / math.sqrt(H), device=dev)
    ws = ffi.workspace(ffi.experts_swiglu_w4a4_workspace_bytes(T, k, E, H, I), dev)
    out = ffi.experts_swiglu_w4a4(x, ids, weights, gu, s, s, dn, down[2], I, kind, ws=ws)
    assert ffi.nvfp4_workspace_status(ws) == 0
    # the same by its parts
    start, source, place = ffi.experts_order(ids, E)
    rows = ffi.w4a4_quantize_routed(x, ids, place, start)
    h = torch.zeros((T * k, I), dtype=BF, device=dev)
    ffi.w4a4_gate_up(rows, gu, s, s, I, kind, h=h)
    y = torch.zeros((T * k, H), dtype=BF, device=dev)
    ffi.w4a4_gemm(ffi.w4a4_quantize(h, start=start), dn, down[2], H, out=y)
    assert torch.equal(out, ffi.experts_sum(y, place, weights))
    # and each part against its definition
    at, src = start.tolist(), source.long()
    live = at[-1]
    assert torch.equal(ffi.w4a4_dequantize(rows)[:live].double(), ref.values(x[src[:live]]))
    for e in range(E):
        mine = slice(at[e], at[e + 1])
        if at[e + 1] > at[e]:
            v = ref.values(x[src[mine]])
            check_gated(h[mine], kind, v, of_expert((gate[0], gate[1], s), e),
                        of_expert((up[0], up[1], s), e))
            check(y[mine], *ref.product(ref.values(h[mine]), of_expert(down, e)))
    if T > 1:
        assert bool((out[T - 1] == 0).all())


# ------------------------------------------------------------------ as programs call it

def test_captured_and_replayed_with_other_rows_and_lists(dev):
    T, k, E, H, I = 70, 2, 4, 256, 128
    gate, up, down = [draw_weight(*s, i, dev, E) for i, s in enumerate(((I, H), (I, H), (H, I)))]
    gu, dn = ffi.w4a4_repack_gate_up(*gate[:2], *up[:2]), ffi.w4a4_repack(*down[:2])
    s = torch.full((E,), 1e-4, device=dev)
    x, ids = draw(T, H, 1, dev), draw_ids(T, k, E, 1, dev)
    weights = torch.rand((T, k), device=dev)
    ws = ffi.workspace(ffi.experts_swiglu_w4a4_workspace_bytes(T, k, E, H, I), dev)
    out = torch.empty_like(x)
    dense = draw_weight(H, H, 9, dev)
    packed = ffi.w4a4_repack(*dense[:2])
    rows = ffi.W4a4Rows.empty(T, H, dev)
    dense_ws = ffi.workspace(ffi.w4a4_gemm_workspace_bytes(T, H, H), dev)
    dense_out = torch.empty_like(x)

    def step():
        ffi.experts_swiglu_w4a4(x, ids, weights, gu, s, s, dn, down[2], I, ws=ws, out=out)
        ffi.w4a4_quantize(out, out=rows)
        ffi.w4a4_gemm(rows, packed, dense[2], H, ws=dense_ws, out=dense_out)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (5, 6, 7):
        x.copy_(draw(T, H, seed, dev))
        ids.copy_(draw_ids(T, k, E, seed, dev))
        graph.replay()
        got = out.clone(), dense_out.clone()
        step()
        assert torch.equal(got[0], out) and torch.equal(got[1], dense_out)


def test_two_streams_with_their_own_workspaces(dev):
    M, K, N = 900, 8192, 1024
    w = draw_weight(N, K, 1, dev)
    packed = ffi.w4a4_repack(*w[:2])
    xs = [draw(M, K, s, dev) for s in (1, 2)]
    want = [ffi.w4a4_gemm(ffi.w4a4_quantize(x), packed, w[2], N) for x in xs]
    streams = [torch.cuda.Stream(dev) for _ in xs]
    kept = [(ffi.W4a4Rows.empty(M, K, dev), torch.empty((M, N), dtype=BF, device=dev),
             ffi.workspace(ffi.w4a4_gemm_workspace_bytes(M, N, K), dev)) for _ in xs]
    torch.cuda.synchronize()
    for _ in range(20):
        for x, st, (rows, out, ws) in zip(xs, streams, kept):
            with torch.cuda.stream(st):
                ffi.w4a4_quantize(x, out=rows)
                ffi.w4a4_gemm(rows, packed, w[2], N, ws=ws, out=out)
    torch.cuda.synchronize()
    for (_, out, ws), y in zip(kept, want):
        assert torch.equal(out, y)
        assert ffi.nvfp4_workspace_status(ws) == 0


def test_a_workspace_serves_any_sequence_of_calls(dev):
    shapes = [(700, 10240, 1111), (1, 5120, 300), (40, 1024, 30000), (129, 256, 64), (100, 5376, 513)]
    ws = ffi.workspace(max(ffi.w4a4_gemm_workspace_bytes(m, n, k) for m, k, n in shapes), dev)
    for M, K, N in shapes * 2:
        x, w = draw(M, K, M, dev), draw_weight(N, K, N, dev)
        rows, packed = ffi.w4a4_quantize(x), ffi.w4a4_repack(*w[:2])
        assert torch.equal(ffi.w4a4_gemm(rows, packed, w[2], N, ws=ws),
                           ffi.w4a4_gemm(rows, packed, w[2], N))


def test_refusals_that_need_a_device(dev):
    x, w = draw(200, 256, 1, dev), draw_weight(256, 256, 2, dev)
    rows, packed = ffi.w4a4_quantize(x), ffi.w4a4_repack(*w[:2])
    with pytest.raises(ffi.Nvfp4Error) as e:
        ffi.w4a4_gemm(rows, packed, w[2], 256, ws=torch.zeros(1024, dtype=torch.uint8, device=dev))
    assert e.value.code == 5
    ws = ffi.workspace(ffi.w4a4_gemm_workspace_bytes(200, 256, 256), dev)
    inside = ws[256:256 + 200 * 256 * 2].view(BF).view(200, 256)
    with pytest.raises(ffi.Nvfp4Error) as e:
        ffi.w4a4_gemm(rows, packed, w[2], 256, ws=ws, out=inside)
    assert e.value.code == 8
    gu = ffi.w4a4_repack_gate_up(*w[:2], *w[:2])
    ws = ffi.workspace(ffi.ffn_swiglu_w4a4_workspace_bytes(200, 256, 256), dev)
    with pytest.raises(ffi.Nvfp4Error) as e:
        ffi.ffn_swiglu_w4a4(x, gu, 1.0, 1.0, packed, 1.0, 256, ws=ws, out=x)
    assert e.value.code == 8
    with pytest.raises(ffi.Nvfp4Error) as e:
        ffi.ffn_swiglu_w4a4(x, gu, 1.0, 1.0, packed, 1.0, 256, ws=ws[:-256])
    assert e.value.code == 5
    for bad in (lambda: ffi.w4a4_gemm(rows, packed[:-1], w[2], 256),
                lambda: ffi.w4a4_gemm(rows, packed, w[2], 255 + 257),
                lambda: ffi.w4a4_gemm(rows, packed, w[2], 256, out=x[:100]),
                lambda: ffi.w4a4_quantize(x, out=ffi.W4a4Rows.empty(199, 256, dev)),
                lambda: ffi.w4a4_quantize(x.t())):
        with pytest.raises(ValueError):
            bad()
