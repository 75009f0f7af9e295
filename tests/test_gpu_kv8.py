"""The paged 8-bit cache and the attention over it against plain statements in 64 bits.

Error bounds, from the number formats.  A bf16 output is the rounding of a value within the bound.
E4M3 codes of an exactly known value have to be equal; a value computed in fp32 (a rotated one:
two products and a sum, 3 * 2^-24 of |a| + |b|) may fall on the other side of a tie, so a code may
be the neighbouring one where the exact quotient is that near to a tie.  Attention: a score is off
by at most (dim + 8) 2^-24 of sum |q_d k_d| scale =: d (fp32 sums of exact products), a weight by
2d and by its rounding to 11 bits, so the output by (2d + 2^-10) sum w |v| before its rounding; the
log-sum-exp by d + 2^-20 + keys 2^-24 (a sum of positive terms) + 2^-22 |lse|."""
import math

import pytest
import torch

import kv8_reference as ref
from nvfp4_weight_only_gb300 import ffi

pytestmark = pytest.mark.gpu

NAN_CODE = 0x7F


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ffi.load(build_if_missing=True)
    return torch.device("cuda:0")


def gen(seed):
    return torch.Generator().manual_seed(seed)


class Setup:
    """Sequences in a cache: CPU copies of everything, and the library's cache and batch on it.
    Rows that no sequence holds, and pages of nobody, hold NaN (codes and scales)."""

    def __init__(self, dev, q_lens, kv_lens, kv_heads, dim, page, seed=0, spare=2, width=None):
        g = gen(seed)
        need = [-(-k // page) for k in kv_lens]
        pages = sum(need) + spare
        order = torch.randperm(pages, generator=g)
        self.width = width or max(1, max(need))
        self.table = torch.full((len(kv_lens), self.width), pages - 1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.q_lens, self.kv_lens, self.page, self.dim = q_lens, kv_lens, page, dim
        shape = (pages, kv_heads, page, dim)
        self.codes = {n: torch.full(shape, NAN_CODE, dtype=torch.uint8) for n in "kv"}
        self.scales = {n: torch.full((pages, kv_heads), math.nan) for n in "kv"}
        for n in "kv":
            for b, kv in enumerate(kv_lens):
                for j in range(need[b]):
                    p, rows = int(self.table[b, j]), min(page, kv - j * page)
                    x = torch.randn((kv_heads, rows, dim), generator=g) * 100
                    self.codes[n][p, :, :rows] = ref.round_e4m3(x)
                    # any positive scale, powers of two or not
                    self.scales[n][p] = 2.0 ** (torch.rand(kv_heads, generator=g) * 4 - 9)
        self.dev = dev
        self.upload()

    def upload(self):
        d = self.dev
        self.cache = ffi.Kv8Cache(self.codes["k"].to(d), self.codes["v"].to(d),
                                  self.scales["k"].to(d), self.scales["v"].to(d))
        starts = [sum(self.q_lens[:b]) for b in range(len(self.q_lens) + 1)]
        self.tokens = starts[-1]
        self.batch = ffi.Kv8Batch(torch.tensor(starts, dtype=torch.int32, device=d),
                                  torch.tensor(self.kv_lens, dtype=torch.int32, device=d),
                                  self.table.to(d))

    def values(self, n):
        return ref.dequantise(self.codes[n], self.scales[n])


def draw_q(tokens, heads, dim, seed, scale=1.0):
    return (torch.randn((tokens, heads, dim), generator=gen(seed)) * scale).bfloat16()


def check_attention(s, q, out, lse, scale, window, sinks):
    want, want_lse, weight, reach = ref.attention(q, s.values("k"), s.values("v"), s.page, s.table,
                                                  s.q_lens, s.kv_lens, scale, window, sinks)
    d = (s.dim + 8) * 2.0 ** -24 * reach
    assert bool(ref.rounds_to(out, want, (2 * d[..., None] + 2.0 ** -10) * weight).all())
    empty = torch.isinf(want_lse)
    got = lse.cpu().double()
    assert bool((got[empty] == -math.inf).all()) and bool((out.cpu()[empty] == 0).all())
    limit = d + 2.0 ** -20 + max(s.kv_lens) * 2.0 ** -24 + 2.0 ** -22 * want_lse.abs()
    off = (got - want_lse).abs()
    assert bool((off[~empty] <= limit[~empty]).all())


def run_attention(s, q, scale, window=0, sinks=0, ws=None):
    lse = torch.empty(q.shape[:2], device=s.dev)
    out = ffi.kv8_attention(q.to(s.dev), s.cache, s.batch, scale, window, sinks, ws=ws, lse=lse)
    torch.cuda.synchronize()
    return out, lse


CASES = [
    # q_lens, kv_lens, heads, kv_heads, dim, page, window, sinks
    ([1], [1], 1, 1, 64, 16, 0, 0),
    ([1], [37], 8, 8, 128, 16, 0, 0),
    ([1], [300], 40, 8, 128, 64, 0, 0),
    ([1, 1, 1], [5, 129, 64], 16, 2, 128, 32, 0, 0),
    ([1, 0, 3, 1], [33, 70, 3, 16], 6, 2, 64, 16, 0, 0),
    ([0, 1], [0, 40], 4, 4, 128, 16, 0, 0),
    ([2, 5], [2, 100], 7, 1, 128, 64, 0, 0),
    ([1, 1], [257, 511], 5, 1, 256, 128, 0, 0),
    ([3], [200], 16, 1, 256, 256, 0, 0),
    ([4, 4], [190, 77], 12, 4, 64, 32, 0, 0),
    ([17], [150], 8, 1, 128, 64, 0, 0),
    ([33, 1], [33, 90], 3, 3, 128, 16, 0, 0),
    ([64], [201], 2, 1, 64, 64, 0, 0),
    # windows and first tokens that stay visible
    ([1], [100], 8, 2, 128, 16, 1, 0),
    ([1], [333], 8, 2, 128, 64, 50, 4),
    ([1, 1], [20, 400], 4, 4, 64, 32, 64, 3),
    ([6, 2], [180, 260], 6, 2, 128, 32, 7, 1),
    ([20], [170], 4, 1, 256, 16, 33, 40),
    ([70], [70], 2, 2, 128, 16, 16, 2),
    ([1], [90], 4, 4, 128, 64, 500, 4),
    ([2], [140], 8, 1, 64, 16, 20, 100),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x) for x in c).replace(" ", ""))
def test_attention(dev, case):
    q_lens, kv_lens, heads, kv_heads, dim, page, window, sinks = case
    s = Setup(dev, q_lens, kv_lens, kv_heads, dim, page, seed=len(str(case)))
    q = draw_q(s.tokens, heads, dim, 7)
    scale = 1.3 / math.sqrt(dim)
    out, lse = run_attention(s, q, scale, window, sinks)
    check_attention(s, q, out, lse, scale, window, sinks)
    assert ffi.kv8_batch_status(s.batch) == 0
    # the same bits again
    again, lse2 = run_attention(s, q, scale, window, sinks)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("q_lens,kv_lens,group,dim,window", [
    ([1], [9000], 8, 128, 0), ([1], [90001], 8, 128, 0), ([1, 2], [70000, 20011], 2, 64, 0),
    ([3], [70003], 1, 128, 30000), ([1] * 9, [700, 3, 1500, 90, 64, 65, 2048, 31, 1000], 4, 128, 0),
    ([40], [1400], 8, 128, 0), ([130], [600], 1, 64, 100), ([64, 7], [900, 1100], 16, 64, 0),
    ([35], [1000], 4, 256, 0), ([1] * 40, [64 * i + 1 for i in range(40)], 3, 128, 0),
    ([5], [40000], 8, 256, 0), ([64], [3000], 8, 128, 0), ([100, 3, 130], [700, 1200, 130], 4, 64, 0),
    ([300], [900], 2, 128, 77), ([16, 90], [2000, 95], 16, 64, 500), ([256], [257], 5, 128, 0),
    ([97], [4001], 1, 128, 0)])
def test_attention_on_longer_rows(dev, q_lens, kv_lens, group, dim, window):
    """Longer sequences than the loops of the plain statement serve, in fp64 tensor form."""
    s = Setup(dev, q_lens, kv_lens, 2, dim, 64, seed=11)
    q = draw_q(s.tokens, 2 * group, dim, 3, 2.0)
    scale = 1.0 / math.sqrt(dim)
    out, lse = run_attention(s, q, scale, window, 2)
    t0 = 0
    for b, (n, kv) in enumerate(zip(q_lens, kv_lens)):
        rows = s.table[b, :-(-kv // 64)].long()
        k, v = (s.values(x)[rows].transpose(1, 2).flatten(0, 1)[:kv] for x in "kv")
        p = torch.arange(kv - n, kv)[:, None]
        at = torch.arange(kv)[None]
        seen = at <= p
        if window:
            seen &= (at > p - window) | (at < 2)
        for h in range(2 * group):
            x = q[t0:t0 + n, h].double()
            sc = (x @ k[:, h // group].T) * scale
            d = (dim + 8) * 2.0 ** -24 * (x.abs() @ k[:, h // group].abs().T).amax(1) * scale
            sc = sc.masked_fill(~seen, -math.inf)
            want_lse = torch.logsumexp(sc, 1)
            w = torch.exp(sc - want_lse[:, None])
            want, weight = w @ v[:, h // group], w @ v[:, h // group].abs()
            bound = (2 * d[:, None] + 2.0 ** -10) * weight
            assert bool(ref.rounds_to(out[t0:t0 + n, h], want, bound).all())
            off = (lse[t0:t0 + n, h].cpu().double() - want_lse).abs()
            assert bool((off <= d + 2.0 ** -20 + kv * 2.0 ** -24
                         + 2.0 ** -22 * want_lse.abs()).all())
        t0 += n


def test_attention_strided_q_and_other_stream(dev):
    s = Setup(dev, [1, 3], [50, 80], 2, 128, 16)
    fused = torch.randn((4, 8 + 4, 128), generator=gen(2)).bfloat16().to(dev)
    q = fused[:, :8]
    assert not q.is_contiguous()
    want = ffi.kv8_attention(q.contiguous(), s.cache, s.batch, 0.1)
    side = torch.cuda.Stream(dev)
    ws = ffi.workspace(ffi.kv8_attention_workspace_bytes(s.cache, s.batch, 4, 8), dev)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        got = ffi.kv8_attention(q, s.cache, s.batch, 0.1, ws=ws)
    side.synchronize()
    assert torch.equal(got, want)


def test_attention_in_a_graph_follows_the_lengths(dev):
    """Lengths live on the device: a captured call serves the next step."""
    s = Setup(dev, [1, 1], [64, 200], 4, 128, 32, width=9)
    q = draw_q(2, 16, 128, 5).to(dev)
    out = torch.empty_like(q)
    ws = ffi.workspace(ffi.kv8_attention_workspace_bytes(s.cache, s.batch, 2, 16), dev)
    ffi.kv8_attention(q, s.cache, s.batch, 0.1, ws=ws, out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ffi.kv8_attention(q, s.cache, s.batch, 0.1, ws=ws, out=out)
    for lens in ([64, 200], [1, 150], [33, 7]):
        s.batch.kv_len.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        want = ffi.kv8_attention(q, s.cache, s.batch, 0.1)
        assert torch.equal(out, want)


def test_workspace_serves_any_sequence_of_shapes(dev):
    big = Setup(dev, [1], [5000], 8, 128, 64, seed=1)
    small = Setup(dev, [1, 2, 30], [9, 40, 700], 1, 128, 16, seed=2)
    qb, qs = draw_q(1, 64, 128, 1).to(dev), draw_q(33, 4, 128, 2).to(dev)
    ws = ffi.workspace(max(ffi.kv8_attention_workspace_bytes(big.cache, big.batch, 1, 64),
                           ffi.kv8_attention_workspace_bytes(small.cache, small.batch, 33, 4)), dev)
    want_b = ffi.kv8_attention(qb, big.cache, big.batch, 0.1)
    want_s = ffi.kv8_attention(qs, small.cache, small.batch, 0.1)
    for _ in range(3):
        assert torch.equal(ffi.kv8_attention(qb, big.cache, big.batch, 0.1, ws=ws), want_b)
        assert torch.equal(ffi.kv8_attention(qs, small.cache, small.batch, 0.1, ws=ws), want_s)


@pytest.mark.parametrize("n,kv,window,dim", [(9, 60, 11, 128), (9, 60, 11, 64), (9, 60, 11, 256),
                                             (40, 300, 90, 128), (64, 200, 100, 64)])
def test_masked_values_do_not_enter(dev, n, kv, window, dim):
    """NaN in a later token's k and v, and in tokens that the window has left behind, changes no
    query that does not see them (stale rows hold NaN in every test here)."""
    page = 16
    s = Setup(dev, [n], [kv], 2, dim, page)
    q = draw_q(n, 8, dim, 4)
    for name in "kv":
        for j in list(range(0, kv - n + 1 - window)) + [kv - 1, kv - 4]:
            s.codes[name][int(s.table[0, j // page]), :, j % page] = NAN_CODE
    s.upload()
    out, _ = run_attention(s, q, 0.1, window)
    assert not torch.isnan(out[:n - 4].float()).any()
    assert torch.isnan(out[n - 4:].float()).all()
    clean = {x: s.codes[x].clone() for x in "kv"}
    for name in "kv":
        s.codes[name] = torch.where(s.codes[name] == NAN_CODE, 0, s.codes[name])
    s.upload()
    want, lse = run_attention(s, q, 0.1, window)
    assert torch.equal(out[:n - 4], want[:n - 4])
    s.codes = clean


@pytest.mark.parametrize("n,dim", [(2, 64), (2, 128), (60, 64), (60, 128)])
def test_one_value_code_nan_spoils_only_its_column(dev, n, dim):
    kv = n + 28
    s = Setup(dev, [n], [kv], 1, dim, 16)
    for j, d in ((kv - 1, 5), (kv - 2, 33)):
        s.codes["v"][int(s.table[0, j // 16]), 0, j % 16, d] = NAN_CODE
    s.upload()
    out, _ = run_attention(s, draw_q(n, 4, dim, 9), 0.1)
    bad = torch.isnan(out.float())
    assert not bad[:n - 2].any()
    assert bad[n - 2, :, 33].all() and bad[n - 2].sum() == 4
    assert bad[n - 1, :, [5, 33]].all() and bad[n - 1].sum() == 8


def test_large_scores_and_values(dev):
    """Scores over thousands, q up to the top of bf16's practical range, page scales 2^24 apart."""
    s = Setup(dev, [1], [100], 1, 128, 16, seed=5)
    for i in range(7):
        s.scales["v"][int(s.table[0, i])] = 2.0 ** (4 * i - 12)
        s.scales["k"][int(s.table[0, i])] = 2.0 ** (-i)
    s.upload()
    q = draw_q(1, 8, 128, 3, 1.0)
    q[0, 3] *= 1e4
    q[0, 4] *= 2.0 ** 60
    q[0, 5] *= 2.0 ** -100
    scale = torch.tensor([1.0])
    out, lse = run_attention(s, q, float(scale))
    keep = [0, 1, 2, 3, 5, 6, 7]
    want, want_lse, weight, reach = ref.attention(q, s.values("k"), s.values("v"), 16, s.table,
                                                  [1], [100], 1.0)
    d = (128 + 8) * 2.0 ** -24 * reach
    err = (out.cpu().double() - want).abs()
    # differences of scores this large are off by d, so weights by a factor e^(2d)
    bound = (torch.expm1(2 * d)[..., None] + 2.0 ** -10) * weight
    assert bool(ref.rounds_to(out, want, bound)[0, keep].all())
    # the largest score takes all the weight at 2^60
    assert bool((err[0, 4] <= 2.0 ** -8 * want[0, 4].abs() + 1e-30).all())


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("window,marks", [
    (0, [(10, 3), (551, 1), (600, -1), (639, 40), (640, 32), (699, 7)]),
    (200, [(360, 2), (400, 35), (511, 0), (512, -1), (575, 20)])])
def test_value_nans_of_many_rows_reach_the_rows_that_see_them(dev, dim, window, marks):
    """150 tokens of 4 heads per kv head: several units of two row tiles, cut into parts."""
    n, kv, page = 150, 700, 32
    s = Setup(dev, [n], [kv], 2, dim, page, seed=21)
    want = torch.zeros((n, dim), dtype=torch.bool)
    p = torch.arange(kv - n, kv)
    for j, d in marks:
        s.codes["v"][int(s.table[0, j // page]), 1, j % page, d] = NAN_CODE
        want[(j <= p) & ((j > p - window) if window else True), d] = True
    s.upload()
    out, lse = run_attention(s, draw_q(n, 8, dim, 5), 0.02, window)
    bad = torch.isnan(out.cpu().float())
    assert not bad[:, :4].any()
    assert torch.equal(bad[:, 4:], want[:, None].expand(n, 4, dim))
    assert not torch.isnan(lse).any()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("rising", [True, False])
@pytest.mark.parametrize("n", [1, 40])
def test_largest_score_moves_from_tile_to_tile(dev, dim, rising, n):
    """Keys' scales that rise (or fall) by 2^0.75 from page to page, values' that jump by 2^10:
    scores to over a thousand, a new maximum in nearly every tile."""
    kv, heads = 1000, 8
    s = Setup(dev, [n], [kv], 1, dim, 64, seed=23)
    for i in range(16):
        at = int(s.table[0, i])
        s.scales["k"][at] = 2.0 ** (0.75 * (i if rising else 15 - i) - 9)
        s.scales["v"][at] *= 2.0 ** (10 * (i % 3))
    s.upload()
    q = draw_q(n, heads, dim, 6)
    scale = 1.0 / math.sqrt(dim)
    out, lse = run_attention(s, q, scale)
    rows = s.table[0].long()
    k, v = (s.values(x)[rows, 0].flatten(0, 1)[:kv] for x in "kv")
    hidden = torch.arange(kv)[None] > torch.arange(kv - n, kv)[:, None]
    for h in range(heads):
        x = q[:, h].double()
        sc = (x @ k.T) * scale
        d = (dim + 8) * 2.0 ** -24 * (x.abs() @ k.abs().T).masked_fill(hidden, 0).amax(1) * scale
        sc = sc.masked_fill(hidden, -math.inf)
        want_lse = torch.logsumexp(sc, 1)
        w = torch.exp(sc - want_lse[:, None])
        # scores this large are off by d, so weights by a factor e^(2d)
        bound = (torch.expm1(2 * d)[:, None] + 2.0 ** -10) * (w @ v.abs())
        assert bool(ref.rounds_to(out[:, h], w @ v, bound).all())
        off = (lse[:, h].cpu().double() - want_lse).abs()
        assert bool((off <= d + 2.0 ** -20 + kv * 2.0 ** -24 + 2.0 ** -22 * want_lse.abs()).all())


@pytest.mark.parametrize("q_lens,kv_lens,heads,kv_heads,dim", [
    ([8, 8], [500, 700], 8, 2, 128),        # 32 rows each: one pass
    ([9, 8], [500, 700], 8, 2, 128),        # one row more on average
    ([33, 0], [400, 90], 4, 4, 64),         # an empty sequence in the average
    ([1] * 9 + [300], [50] * 9 + [310], 3, 1, 128),  # single tokens beside a prompt
    ([1] * 9 + [300], [50] * 9 + [310], 3, 1, 64),
    ([1] * 9, [2000 + i for i in range(9)], 40, 8, 128),  # 72 units, 76 the most that count as few
    ([1] * 10, [2000 + i for i in range(10)], 40, 8, 128),
    ([2] * 3, [1500, 1, 2], 24, 8, 128)])
def test_attention_around_the_rules(dev, q_lens, kv_lens, heads, kv_heads, dim):
    """Sizes on both sides of where one kernel or way of cutting gives way to another."""
    q_lens = [min(n, kv) for n, kv in zip(q_lens, kv_lens)]
    s = Setup(dev, q_lens, kv_lens, kv_heads, dim, 64, seed=29)
    q = draw_q(s.tokens, heads, dim, 8)
    scale = 1.0 / math.sqrt(dim)
    out, lse = run_attention(s, q, scale)
    check_attention(s, q, out, lse, scale, 0, 0)


def test_long_cache_offsets(dev):
    """Pages whose codes lie beyond 2^32 bytes and 2^31 rows of the buffers."""
    pages, kv_heads, page, dim = 33000, 8, 128, 128
    k = torch.zeros((pages, kv_heads, page, dim), dtype=torch.uint8, device=dev)
    v = torch.zeros_like(k)
    ks = torch.ones((pages, kv_heads), device=dev)
    vs = torch.ones_like(ks)
    cache = ffi.Kv8Cache(k, v, ks, vs)
    table = torch.tensor([[pages - 1, 2, pages - 2]], dtype=torch.int32, device=dev)
    batch = ffi.Kv8Batch(torch.tensor([0, 300], dtype=torch.int32, device=dev),
                         torch.tensor([300], dtype=torch.int32, device=dev), table)
    x = torch.randn((300, 2 * kv_heads, dim), generator=gen(1)).bfloat16().to(dev)
    ffi.kv8_append(cache, batch, x[:, :kv_heads], x[:, kv_heads:])
    small = ffi.Kv8Cache.empty(3, kv_heads, page, dim, dev)
    table2 = torch.tensor([[0, 1, 2]], dtype=torch.int32, device=dev)
    batch2 = ffi.Kv8Batch(batch.q_start, batch.kv_len, table2)
    ffi.kv8_append(small, batch2, x[:, :kv_heads], x[:, kv_heads:])
    q = draw_q(300, 16, dim, 6).to(dev)
    assert torch.equal(ffi.kv8_attention(q, cache, batch, 0.1),
                       ffi.kv8_attention(q, small, batch2, 0.1))
    a, b = [torch.empty((300, kv_heads, dim), dtype=torch.bfloat16, device=dev) for _ in "kv"]
    c, d = torch.empty_like(a), torch.empty_like(a)
    ffi.kv8_read(cache, batch, a, b)
    ffi.kv8_read(small, batch2, c, d)
    assert torch.equal(a, c) and torch.equal(b, d)


# ------------------------------------------------------------------------------ append and read

def rotation(dev, positions, rot):
    return ffi.rope_table(positions, rot, 10000.0, dev) if rot else None


def near_a_tie(x, scale, dim_error):
    """Where x / scale lies within dim_error / scale of a midpoint of two E4M3 values."""
    v = (x / scale).abs().clamp(max=448.0)
    step = torch.exp2(torch.floor(torch.log2(v.clamp(min=2.0 ** -6))) - 3)
    frac = v / step - torch.floor(v / step)
    return (frac - 0.5).abs() * step <= dim_error / scale


@pytest.mark.parametrize("q_lens,kv_lens,heads,kv_heads,dim,page,rot,inter", [
    ([1], [1], 1, 1, 64, 16, 0, False),
    ([1], [100], 8, 8, 128, 64, 128, False),
    ([1, 1, 1], [16, 17, 32], 6, 2, 128, 16, 64, True),
    ([3, 0, 20], [3, 50, 45], 4, 4, 64, 16, 64, False),
    ([40, 1], [90, 33], 2, 1, 256, 32, 128, True),
    ([130], [300], 3, 3, 128, 128, 48, False),
    ([70], [70], 16, 1, 128, 256, 16, True),
    ([5], [260], 2, 2, 256, 256, 256, False),
])
def test_append_and_read(dev, q_lens, kv_lens, heads, kv_heads, dim, page, rot, inter):
    s = Setup(dev, q_lens, kv_lens, kv_heads, dim, page, seed=3)
    # what the cache holds before: scales of powers of two, small enough that some have to grow
    g = gen(8)
    for n in "kv":
        s.scales[n] = 2.0 ** torch.randint(-9, -5, s.scales[n].shape, generator=g).float()
    s.upload()
    fused = torch.randn((s.tokens, heads + 2 * kv_heads, dim), generator=g)
    fused *= torch.exp(torch.randn((s.tokens, 1, 1), generator=g))
    fused = fused.bfloat16()
    fused[0, heads + 2 * kv_heads - 1, :3] = torch.tensor([3.5, -0.0, 0.0])
    on = fused.to(dev)
    q, k, v = on.split((heads, kv_heads, kv_heads), 1)
    rope = rotation(dev, max(kv_lens), rot)
    before = {n: s.codes[n].clone() for n in "kv"}
    q_out = ffi.kv8_append(s.cache, s.batch, k, v, q=q, rope=rope, interleaved=inter)
    torch.cuda.synchronize()
    assert ffi.kv8_batch_status(s.batch) == 0
    positions = [kv - n + i for n, kv in zip(q_lens, kv_lens) for i in range(n)]
    hq, hk, hv = (x.double() for x in fused.split((heads, kv_heads, kv_heads), 1))
    table = rope.cpu() if rot else torch.zeros((1, 0, 2))
    hq = ref.rotate(hq, table, positions, inter)
    hk = ref.rotate(hk, table, positions, inter)
    size = fused.double().abs().amax()
    assert bool(ref.rounds_to(q_out, hq, 6 * 2.0 ** -24 * size).all())
    got = {"k": (s.cache.k_codes.cpu(), s.cache.k_scales.cpu()),
           "v": (s.cache.v_codes.cpu(), s.cache.v_scales.cpu())}
    for n, x in (("k", hk), ("v", hv)):
        codes, scales = s.codes[n], s.scales[n]
        ref.append(codes, scales, page, x, q_lens, kv_lens, s.table)
        assert torch.equal(got[n][1], scales)
        if n == "v" or not rot:
            assert torch.equal(got[n][0], codes)
            continue
        # where fp32's rounding can cross a tie, the neighbouring code
        differ = got[n][0] != codes
        assert differ.sum() <= 4 + 1e-4 * differ.numel()
        a, b = ref.e4m3_value(got[n][0]), ref.e4m3_value(codes)
        t = 0
        allowed = torch.zeros_like(differ)
        for b_, (m, kv) in enumerate(zip(q_lens, kv_lens)):
            for i in range(m):
                p = kv - m + i
                pg = int(s.table[b_, p // page])
                allowed[pg, :, p % page] = near_a_tie(x[t], scales[pg][:, None].double(),
                                                      3 * 2.0 ** -24 * 2 * size)
                t += 1
        assert bool((differ <= allowed).all())
        nan = torch.isnan(a)
        assert torch.equal(nan, torch.isnan(b))
    assert not all(torch.equal(before[n], got[n][0]) for n in "kv")
    # read back
    ko = torch.empty((s.tokens, kv_heads, dim), dtype=torch.bfloat16, device=dev)
    vo = torch.empty_like(ko)
    ffi.kv8_read(s.cache, s.batch, ko, vo)
    torch.cuda.synchronize()
    t = 0
    for b, (m, kv) in enumerate(zip(q_lens, kv_lens)):
        for i in range(m):
            p = kv - m + i
            pg = int(s.table[b, p // page])
            for o, n in ((ko, "k"), (vo, "v")):
                want = ref.e4m3_value(got[n][0][pg, :, p % page]) * got[n][1][pg].double()[:, None]
                assert torch.equal(o[t].cpu(), want.float().bfloat16())
            t += 1


def test_append_special_values(dev):
    """NaN is kept and does not enter the scale; infinities saturate; zeros get the least scale."""
    s = Setup(dev, [3], [3], 1, 64, 16)
    k = torch.zeros((3, 1, 64)).bfloat16()
    v = torch.zeros_like(k)
    k[0, 0, 0], k[1, 0, 1] = math.nan, 2.0
    v[0, 0, 0], v[1, 0, 3], v[2, 0, 5] = math.inf, -math.inf, 1.0
    ffi.kv8_append(s.cache, s.batch, k.to(dev), v.to(dev))
    p = int(s.table[0, 0])
    assert float(s.cache.k_scales[p, 0]) == 2.0 ** -7  # 2 <= 448 * 2^-7 = 3.5
    assert int(s.cache.k_codes[p, 0, 0, 0]) & 0x7F == 0x7F
    assert float(s.cache.v_scales[p, 0]) == 2.0 ** 119
    assert s.cache.v_codes[p, 0, :3].cpu().view(ref.E4M3).float()[0, 0] == 448
    assert s.cache.v_codes[p, 0, :3].cpu().view(ref.E4M3).float()[1, 3] == -448
    z = Setup(dev, [1], [1], 1, 64, 16)
    zero = torch.zeros((1, 1, 64), dtype=torch.bfloat16, device=dev)
    ffi.kv8_append(z.cache, z.batch, zero, zero)
    p = int(z.table[0, 0])
    assert float(z.cache.k_scales[p, 0]) == 2.0 ** -60
    assert int(z.cache.k_codes[p, 0, 0].max()) == 0


def test_append_token_by_token_grows_the_scale(dev):
    """Decoding into one page: each step's cache equals the plain statement's."""
    s = Setup(dev, [1], [1], 2, 128, 16, width=3)
    g = gen(4)
    for n in "kv":
        s.codes[n].fill_(NAN_CODE)
        s.scales[n].fill_(math.nan)
    s.upload()
    for step in range(1, 37):
        x = (torch.randn((1, 4, 128), generator=g) * 2.0 ** (step % 5)).bfloat16()
        s.batch.kv_len.fill_(step)
        s.batch.page_table.copy_(torch.tensor([[2, 0, 1]], dtype=torch.int32))
        on = x.to(dev)
        ffi.kv8_append(s.cache, s.batch, on[:, :2], on[:, 2:])
        for n, part in (("k", x[:, :2]), ("v", x[:, 2:])):
            ref.append(s.codes[n], s.scales[n], 16, part.double(), [1], [step],
                       torch.tensor([[2, 0, 1]]))
        assert torch.equal(s.cache.k_codes.cpu(), s.codes["k"])
        assert torch.equal(s.cache.v_codes.cpu(), s.codes["v"])
        used = ~torch.isnan(s.scales["k"])
        assert torch.equal(s.cache.k_scales.cpu()[used], s.scales["k"][used])


def test_append_q_in_place_and_without_q(dev):
    s = Setup(dev, [2], [9], 1, 64, 16)
    rope = ffi.rope_table(9, 64, 10000.0, dev)
    k = draw_q(2, 1, 64, 1).to(dev)
    q = draw_q(2, 3, 64, 2).to(dev)
    want = ffi.kv8_append(s.cache, s.batch, k, k, q=q, rope=rope)
    first = s.cache.k_codes.clone()
    assert ffi.kv8_append(s.cache, s.batch, k, k, rope=rope) is None
    assert torch.equal(first, s.cache.k_codes)
    ffi.kv8_append(s.cache, s.batch, k, k, q=q, q_out=q, rope=rope)
    assert torch.equal(q, want)


@pytest.mark.parametrize("scaling,kw", [
    (0, {}), (1, dict(factor=8.0)), (2, dict(factor=4.0)),
    (3, dict(factor=16.0, context=4096.0, slow=1.0, fast=32.0, magnitude=1.2)),
    (3, dict(factor=8.0, context=8192.0, slow=1.0, fast=4.0))])
@pytest.mark.parametrize("rot", [16, 64, 128])
def test_rope_table(dev, scaling, kw, rot):
    positions, base = 5000, 500000.0
    got = ffi.rope_table(positions, rot, base, dev, scaling=scaling, **kw).cpu().double()
    magnitude = kw.pop("magnitude", 1.0)
    f = torch.tensor(ref.rope_frequencies(rot, base, scaling, **kw), dtype=torch.float64)
    a = torch.arange(positions, dtype=torch.float64)[:, None] * f
    want = torch.stack((a.cos(), a.sin()), -1) * magnitude
    # fp32 rounding, and an angle of up to 5000 from frequencies a few fp64 ulps apart
    assert bool(((got - want).abs() <= 2.0 ** -24 * want.abs() + 1e-11).all())


# ------------------------------------------------------------------------------ indexes out of range

def test_bad_indexes_are_masked_and_reported(dev):
    """Pages outside the cache, lengths beyond the table, more new tokens than the length and
    positions beyond the rotation table: checked in the kernels, nothing outside is touched."""
    s = Setup(dev, [1, 1], [40, 40], 2, 64, 16)
    q = draw_q(2, 4, 64, 1)
    good, _ = run_attention(s, q, 0.1)
    table = s.table.clone()
    for bad in (-1, s.cache.pages, 2 ** 31 - 1):
        s.batch.page_table[1, 1] = bad
        out, lse = run_attention(s, q, 0.1)
        assert ffi.kv8_batch_status(s.batch) == 4
        assert ffi.kv8_batch_status(s.batch) == 0
        assert torch.equal(out[0], good[0])
        # sequence 1 without the tokens 16..31 of its second page
        cut = Setup(dev, [1, 1], [40, 24], 2, 64, 16)
        cut.codes, cut.scales = s.codes, s.scales
        cut.table = torch.tensor([[0, 0], [int(table[1, 0]), int(table[1, 2])]], dtype=torch.int32)
        cut.upload()
        want, _ = run_attention(cut, q, 0.1)
        assert float((out[1].float() - want[1].float()).abs().max()) < 2 ** -6
        k = draw_q(2, 2, 64, 3).to(dev)
        s.batch.kv_len.copy_(torch.tensor([40, 20], dtype=torch.int32))
        before = s.cache.k_codes.clone()
        ffi.kv8_append(s.cache, s.batch, k, k)
        assert ffi.kv8_batch_status(s.batch) == 4
        after = s.cache.k_codes.clone()
        changed = (before != after).flatten(1).any(1).nonzero().flatten().tolist()
        assert changed in ([], [int(table[0, 2])])
        s.upload()
    s.batch.kv_len.copy_(torch.tensor([10 ** 9, 0], dtype=torch.int32))
    run_attention(s, q, 0.1)
    assert ffi.kv8_batch_status(s.batch) == 4
    s.batch.kv_len.copy_(torch.tensor([40, 40], dtype=torch.int32))
    s.batch.q_start.copy_(torch.tensor([0, 50, -7], dtype=torch.int32))
    run_attention(s, q, 0.1)
    assert ffi.kv8_batch_status(s.batch) == 4
    s.upload()
    rope = ffi.rope_table(8, 64, 10000.0, dev)
    k = draw_q(2, 2, 64, 3).to(dev)
    ffi.kv8_append(s.cache, s.batch, k, k, q=q.to(dev), rope=rope)
    assert ffi.kv8_batch_status(s.batch) == 4


def test_more_new_tokens_than_the_length(dev):
    """Tokens in front of position 0 are left out: not written, and they see nothing."""
    s = Setup(dev, [4], [2], 1, 64, 16)
    k = draw_q(4, 1, 64, 1).to(dev)
    ffi.kv8_append(s.cache, s.batch, k, k)
    q = draw_q(4, 2, 64, 2)
    out, lse = run_attention(s, q, 0.1)
    assert ffi.kv8_batch_status(s.batch) == 4
    assert bool((out[:2] == 0).all()) and bool((lse[:2] == -math.inf).all())
    assert bool(torch.isfinite(lse[2:]).all())
    only = Setup(dev, [2], [2], 1, 64, 16)
    ffi.kv8_append(only.cache, only.batch, k[2:], k[2:])
    want, _ = run_attention(only, q[2:], 0.1)
    assert torch.equal(out[2:], want)
