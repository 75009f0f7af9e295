"""The paged cache at sizes that test_gpu_kv8.py does not reach: batches of hundreds of sequences,
long runs in batches that are short on average, and pages beyond 2^32 bytes compared one by one.
Tolerances are those of test_gpu_kv8.py."""
import math

import pytest
import torch

import test_gpu_kv8 as base
from nvfp4_weight_only_gb300 import ffi

pytestmark = pytest.mark.gpu

NAN_CODE = 0x7F


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ffi.load(build_if_missing=True)
    return torch.device("cuda:0")


def lens(n, most, seed):
    return [int(x) for x in torch.randint(0, most + 1, (n,),
                                          generator=torch.Generator().manual_seed(seed))]


@pytest.mark.parametrize("q_lens,kv_lens,heads,kv_heads,dim,page,rot,inter", [
    # one prompt among single tokens: a warp takes each run, of more rows than it holds
    ([100] + [1] * 9, [230] + [40] * 9, 4, 2, 128, 64, 128, False),
    ([100] + [1] * 9, [230] + [40] * 9, 3, 1, 256, 128, 64, True),
    ([1] * 9 + [110], [33] * 9 + [111], 2, 2, 64, 256, 64, True),
    ([90, 1, 1, 1, 1, 1], [100, 5, 17, 16, 1, 64], 2, 1, 256, 64, 256, False),
    # hundreds of sequences
    ([1] * 300, [1 + i % 50 for i in range(300)], 2, 1, 64, 16, 64, False),
    ([1 - (i % 7 == 3) for i in range(1024)], [1 + i % 20 for i in range(1024)], 1, 1, 64, 16, 32,
     True),
    ([17] * 65, [17 + i for i in range(65)], 2, 1, 64, 32, 64, False)])
def test_append_and_read(dev, q_lens, kv_lens, heads, kv_heads, dim, page, rot, inter):
    base.test_append_and_read(dev, q_lens, kv_lens, heads, kv_heads, dim, page, rot, inter)


@pytest.mark.parametrize("sequences,new,most_kv,heads,kv_heads,dim,window", [
    (65, 1, 300, 8, 1, 128, 0), (300, 1, 60, 4, 2, 64, 0), (1024, 1, 40, 4, 1, 128, 0),
    (1024, 1, 40, 2, 1, 256, 9), (300, 12, 60, 8, 2, 64, 0), (257, 20, 90, 4, 2, 128, 30)])
def test_attention_of_many_sequences(dev, sequences, new, most_kv, heads, kv_heads, dim, window):
    q_lens = [new] * sequences if new == 1 else [max(1, n) for n in lens(sequences, 2 * new, 1)]
    kv_lens = [n + k for n, k in zip(q_lens, lens(sequences, most_kv, 2))]
    q_lens[7] = 0
    s = base.Setup(dev, q_lens, kv_lens, kv_heads, dim, 16, seed=51)
    q = base.draw_q(s.tokens, heads, dim, 52)
    scale = 1.0 / math.sqrt(dim)
    out, lse = base.run_attention(s, q, scale, window, 2)
    base.check_attention(s, q, out, lse, scale, window, 2)
    assert ffi.kv8_batch_status(s.batch) == 0


@pytest.mark.parametrize("new", [1, 300])
def test_pages_beyond_32_bits_are_the_ones_written_and_read(dev, new):
    """Pages whose codes begin beyond 2^32 bytes, compared with a small cache's one by one; the pages
    that a 32-bit offset would reach instead hold NaN."""
    pages, kv_heads, page, dim = 33000, 8, 128, 128
    bytes_of_one = kv_heads * page * dim
    used = [pages - 1, 2, pages - 2]
    lower = [p - 2 ** 32 // bytes_of_one for p in used if p * bytes_of_one >= 2 ** 32]
    assert len(lower) == 2 and not set(lower) & set(used)
    codes = [torch.zeros((pages, kv_heads, page, dim), dtype=torch.uint8, device=dev) for _ in "kv"]
    for c in codes:
        c[lower] = NAN_CODE
    cache = ffi.Kv8Cache(*codes, *[torch.ones((pages, kv_heads), device=dev) for _ in "kv"])
    small = ffi.Kv8Cache(*[torch.zeros((3, kv_heads, page, dim), dtype=torch.uint8, device=dev)
                           for _ in "kv"], *[torch.ones((3, kv_heads), device=dev) for _ in "kv"])
    x = torch.randn((300, 2 * kv_heads, dim), generator=base.gen(1)).bfloat16().to(dev)
    q = base.draw_q(300, 16, dim, 6).to(dev)
    for c, table in ((cache, used), (small, [0, 1, 2])):
        table = torch.tensor([table], dtype=torch.int32, device=dev)
        outs = []
        for first in range(0, 300, new):  # in one call, or token by token
            batch = ffi.Kv8Batch(torch.tensor([0, new], dtype=torch.int32, device=dev),
                                 torch.tensor([first + new], dtype=torch.int32, device=dev), table)
            part = x[first:first + new]
            ffi.kv8_append(c, batch, part[:, :kv_heads], part[:, kv_heads:])
            outs.append(ffi.kv8_attention(q[first:first + new], c, batch, 0.1))
        back = [torch.empty((new, kv_heads, dim), dtype=torch.bfloat16, device=dev) for _ in "kv"]
        ffi.kv8_read(c, batch, *back)
        assert ffi.kv8_batch_status(batch) == 0
        if c is cache:
            large = torch.cat(outs), back
    assert torch.equal(large[0], torch.cat(outs))
    assert all(torch.equal(a, b) for a, b in zip(large[1], back))
    for a, b, sa, sb in ((cache.k_codes, small.k_codes, cache.k_scales, small.k_scales),
                         (cache.v_codes, small.v_codes, cache.v_scales, small.v_scales)):
        assert torch.equal(a[used], b) and torch.equal(sa[used], sb)
        assert bool((a[lower] == NAN_CODE).all())
        touched = (a.view(torch.int64).view(pages, -1) != 0).any(1)
        touched[used + lower] = False
        assert not bool(touched.any())
        sa[used] = 1.0
        assert bool((sa == 1).all())
