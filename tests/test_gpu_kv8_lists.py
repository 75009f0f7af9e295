"""Lists that do not fit the call's buffers, or strain the kernels' index arithmetic: what they
concern is left out and reported, everything else is right, and the workspace serves the next call.
Tolerances are those of test_gpu_kv8.py."""
import math

import pytest
import torch

import kv8_reference as ref
from nvfp4_weight_only_gb300 import ffi
from test_gpu_kv8 import Setup, check_attention, draw_q, run_attention

pytestmark = pytest.mark.gpu

RANGE = 4


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ffi.load(build_if_missing=True)
    return torch.device("cuda:0")


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("sequences,tokens,group,keys", [
    (60, 2048, 1, 2 ** 20),  # many rows per sequence: 240 units of 256 rows where 68 are the bound
    (64, 64, 8, 2 ** 19)])   # few rows: 2048 units of 8 rows where 64 are the bound
def test_overlapping_sequences_leave_the_workspace_whole(dev, dim, sequences, tokens, group, keys):
    """q_start = 0, T, 0, T, ...: every second sequence has all T tokens, so there are many more
    units than tokens allow.  The call reports it; the next, on the same workspace, is right."""
    page = 256
    pages = 8
    shape = (pages, 1, page, dim)
    g = torch.Generator().manual_seed(3)
    codes = [ref.round_e4m3(torch.randn(shape, generator=g) * 100).to(dev) for _ in "kv"]
    cache = ffi.Kv8Cache(*codes, *[torch.full((pages, 1), 2.0 ** -7, device=dev) for _ in "kv"])
    starts = [tokens * (b % 2) for b in range(sequences + 1)]
    lens = [tokens] * sequences
    lens[36] = keys  # its units stand where the blocks would end
    # pages may be shared by sequences that are only read
    table = (torch.arange(keys // page, dtype=torch.int32) % pages).expand(sequences, -1)
    bad = ffi.Kv8Batch(torch.tensor(starts, dtype=torch.int32, device=dev),
                       torch.tensor(lens, dtype=torch.int32, device=dev),
                       table.contiguous().to(dev))
    q = draw_q(tokens, group, dim, 5).to(dev)
    ws = ffi.workspace(ffi.kv8_attention_workspace_bytes(cache, bad, tokens, group), dev)
    ffi.kv8_attention(q, cache, bad, 0.1, ws=ws)
    assert ffi.kv8_batch_status(bad) == RANGE
    assert ffi.nvfp4_workspace_status(ws) == 0
    # the same sizes in order: T / sequences tokens each, and one sequence with all of them
    for batch in (ffi.Kv8Batch(
            torch.tensor([tokens * b // sequences for b in range(sequences + 1)], dtype=torch.int32,
                         device=dev), bad.kv_len, bad.page_table),
                  ffi.Kv8Batch(torch.tensor([0, tokens], dtype=torch.int32, device=dev),
                               bad.kv_len[36:37].contiguous(), bad.page_table[36:37].contiguous())):
        fresh = ffi.workspace(ffi.kv8_attention_workspace_bytes(cache, batch, tokens, group), dev)
        want = ffi.kv8_attention(q, cache, batch, 0.1, ws=fresh)
        if fresh.numel() <= ws.numel():
            for _ in range(2):
                assert torch.equal(ffi.kv8_attention(q, cache, batch, 0.1, ws=ws), want)
        assert ffi.kv8_batch_status(batch) == 0


@pytest.mark.parametrize("q_lens,kv_lens,group", [([7, 1], [2, 50], 1), ([40, 1], [10, 50], 2)])
def test_a_window_of_any_size_beside_missing_positions(dev, q_lens, kv_lens, group):
    """More new tokens than the length, by more than one, under the largest windows, few rows and
    many: the tokens that have a position, and the other sequence, get their results."""
    s = Setup(dev, q_lens, kv_lens, 2, 64, 16)
    q = draw_q(s.tokens, 2 * group, 64, 2)
    none = q_lens[0] - kv_lens[0]
    want, want_lse = run_attention(s, q, 0.1)
    assert ffi.kv8_batch_status(s.batch) == RANGE
    assert bool((want[:none] == 0).all()) and bool((want_lse[:none] == -math.inf).all())
    assert bool(torch.isfinite(want_lse[none:]).all())
    for window in (2 ** 31 - 1, 2 ** 31 - 2, 2 ** 30):
        out = torch.full_like(want, 7.0)
        lse = torch.full_like(want_lse, 7.0)
        ffi.kv8_attention(q.to(dev), s.cache, s.batch, 0.1, window, 3, out=out, lse=lse)
        assert ffi.kv8_batch_status(s.batch) == RANGE
        assert torch.equal(out, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("q_lens,kv_lens,heads,kv_heads,dim,inter", [
    ([1, 1], [8, 9], 4, 2, 64, False),         # the second token just behind the table
    ([3, 2], [10, 3], 6, 1, 128, True),        # a run that crosses the table's end
    ([40, 1], [60, 5], 4, 2, 128, False),      # a prompt, of which 8 rows stay
])
def test_positions_behind_the_rotation_table_are_not_written(dev, q_lens, kv_lens, heads, kv_heads,
                                                             dim, inter):
    positions = 28 if max(q_lens) > 16 else 8
    page = 16
    s = Setup(dev, q_lens, kv_lens, kv_heads, dim, page, seed=41)
    t = sum(q_lens)
    x = torch.randn((t, heads + 2 * kv_heads, dim), generator=torch.Generator().manual_seed(6))
    x = x.bfloat16().to(dev)
    q, k, v = x.split((heads, kv_heads, kv_heads), 1)
    rope = ffi.rope_table(positions, dim, 10000.0, dev)
    q_out = torch.full((t, heads, dim), 7.0, dtype=torch.bfloat16, device=dev)
    before = [c.clone() for c in (s.cache.k_codes, s.cache.v_codes)]
    scales = [c.clone() for c in (s.cache.k_scales, s.cache.v_scales)]
    ffi.kv8_append(s.cache, s.batch, k, v, q=q, q_out=q_out, rope=rope, interleaved=inter)
    assert ffi.kv8_batch_status(s.batch) == RANGE
    # the same with a table that holds every position, and only the tokens that the short one holds
    kept = [i for i in range(t)]
    at, n_lens, m_lens = 0, [], []
    keep = []
    for n, kv in zip(q_lens, kv_lens):
        some = [i for i in range(n) if kv - n + i < positions]
        keep += [at + i for i in some]
        n_lens.append(len(some))
        m_lens.append(kv - n + len(some))
        at += n
    assert 0 < len(keep) < len(kept)
    o = Setup(dev, q_lens, kv_lens, kv_heads, dim, page, seed=41)
    starts = [sum(n_lens[:b]) for b in range(len(n_lens) + 1)]
    batch = ffi.Kv8Batch(torch.tensor(starts, dtype=torch.int32, device=dev),
                         torch.tensor(m_lens, dtype=torch.int32, device=dev), o.batch.page_table)
    some = x[keep]
    want_q = ffi.kv8_append(o.cache, batch, some[:, heads:heads + kv_heads],
                            some[:, heads + kv_heads:], q=some[:, :heads],
                            rope=ffi.rope_table(100, dim, 10000.0, dev), interleaved=inter)
    assert ffi.kv8_batch_status(batch) == 0
    for a, b in ((s.cache.k_codes, o.cache.k_codes), (s.cache.v_codes, o.cache.v_codes)):
        assert torch.equal(a, b)
    for a, b in ((s.cache.k_scales, o.cache.k_scales), (s.cache.v_scales, o.cache.v_scales)):
        assert torch.equal(torch.nan_to_num(a), torch.nan_to_num(b))
    assert torch.equal(q_out[keep], want_q)
    left = [i for i in kept if i not in keep]
    assert bool((q_out[left] == 7).all())


def test_rows_of_no_sequence_take_no_part(dev):
    """A call of a fixed number of rows (a captured step, say) of which the last belong to nobody:
    no call computes or reports anything for them."""
    s = Setup(dev, [2, 1], [30, 9], 2, 64, 16, seed=43)
    x = torch.randn((6, 4 + 4, 64), generator=torch.Generator().manual_seed(9)).bfloat16().to(dev)
    rope = ffi.rope_table(40, 64, 10000.0, dev)
    q_out = torch.full((6, 4, 64), 7.0, dtype=torch.bfloat16, device=dev)
    out = torch.full((6, 4, 64), 7.0, dtype=torch.bfloat16, device=dev)
    ffi.kv8_append(s.cache, s.batch, x[:, 4:6], x[:, 6:], q=x[:, :4], q_out=q_out, rope=rope)
    ffi.kv8_attention(q_out, s.cache, s.batch, 0.1, out=out)
    k, v = [torch.full((6, 2, 64), 7.0, dtype=torch.bfloat16, device=dev) for _ in "kv"]
    ffi.kv8_read(s.cache, s.batch, k, v)
    assert ffi.kv8_batch_status(s.batch) == 0
    for t in (q_out, out, k, v):
        assert bool((t[3:] == 7).all()) and not bool((t[:3] == 7).all(-1).any())


def test_tokens_in_front_of_position_0_keep_their_q(dev):
    """More new tokens than the length: rotated q is written for those that have a position."""
    s = Setup(dev, [4], [2], 1, 64, 16, seed=44)
    x = torch.randn((4, 4, 64), generator=torch.Generator().manual_seed(9)).bfloat16().to(dev)
    rope = ffi.rope_table(40, 64, 10000.0, dev)
    q_out = torch.full((4, 2, 64), 7.0, dtype=torch.bfloat16, device=dev)
    ffi.kv8_append(s.cache, s.batch, x[:, 2:3], x[:, 3:], q=x[:, :2], q_out=q_out, rope=rope)
    assert ffi.kv8_batch_status(s.batch) == RANGE
    assert bool((q_out[:2] == 7).all())
    only = Setup(dev, [2], [2], 1, 64, 16, seed=44)
    want = ffi.kv8_append(only.cache, only.batch, x[2:, 2:3], x[2:, 3:], q=x[2:, :2], rope=rope)
    assert torch.equal(q_out[2:], want)
