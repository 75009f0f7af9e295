"""Products on 4-bit activations at sizes that pairs of blocks take, from the device's number of SMs:
several streams, shared workspaces, captured calls, both ends of the row scales, a layer's prompt."""
import pytest
import torch

import w4a4_reference as ref
from nvfp4_weight_only_gb300 import ffi, synth
from nvfp4_weight_only_gb300.decode_layer import DecodeLayer
from test_gpu_decode_layer_prompt import lists
from test_gpu_w4a4 import BF, check, check_gated, draw, draw_ids, draw_weight

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ffi.load(build_if_missing=True)
    return torch.device("cuda:0")


def sms(dev):
    return torch.cuda.get_device_properties(dev).multi_processor_count


def features(M, dev, turns=1.0):
    """Features of a weight whose 128 x 128 tiles with M rows are more than so many turns of the SMs;
    the last is ragged.  Pairs take 256 x 256: from 2.1 turns on a few tiles are left behind theirs,
    which long rows have cut and joined."""
    return 256 * (int(turns * sms(dev)) // (2 * ((M + 127) // 128)) + 1) - 56


def make(M, K, N, seed, dev):
    x, w = draw(M, K, seed, dev), draw_weight(N, K, seed + 1, dev)
    return x, ffi.w4a4_repack(*w[:2]), w


@pytest.mark.parametrize("other", ["pairs", "few", "experts"])
def test_two_streams(dev, other):
    """Products of pairs, with cut tiles and their join, beside others on a second stream."""
    calls = []
    for i, kind in enumerate(("pairs", other)):
        if kind == "experts":
            M, K, N, E = 1500, 4096, 500, 4
            x, w = draw(M, K, i, dev), draw_weight(N, K, 9, dev, E)
            start = torch.tensor([0, 700, 701, 1100, 1500], dtype=torch.int32, device=dev)
            packed, scale = ffi.w4a4_repack(*w[:2]), w[2]
        else:
            M, K = (1000, 8192) if kind == "pairs" else (40, 8192)
            N = features(M, dev, 2.1) if kind == "pairs" else 1000
            x, packed, w = make(M, K, N, 3 * i, dev)
            start, scale, E = None, w[2], 1
        rows = ffi.W4a4Rows.empty(M, K, dev, start)
        ws = ffi.workspace(ffi.w4a4_gemm_workspace_bytes(M, N, K, E), dev)
        out = torch.empty((M, N), dtype=BF, device=dev)

        def call(x=x, rows=rows, packed=packed, scale=scale, N=N, ws=ws, out=out):
            ffi.w4a4_quantize(x, out=rows)
            return ffi.w4a4_gemm(rows, packed, scale, N, ws=ws, out=out)

        calls.append((call, call().clone(), out, ws, torch.cuda.Stream(dev)))
    torch.cuda.synchronize()
    for _ in range(30):
        for call, _, _, _, stream in calls:
            with torch.cuda.stream(stream):
                call()
    torch.cuda.synchronize()
    for _, want, out, ws, _ in calls:
        assert torch.equal(out, want)
        assert ffi.nvfp4_workspace_status(ws) == 0


def test_a_workspace_serves_both_kernels_and_their_joins_in_turn(dev):
    shapes = [(1000, 8192, features(1000, dev, 2.1)), (1, 17408, 300), (300, 16384, 528),
              (2000, 272, features(2000, dev)), (40, 1024, 30000), (129, 16384, features(129, dev, 2.05)),
              (100, 5376, 513)]
    ws = ffi.workspace(max(ffi.w4a4_gemm_workspace_bytes(m, n, k) for m, k, n in shapes), dev)
    wants = []
    for turn in range(3):
        for i, (M, K, N) in enumerate(shapes):
            x, packed, w = make(M, K, N, 2 * i, dev)
            rows = ffi.w4a4_quantize(x)
            got = ffi.w4a4_gemm(rows, packed, w[2], N, ws=ws)
            if turn == 0:
                check(got, *ref.product(ref.values(x), ref.weight(*w)))
                wants.append(got)
            assert torch.equal(got, wants[i])
    assert ffi.nvfp4_workspace_status(ws) == 0
    assert int(ws[256:256 + (128 << 10)].count_nonzero()) == 0


def test_rows_at_both_ends_of_the_scales(dev):
    M, K = 300, 256
    N = features(M, dev)
    x = draw(M, K, 5, dev).double()
    x *= torch.exp2(torch.linspace(-118, 112, M, device=dev, dtype=torch.float64).round())[:, None]
    x = x.to(BF)
    w = draw_weight(N, K, 6, dev)
    want, off = ref.product(ref.values(x), ref.weight(*w))
    y = ffi.w4a4_gemm(ffi.w4a4_quantize(x), ffi.w4a4_repack(*w[:2]), w[2], N)
    # r times the scaled sum is an fp32 value: beyond its range, or rounded beyond bf16's, infinite
    near = want.abs() + off < 2.0 ** 128 * (1 - 2.0 ** -8)
    assert bool(torch.isinf(y[want.abs() - off > 2.0 ** 128]).all())
    assert bool(near.any(1).sum() > 290)
    check(torch.where(near, y.double(), 0.0), torch.where(near, want, 0.0), off)


def test_captured_calls_that_share_a_workspace(dev):
    """A product, an FFN and an experts' FFN of pairs in one graph, a product in another, on one
    workspace, replayed in turn with other inputs."""
    M, H, I, E = 1100, 8192, 2064, 2
    N = features(M, dev, 2.1)
    x, ids = draw(M, H, 1, dev), draw_ids(M, 2, E, 1, dev)
    weights = torch.rand((M, 2), device=dev)
    dense = draw_weight(N, H, 2, dev)
    packed = ffi.w4a4_repack(*dense[:2])
    one = [draw_weight(*s, i, dev) for i, s in enumerate(((I, H), (I, H), (H, I)))]
    gu, dn = ffi.w4a4_repack_gate_up(*one[0][:2], *one[1][:2]), ffi.w4a4_repack(*one[2][:2])
    many = [draw_weight(*s, i, dev, E) for i, s in enumerate(((I, H), (I, H), (H, I)))]
    egu, edn = ffi.w4a4_repack_gate_up(*many[0][:2], *many[1][:2]), ffi.w4a4_repack(*many[2][:2])
    s, es = 1e-5, torch.full((E,), 1e-5, device=dev)
    ws = ffi.workspace(max(ffi.w4a4_gemm_workspace_bytes(M, N, H),
                           ffi.ffn_swiglu_w4a4_workspace_bytes(M, H, I),
                           ffi.experts_swiglu_w4a4_workspace_bytes(M, 2, E, H, I)), dev)
    rows = ffi.W4a4Rows.empty(M, H, dev)
    outs = [torch.empty((M, n), dtype=BF, device=dev) for n in (N, H, H, N)]

    def first():
        ffi.w4a4_gemm(ffi.w4a4_quantize(x, out=rows), packed, dense[2], N, ws=ws, out=outs[0])
        ffi.ffn_swiglu_w4a4(x, gu, s, s, dn, 1e-3, I, ws=ws, out=outs[1])
        ffi.experts_swiglu_w4a4(x, ids, weights, egu, es, es, edn, many[2][2], I, ws=ws, out=outs[2])

    def second():
        ffi.w4a4_gemm(ffi.w4a4_quantize(outs[1], out=rows), packed, dense[2], N, ws=ws, out=outs[3])

    first()
    second()
    graphs = []
    for step in (first, second):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            step()
    for seed in (5, 6, 7):
        x.copy_(draw(M, H, seed, dev))
        ids.copy_(draw_ids(M, 2, E, seed, dev))
        for g in graphs + graphs[:1] + graphs[1:]:
            g.replay()
        got = [t.clone() for t in outs]
        first()
        second()
        for a, b in zip(got, outs):
            assert torch.equal(a, b)
        assert ffi.nvfp4_workspace_status(ws) == 0
    check(outs[0], *ref.product(ref.values(x), ref.weight(*dense)))


@pytest.mark.parametrize("kind", [0, 1])
def test_gate_up_and_ffn(dev, kind):
    M, H = 500, 8192
    I = features(M, dev, 2.1) // 2 // 16 * 16
    x = draw(M, H, 1, dev)
    gate, up, down = draw_weight(I, H, 1, dev), draw_weight(I, H, 2, dev), draw_weight(H, I, 3, dev)
    gu, dn = ffi.w4a4_repack_gate_up(*gate[:2], *up[:2]), ffi.w4a4_repack(*down[:2])
    s = 1e-3 / H ** 0.5
    h = ffi.w4a4_gate_up(ffi.w4a4_quantize(x), gu, s, 2 * s, I, kind)
    check_gated(h, kind, ref.values(x), ref.weight(*gate[:2], s), ref.weight(*up[:2], 2 * s))
    out = ffi.ffn_swiglu_w4a4(x, gu, s, 2 * s, dn, down[2], I, kind)
    check(out, *ref.product(ref.values(h), ref.weight(*down)))


@pytest.mark.parametrize("pieces", [[1.0], [0.25, 0.75]])
def test_a_layer_s_prompt(dev, pieces):
    """So many tokens that each projection takes pairs; by itself, its calls one by one, captured."""
    H, I, HEADS, KV_HEADS, DIM = 1024, 1040, 8, 2, 64
    # the projection with the fewest features is q, k and v's: 12 heads of 64, 6 tiles of 128
    T = 128 * (sms(dev) // 6 + 1) - 5
    layer = DecodeLayer.synthetic(H, I, HEADS, KV_HEADS, DIM, dev, layer=3, prompt_tokens=T,
                                  rope=ffi.rope_table(T + 64, DIM, 10000.0, dev))
    lens = [int(p * T) for p in pieces]
    lens[-1] = T - sum(lens[:-1])
    x, residual = [synth.activations_bf16(T, H, seed=i, device=dev) for i in range(2)]
    cache, batch = lists(dev, lens, lens)
    out, r = [t.clone() for t in layer.prompt(x, residual, cache, batch)]
    assert ffi.kv8_batch_status(batch) == 0 and ffi.nvfp4_workspace_status(layer.p_ws) == 0
    cache, batch = lists(dev, lens, lens)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again, r_again = layer.prompt(x, residual, cache, batch)
    graph.replay()
    assert torch.equal(out, again) and torch.equal(r, r_again)

    def weight(i, n, k):
        q = ffi.nvfp4_quantize(synth.weights_f32(n, k, seed=synth.layer_seed(3, i), device=dev))
        return ref.weight(*q)

    s = layer.scales
    cache, batch = lists(dev, lens, lens)
    r1 = torch.empty_like(x)
    n = ffi.add_rmsnorm_bf16(x, layer.norm_in, layer.eps, residual=residual, sum_out=r1)
    fused = ffi.w4a4_gemm(ffi.w4a4_quantize(n), layer.p_qkv, s["qkv"], layer.rows)
    check(fused, *ref.product(ref.values(n), weight(0, (HEADS + 2 * KV_HEADS) * DIM, H)))
    q, k, v = fused.view(T, -1, DIM).split((HEADS, KV_HEADS, KV_HEADS), 1)
    q = ffi.kv8_append(cache, batch, k, v, q=q, rope=layer.rope)
    a = ffi.kv8_attention(q, cache, batch, layer.softmax_scale).view(T, -1)
    p = ffi.w4a4_gemm(ffi.w4a4_quantize(a), layer.p_out, s["out"], H)
    check(p, *ref.product(ref.values(a), weight(1, H, HEADS * DIM)))
    r2 = torch.empty_like(x)
    n2 = ffi.add_rmsnorm_bf16(p, layer.norm_ffn, layer.eps, residual=r1, sum_out=r2)
    h = ffi.w4a4_gate_up(ffi.w4a4_quantize(n2), layer.p_gate_up, s["gate"], s["up"], I)
    f = ffi.w4a4_gemm(ffi.w4a4_quantize(h), layer.p_down, s["down"], H)
    check(f, *ref.product(ref.values(h), weight(4, H, I)))
    assert torch.equal(out, f) and torch.equal(r, r2)
