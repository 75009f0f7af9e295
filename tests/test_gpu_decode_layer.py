"""A decoder layer's step (norms, projections, cache, attention, FFN together) against 64 bits.

The reference rounds to bf16 where the layer's buffers are bf16 and attends over the keys and
values that the cache holds (read back), so what is left are roundings that fall differently: eight
bf16 stages of about 2^-9 of a row's norm each, through maps that keep relative errors within a
small factor.  0.02 of the norm is several times their sum."""
import math

import pytest
import torch

import kv8_reference as ref
from nvfp4_weight_only_gb300 import ffi, synth
from nvfp4_weight_only_gb300.decode_layer import DecodeLayer

pytestmark = pytest.mark.gpu

H, I, HEADS, KV_HEADS, DIM, PAGE = 512, 1024, 8, 2, 64, 16
BOUND = 0.02


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ffi.load(build_if_missing=True)
    return torch.device("cuda:0")


def bf16(x):
    return x.float().bfloat16().double()


def weights(layer_seed, dev):
    shapes = [((HEADS + 2 * KV_HEADS) * DIM, H), (H, HEADS * DIM), (I, H), (I, H), (H, I)]
    out = []
    for i, (n, k) in enumerate(shapes):
        q = ffi.nvfp4_quantize(synth.weights_f32(n, k, seed=synth.layer_seed(layer_seed, i),
                                                 device=dev))
        codes, scales = q[0].cpu(), q[1].cpu()
        table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6]).double()
        c = torch.stack((codes & 15, codes >> 4), -1).flatten(1).long()
        out.append(table[c] * ref.e4m3_value(scales).repeat_interleave(16, 1) * q[2])
    return out


def reference(layer, w, x, residual, cache, batch, q_lens, kv_lens, table):
    """(out, r) of one step, the cache already holding this step's tokens."""
    M = x.shape[0]
    r, y = ref.norm(x, residual, layer.norm_in.cpu(), layer.eps)
    r = bf16(r)
    fused = bf16(bf16(y) @ w[0].T).view(M, -1, DIM)
    positions = [kv - n + i for n, kv in zip(q_lens, kv_lens) for i in range(n)]
    q = bf16(ref.rotate(fused[:, :HEADS], layer.rope.cpu(), positions, layer.interleaved))
    k_values = ref.dequantise(cache.k_codes.cpu(), cache.k_scales.cpu())
    v_values = ref.dequantise(cache.v_codes.cpu(), cache.v_scales.cpu())
    a = bf16(ref.attention(q, k_values, v_values, PAGE, table, q_lens, kv_lens,
                           layer.softmax_scale, layer.window, layer.sinks)[0])
    p = bf16(a.reshape(M, -1) @ w[1].T)
    r2, y = ref.norm(p, r, layer.norm_ffn.cpu(), layer.eps)
    n = bf16(y)
    g, u = bf16(n @ w[2].T), bf16(n @ w[3].T)
    h = bf16(g / (1 + torch.exp(-g)) * u)
    return h @ w[4].T, bf16(r2), fused


@pytest.mark.parametrize("q_lens,window,interleaved", [([1], 0, False), ([1, 1, 1], 0, True),
                                                       ([4, 2], 20, False), ([40], 0, False)])
def test_steps(dev, q_lens, window, interleaved):
    B = len(q_lens)
    rope = ffi.rope_table(200, DIM, 10000.0, dev)
    layer = DecodeLayer.synthetic(H, I, HEADS, KV_HEADS, DIM, dev, layer=3, rope=rope, window=window,
                                  sinks=2, interleaved=interleaved)
    w = weights(3, dev)
    width = 9
    cache = ffi.Kv8Cache.empty(B * width, KV_HEADS, PAGE, DIM, dev)
    table = torch.randperm(B * width, generator=torch.Generator().manual_seed(1)).int().view(B,
                                                                                              width)
    starts = [sum(q_lens[:b]) for b in range(B + 1)]
    batch = ffi.Kv8Batch(torch.tensor(starts, dtype=torch.int32, device=dev),
                         torch.zeros(B, dtype=torch.int32, device=dev), table.to(dev))
    kv_lens = [0] * B
    for step in range(3):
        kv_lens = [kv + n for kv, n in zip(kv_lens, q_lens)]
        batch.kv_len.copy_(torch.tensor(kv_lens, dtype=torch.int32))
        x = synth.activations_bf16(starts[-1], H, seed=10 + step)
        residual = synth.activations_bf16(starts[-1], H, seed=20 + step)
        out, r = layer.step(x.to(dev), residual.to(dev), cache, batch)
        torch.cuda.synchronize()
        assert ffi.kv8_batch_status(batch) == 0
        want, want_r, fused = reference(layer, w, x, residual, cache, batch, q_lens, kv_lens, table)
        for got, ideal in ((out, want), (r, want_r)):
            err = (got.cpu().double() - ideal).norm(dim=1) / ideal.norm(dim=1)
            assert float(err.max()) < BOUND
        # the cache holds this step's v within E4M3's rounding (2^-4 of the value, 2^-10 of the
        # page's largest for the smallest codes)
        k_out = torch.empty((starts[-1], KV_HEADS, DIM), dtype=torch.bfloat16, device=dev)
        v_out = torch.empty_like(k_out)
        ffi.kv8_read(cache, batch, k_out, v_out)
        v = fused[:, HEADS + KV_HEADS:]
        off = (v_out.cpu().double() - v).norm() / v.norm()
        assert float(off) < 2 ** -4


def test_step_is_the_calls_one_by_one(dev):
    """The same bits as separate calls on separate buffers, and in a graph."""
    rope = ffi.rope_table(100, DIM, 10000.0, dev)
    layer = DecodeLayer.synthetic(H, I, HEADS, KV_HEADS, DIM, dev, layer=1, rope=rope)
    make = lambda: ffi.Kv8Cache(  # noqa: E731
        *[torch.zeros((8, KV_HEADS, PAGE, DIM), dtype=torch.uint8, device=dev) for _ in "kv"],
        *[torch.ones((8, KV_HEADS), device=dev) for _ in "kv"])
    batch = ffi.Kv8Batch(torch.tensor([0, 1, 2], dtype=torch.int32, device=dev),
                         torch.tensor([17, 40], dtype=torch.int32, device=dev),
                         torch.arange(8, dtype=torch.int32, device=dev).view(2, 4).contiguous())
    x, residual = [synth.activations_bf16(2, H, seed=i).to(dev) for i in (1, 2)]
    out, r = [t.clone() for t in layer.step(x, residual, make(), batch)]
    cache, s = make(), layer.scales
    r1 = torch.empty_like(x)
    n = ffi.add_rmsnorm_bf16(x, layer.norm_in, layer.eps, residual=residual, sum_out=r1)
    fused = ffi.nvfp4_gemv(n, layer.qkv, s["qkv"], layer.rows).view(2, -1, DIM)
    q = ffi.kv8_append(cache, batch, fused[:, HEADS:HEADS + KV_HEADS],
                       fused[:, HEADS + KV_HEADS:], q=fused[:, :HEADS], rope=rope)
    a = ffi.kv8_attention(q, cache, batch, 1 / math.sqrt(DIM))
    p = ffi.nvfp4_gemv(a.view(2, -1), layer.out, s["out"], H)
    r2 = torch.empty_like(x)
    n2 = ffi.add_rmsnorm_bf16(p, layer.norm_ffn, layer.eps, residual=r1, sum_out=r2)
    f = ffi.ffn_swiglu_nvfp4(n2, layer.gate_up, s["gate"], s["up"], layer.down, s["down"], I)
    assert torch.equal(out, f) and torch.equal(r, r2)
    held = make()
    layer.step(x, residual, held, batch)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer.step(x, residual, held, batch)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], out) and torch.equal(got[1], r)


def test_step_refuses_other_sizes(dev):
    layer = DecodeLayer.synthetic(H, I, HEADS, KV_HEADS, DIM, dev)
    x = torch.zeros((65, H), dtype=torch.bfloat16, device=dev)
    with pytest.raises(ValueError):
        layer.step(x, x, None, None)


def test_a_softmax_scale_of_zero_is_kept(dev):
    layer = DecodeLayer.synthetic(H, I, HEADS, KV_HEADS, DIM, dev, softmax_scale=0.0)
    assert layer.softmax_scale == 0.0
