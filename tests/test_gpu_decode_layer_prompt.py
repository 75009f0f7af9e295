"""A decoder layer's prompt (norms, products on 4-bit activations, cache, attention, FFN together):
the calls one by one, and what each of them is given against 64 bits."""
import pytest
import torch

import w4a4_reference as ref
from nvfp4_weight_only_gb300 import ffi, synth
from nvfp4_weight_only_gb300.decode_layer import DecodeLayer
from test_gpu_w4a4 import check

pytestmark = pytest.mark.gpu

H, I, HEADS, KV_HEADS, DIM, PAGE, MOST = 256, 528, 6, 2, 64, 16, 400


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ffi.load(build_if_missing=True)
    return torch.device("cuda:0")


def make(dev, **options):
    rope = ffi.rope_table(MOST + 64, DIM, 10000.0, dev)
    return DecodeLayer.synthetic(H, I, HEADS, KV_HEADS, DIM, dev, layer=3, rope=rope,
                                 prompt_tokens=MOST, **options)


def lists(dev, q_lens, kv_lens):
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    width = max(-(-n // PAGE) for n in kv_lens)
    table = torch.randperm(len(kv_lens) * width, generator=torch.Generator().manual_seed(1))
    starts = [0]
    for n in q_lens:
        starts.append(starts[-1] + n)
    batch = ffi.Kv8Batch(ints(starts), ints(kv_lens),
                         table.int().view(len(kv_lens), width).to(dev).contiguous())
    return ffi.Kv8Cache.empty(len(kv_lens) * width, KV_HEADS, PAGE, DIM, dev), batch


def weight(dev, i):
    n, k = [((HEADS + 2 * KV_HEADS) * DIM, H), (H, HEADS * DIM), (I, H), (I, H), (H, I)][i]
    q = ffi.nvfp4_quantize(synth.weights_f32(n, k, seed=synth.layer_seed(3, i), device=dev))
    return ref.weight(*q)


@pytest.mark.parametrize("q_lens", [[1], [65], [130], [400], [7, 0, 200, 128]])
def test_prompt_is_the_calls_one_by_one(dev, q_lens):
    layer = make(dev)
    T, s = sum(q_lens), layer.scales
    x, residual = [synth.activations_bf16(T, H, seed=i, device=dev) for i in range(2)]
    cache, batch = lists(dev, q_lens, q_lens)
    out, r = [t.clone() for t in layer.prompt(x, residual, cache, batch)]
    assert ffi.kv8_batch_status(batch) == 0
    assert ffi.nvfp4_workspace_status(layer.p_ws) == 0
    # one by one, with buffers of their own
    cache, _ = lists(dev, q_lens, q_lens)
    r1 = torch.empty_like(x)
    n = ffi.add_rmsnorm_bf16(x, layer.norm_in, layer.eps, residual=residual, sum_out=r1)
    fused = ffi.w4a4_gemm(ffi.w4a4_quantize(n), layer.p_qkv, s["qkv"], layer.rows)
    check(fused, *ref.product(ref.values(n), weight(dev, 0)))
    q, k, v = fused.view(T, -1, DIM).split((HEADS, KV_HEADS, KV_HEADS), 1)
    q = ffi.kv8_append(cache, batch, k, v, q=q, rope=layer.rope)
    a = ffi.kv8_attention(q, cache, batch, layer.softmax_scale).view(T, -1)
    p = ffi.w4a4_gemm(ffi.w4a4_quantize(a), layer.p_out, s["out"], H)
    check(p, *ref.product(ref.values(a), weight(dev, 1)))
    r2 = torch.empty_like(x)
    n2 = ffi.add_rmsnorm_bf16(p, layer.norm_ffn, layer.eps, residual=r1, sum_out=r2)
    f = ffi.ffn_swiglu_w4a4(n2, layer.p_gate_up, s["gate"], s["up"], layer.p_down, s["down"], I)
    assert torch.equal(out, f) and torch.equal(r, r2)


def test_a_prompt_in_pieces_then_tokens(dev):
    """Two pieces of a prompt and a token behind them, captured and replayed."""
    layer = make(dev)
    x, residual = [synth.activations_bf16(350, H, seed=i, device=dev) for i in range(2)]

    def run(pieces, graphs):
        cache, _ = lists(dev, [351], [351])
        outs, done = [], 0
        for n in pieces:
            _, batch = lists(dev, [n], [351])
            batch.kv_len.fill_(done + n)
            rows = slice(done, done + n)
            call = layer.prompt if n > 1 else layer.step
            a, b = x[rows].contiguous(), residual[rows].contiguous()
            if graphs:
                call(a, b, cache, batch)
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    out, _ = call(a, b, cache, batch)
                graph.replay()
            else:
                out, _ = call(a, b, cache, batch)
            outs.append(out.clone())
            assert ffi.kv8_batch_status(batch) == 0
            done += n
        return outs

    for a, b in zip(run([200, 149, 1], False), run([200, 149, 1], True)):
        assert bool(torch.isfinite(a.float()).all())
        assert torch.equal(a, b)


def test_prompt_refuses_other_sizes(dev):
    x = torch.zeros((MOST + 1, H), dtype=torch.bfloat16, device=dev)
    with pytest.raises(ValueError):
        make(dev).prompt(x, x, None, None)
    with pytest.raises(ValueError):
        DecodeLayer.synthetic(H, I, HEADS, KV_HEADS, DIM, dev).prompt(x[:1], x[:1], None, None)
