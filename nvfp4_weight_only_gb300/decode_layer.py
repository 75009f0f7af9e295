"""One decoder layer's step on the library: norms, NVFP4 projections, rotary positions, the paged
8-bit cache with attention over it, and the SwiGLU FFN.

    r      = x + residual
    q,k,v  = Wqkv norm(r)                        add_rmsnorm_bf16, nvfp4_gemv
    cache <- rotated k, v;  q rotated            kv8_append
    a      = attention(q, cache)                 kv8_attention
    r      = Wo a + r                            nvfp4_gemv, add_rmsnorm_bf16
    out    = down(act(gate(n)) * up(n)), n = norm(r)   ffn_swiglu_nvfp4

The step takes 1..64 token rows (the projections' range): one token of each of a batch of
sequences, a few draft tokens of each, or a piece of a prompt.  It returns out and the residual r,
which the next layer's first norm adds.  Buffers are allocated once, the sequences' lengths live on
the device, and every call goes to the current stream, so a step can be captured in a CUDA graph
and replayed while the lengths advance.

Prompts of any length go through `prompt`, in which the projections and the FFN run on activations
quantised to 4 bits (w4a4_quantize, w4a4_gemm, ffn_swiglu_w4a4); a layer made with prompt_tokens
keeps the weights in that layout too, and buffers for so many rows.

`python -m nvfp4_weight_only_gb300.decode_layer` runs steps of a layer with synthetic weights and
prints the time of one.
"""
import math

import torch

from . import ffi, synth

MAX_TOKENS = 64


class DecodeLayer:
    """weights: (codes, scales, scale2) of ffi.nvfp4_quantize for qkv [(heads + 2 kv_heads) head_dim,
    H], out [H, heads head_dim], gate and up [I, H], down [H, I]; norms: two bf16 [H]."""

    def __init__(self, qkv, out, gate, up, down, norm_in, norm_ffn, heads, kv_heads, head_dim,
                 rope=None, interleaved=False, window=0, sinks=0, eps=1e-6, act=ffi.NVFP4_ACT_SILU,
                 softmax_scale=None, prompt_tokens=0):
        self.H, self.I = norm_in.numel(), gate[0].shape[0]
        self.heads, self.kv_heads, self.head_dim = heads, kv_heads, head_dim
        self.rope, self.interleaved = rope, interleaved
        self.window, self.sinks, self.eps, self.act = window, sinks, eps, act
        self.softmax_scale = 1.0 / math.sqrt(head_dim) if softmax_scale is None else softmax_scale
        self.norm_in, self.norm_ffn = norm_in, norm_ffn
        H, I = self.H, self.I
        self.rows = (heads + 2 * kv_heads) * head_dim
        self.qkv = ffi.nvfp4_repack(qkv[0], qkv[1], self.rows, H)
        self.out = ffi.nvfp4_repack(out[0], out[1], H, heads * head_dim)
        self.gate_up = ffi.nvfp4_repack_gate_up(gate[0], gate[1], up[0], up[1], I, H)
        self.down = ffi.nvfp4_repack(down[0], down[1], H, I)
        self.scales = {"qkv": qkv[2], "out": out[2], "gate": gate[2], "up": up[2], "down": down[2]}
        dev = norm_in.device
        M = MAX_TOKENS
        new = lambda *shape: torch.empty(shape, dtype=torch.bfloat16, device=dev)  # noqa: E731
        self.normed, self.fused, self.turned = new(M, H), new(M, self.rows), new(M, heads, head_dim)
        self.attended, self.projected = new(M, heads, head_dim), new(M, H)
        self.residual, self.result = new(M, H), new(M, H)
        L = ffi.load()
        self.ws_bytes = max(L.nvfp4_gemv_workspace_bytes(M, self.rows, H),
                            L.nvfp4_gemv_workspace_bytes(M, H, heads * head_dim),
                            L.ffn_swiglu_nvfp4_workspace_bytes(M, H, I))
        self.ws = ffi.workspace(self.ws_bytes, dev)
        # as much as any step asks for: single tokens of a full batch, or many rows of one sequence
        self.attention_ws = ffi.workspace(
            max(ffi.kv8_attention_workspace_size(kv_heads, head_dim, 1024, 1, heads),
                ffi.kv8_attention_workspace_size(kv_heads, head_dim, 1, M, heads)), dev)
        self.prompt_tokens = prompt_tokens
        if prompt_tokens:
            self._prepare_prompts(qkv, out, gate, up, down, dev)

    def _prepare_prompts(self, qkv, out, gate, up, down, dev):
        M, H, I = self.prompt_tokens, self.H, self.I
        heads, kv_heads, dim = self.heads, self.kv_heads, self.head_dim
        self.p_qkv, self.p_out = ffi.w4a4_repack(*qkv[:2]), ffi.w4a4_repack(*out[:2])
        self.p_gate_up = ffi.w4a4_repack_gate_up(*gate[:2], *up[:2])
        self.p_down = ffi.w4a4_repack(*down[:2])
        new = lambda *shape: torch.empty(shape, dtype=torch.bfloat16, device=dev)  # noqa: E731
        self.p_normed, self.p_fused = new(M, H), new(M, self.rows)
        self.p_turned, self.p_attended = new(M, heads, dim), new(M, heads, dim)
        self.p_projected, self.p_residual, self.p_result = new(M, H), new(M, H), new(M, H)
        # rows of the norm and of attention; a call has fewer rows and takes their front
        size = ffi.load().w4a4_rows_bytes(M, max(H, heads * dim), 1)
        self.p_quantized = torch.empty(size, dtype=torch.uint8, device=dev)
        self.p_ws = ffi.workspace(max(
            ffi.w4a4_gemm_workspace_bytes(M, self.rows, H), ffi.w4a4_gemm_workspace_bytes(M, H, heads * dim),
            ffi.ffn_swiglu_w4a4_workspace_bytes(M, H, I)), dev)
        self.p_attention_ws = ffi.workspace(
            max(ffi.kv8_attention_workspace_size(kv_heads, dim, 1 << s, n, heads)
                for s in range(11) for n in {1 << s, max(M, 1 << s)}), dev)

    def _quantized(self, x):
        M, K = x.shape
        size = ffi.load().w4a4_rows_bytes(M, K, 1)
        return ffi.w4a4_quantize(x, out=ffi.W4a4Rows(self.p_quantized[:size], M, K))

    def prompt(self, x: torch.Tensor, residual: torch.Tensor, cache: ffi.Kv8Cache,
               batch: ffi.Kv8Batch):
        """x, residual bf16 [tokens, H], up to prompt_tokens of one or more sequences -> (out,
        residual), views of the layer's buffers.  As step, with the products on 4-bit activations."""
        M = x.shape[0]
        if not 1 <= M <= self.prompt_tokens:
            raise ValueError(f"this layer's prompts have 1..{self.prompt_tokens} tokens, got {M}")
        s, heads, kv_heads, dim = self.scales, self.heads, self.kv_heads, self.head_dim
        n, r = self.p_normed[:M], self.p_residual[:M]
        ffi.add_rmsnorm_bf16(x, self.norm_in, self.eps, residual=residual, sum_out=r, out=n)
        fused = ffi.w4a4_gemm(self._quantized(n), self.p_qkv, s["qkv"], self.rows, ws=self.p_ws,
                              out=self.p_fused[:M])
        q, k, v = fused.view(M, -1, dim).split((heads, kv_heads, kv_heads), 1)
        q = ffi.kv8_append(cache, batch, k, v, q=q, q_out=self.p_turned[:M], rope=self.rope,
                           interleaved=self.interleaved)
        a = ffi.kv8_attention(q, cache, batch, self.softmax_scale, window=self.window,
                              sinks=self.sinks, ws=self.p_attention_ws, out=self.p_attended[:M])
        p = ffi.w4a4_gemm(self._quantized(a.view(M, -1)), self.p_out, s["out"], self.H,
                          ws=self.p_ws, out=self.p_projected[:M])
        ffi.add_rmsnorm_bf16(p, self.norm_ffn, self.eps, residual=r, sum_out=r, out=n)
        out = ffi.ffn_swiglu_w4a4(n, self.p_gate_up, s["gate"], s["up"], self.p_down, s["down"],
                                  self.I, self.act, ws=self.p_ws, out=self.p_result[:M])
        return out, r

    def step(self, x: torch.Tensor, residual: torch.Tensor, cache: ffi.Kv8Cache,
             batch: ffi.Kv8Batch):
        """x, residual bf16 [tokens, H] -> (out, residual), views of the layer's buffers."""
        M = x.shape[0]
        if not 1 <= M <= MAX_TOKENS:
            raise ValueError(f"a step takes 1..{MAX_TOKENS} tokens, got {M}")
        s, heads, kv_heads, dim = self.scales, self.heads, self.kv_heads, self.head_dim
        n, r = self.normed[:M], self.residual[:M]
        ffi.add_rmsnorm_bf16(x, self.norm_in, self.eps, residual=residual, sum_out=r, out=n)
        fused = ffi.nvfp4_gemv(n, self.qkv, s["qkv"], self.rows, ws=self.ws, out=self.fused[:M])
        q, k, v = fused.view(M, -1, dim).split((heads, kv_heads, kv_heads), 1)
        q = ffi.kv8_append(cache, batch, k, v, q=q, q_out=self.turned[:M], rope=self.rope,
                           interleaved=self.interleaved)
        a = ffi.kv8_attention(q, cache, batch, self.softmax_scale, window=self.window,
                              sinks=self.sinks, ws=self.attention_ws, out=self.attended[:M])
        p = ffi.nvfp4_gemv(a.view(M, -1), self.out, s["out"], self.H, ws=self.ws,
                           out=self.projected[:M])
        ffi.add_rmsnorm_bf16(p, self.norm_ffn, self.eps, residual=r, sum_out=r, out=n)
        out = ffi.ffn_swiglu_nvfp4(n, self.gate_up, s["gate"], s["up"], self.down, s["down"], self.I,
                                   self.act, ws=self.ws, out=self.result[:M])
        return out, r

    @classmethod
    def synthetic(cls, H, I, heads, kv_heads, head_dim, device, layer=0, **options):
        """A layer with seeded random weights, quantised by the library."""
        shapes = [((heads + 2 * kv_heads) * head_dim, H), (H, heads * head_dim), (I, H), (I, H),
                  (H, I)]
        w = [ffi.nvfp4_quantize(synth.weights_f32(n, k, seed=synth.layer_seed(layer, i),
                                                  device=device))
             for i, (n, k) in enumerate(shapes)]
        g = torch.Generator(device=device).manual_seed(synth.layer_seed(layer, 7))
        norms = [(1 + 0.1 * torch.randn(H, generator=g, device=device)).bfloat16()
                 for _ in range(2)]
        return cls(*w, *norms, heads, kv_heads, head_dim, **options)


def main():
    dev = torch.device("cuda:0")
    ffi.load(build_if_missing=True)
    H, I, heads, kv_heads, dim, page, sequences, length = 5120, 17408, 40, 8, 128, 64, 16, 4096
    layer = DecodeLayer.synthetic(H, I, heads, kv_heads, dim, dev, prompt_tokens=length,
                                  rope=ffi.rope_table(length + 64, dim, 500000.0, dev))
    width = (length + 64) // page
    cache = ffi.Kv8Cache.empty(sequences * width, kv_heads, page, dim, dev)
    cache.k_codes.random_(0, 127)
    cache.v_codes.random_(0, 127)
    table = torch.randperm(sequences * width, device=dev).int().view(sequences, width)
    batch = ffi.Kv8Batch(torch.arange(sequences + 1, dtype=torch.int32, device=dev),
                         torch.full((sequences,), length, dtype=torch.int32, device=dev), table)
    x, residual = [synth.activations_bf16(sequences, H, seed=i, device=dev) for i in range(2)]
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    prompt = ffi.Kv8Batch(ints(0, length), ints(length), table[:1].contiguous())
    px, presidual = [synth.activations_bf16(length, H, seed=i, device=dev) for i in (2, 3)]

    def token():
        batch.kv_len += 1  # the next token's position
        layer.step(x, residual, cache, batch)

    what = (f"decoder layer H={H} I={I}, {heads}/{kv_heads} heads of {dim}")
    us = _replayed(lambda: layer.prompt(px, presidual, cache, prompt))
    print(f"{what}, a prompt of {length} tokens: {us:.1f} us")
    us = _replayed(token)
    print(f"{what}, {sequences} sequences of {length} tokens: {us:.1f} us per step")
    assert ffi.kv8_batch_status(batch) == 0 and ffi.kv8_batch_status(prompt) == 0


def _replayed(step, steps=40):
    """Microseconds of one replay of a captured step."""
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    graph.replay()
    begin, end = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    begin.record()
    for _ in range(steps):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    return begin.elapsed_time(end) / steps * 1e3


if __name__ == "__main__":
    main()
