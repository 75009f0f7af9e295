// kv8_attention.cu -- attention of new tokens over the paged E4M3 cache.
//
// Query i of a sequence of n new tokens and length kv has position
// p = kv - n + i and sees key j <= p, and with a window W only j > p - W or
// j < sinks:
//   s_j = softmax_scale * k_scale * (q . k_code_j),  out = sum_j softmax(s)_j v_scale v_code_j
// lse = log(sum exp s).  A query that sees nothing gives 0 and -inf.
//
// One block per token and query head; each warp takes every fourth key with a
// running maximum and sum (fp32), the lanes split the head, and the warps'
// states are joined at the end.
#include "kv8.cuh"

namespace nvf {

namespace {

constexpr int kWarps = 4;

struct AttentionArgs {
    Kv8CacheArgs c;
    Kv8BatchArgs bt;
    const __nv_bfloat16* q;
    __nv_bfloat16* out;
    float* lse;  // or null
    long long q_stride;
    int heads, group;
    float scale;  // softmax_scale
    int window, sinks;
};

template <int kDim>
__global__ void __launch_bounds__(kWarps * 32) kv8_attention_kernel(const AttentionArgs a) {
    constexpr int kPer = kDim / 32;  // values of the head per lane, as pairs 64 apart
    const int head = blockIdx.y, t = blockIdx.x;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int b = kv8_owner(a.bt, t);
    int hi = 0, lo = 0, sinks = 0;
    if (b < a.bt.batch) {
        const Kv8Seq s = kv8_seq(a.bt, b);
        if (s.bad) kv8_report(a.bt);
        hi = max(s.kv - s.len + (t - s.q0) + 1, 0);
        lo = a.window > 0 ? max(hi - a.window, 0) : 0;
        sinks = min(a.sinks, lo);
    } else {
        kv8_report(a.bt);
    }
    float q[kPer], o[kPer];
    const __nv_bfloat16* qh = a.q + t * a.q_stride + (size_t)head * kDim;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        q[i] = __bfloat162float(qh[i * 32 + lane]);
        o[i] = 0.0f;
    }
    const int size = 1 << a.bt.page_shift, kv_head = head / a.group;
    float m = -INFINITY, l = 0.0f;
    for (int x = warp; x < sinks + hi - lo; x += kWarps) {
        const int j = x < sinks ? x : lo + x - sinks;
        const int page = kv8_page(a.bt, a.c, b, j >> a.bt.page_shift);
        if (page < 0) continue;
        const size_t at = (size_t)page * a.c.kv_heads + kv_head;
        const size_t row = (at << a.bt.page_shift) + (j & (size - 1));
        const uint8_t* k = a.c.k_codes + row * kDim;
        const uint8_t* v = a.c.v_codes + row * kDim;
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) s = fmaf(q[i], e4m3_to_f32(k[i * 32 + lane]), s);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
        s *= a.scale * a.c.k_scales[at];
        const float top = fmaxf(m, s);
        const float base = top == -INFINITY ? 0.0f : top;
        const float keep = expf(m - base), p = expf(s - base);
        const float pv = p * a.c.v_scales[at];
        l = l * keep + p;
        m = top;
#pragma unroll
        for (int i = 0; i < kPer; ++i) o[i] = o[i] * keep + pv * e4m3_to_f32(v[i * 32 + lane]);
    }
    __shared__ float sm[kWarps], sl[kWarps], so[kWarps][kDim];
    if (lane == 0) {
        sm[warp] = m;
        sl[warp] = l;
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) so[warp][i * 32 + lane] = o[i];
    __syncthreads();
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sm[w]);
    const float base = top == -INFINITY ? 0.0f : top;
    float total = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) total += sl[w] * expf(sm[w] - base);
    for (int d = threadIdx.x; d < kDim; d += kWarps * 32) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) v += so[w][d] * expf(sm[w] - base);
        const float r = total == 0.0f ? 0.0f : v / total;
        a.out[((size_t)t * a.heads + head) * kDim + d] = __float2bfloat16_rn(r);
    }
    if (threadIdx.x == 0 && a.lse)
        a.lse[(size_t)t * a.heads + head] = total == 0.0f ? -INFINITY : base + logf(total);
}

}  // namespace

size_t kv8_attention_data_bytes(int head_dim, int num_sms) {
    (void)head_dim;
    (void)num_sms;
    return 256;
}

cudaError_t launch_kv8_attention(const void* q, long long q_stride, int heads,
                                 const Kv8CacheArgs& c, const Kv8BatchArgs& bt,
                                 float softmax_scale, int window, int sinks, void* out, float* lse,
                                 int* counters, void* partials, int num_sms, cudaStream_t s) {
    (void)counters;
    (void)partials;
    (void)num_sms;
    AttentionArgs a;
    a.c = c;
    a.bt = bt;
    a.q = reinterpret_cast<const __nv_bfloat16*>(q);
    a.out = reinterpret_cast<__nv_bfloat16*>(out);
    a.lse = lse;
    a.q_stride = q_stride;
    a.heads = heads;
    a.group = heads / c.kv_heads;
    a.scale = softmax_scale;
    a.window = window;
    a.sinks = sinks;
    const dim3 grid(bt.tokens, heads);
    if (c.head_dim == 64)
        kv8_attention_kernel<64><<<grid, kWarps * 32, 0, s>>>(a);
    else if (c.head_dim == 128)
        kv8_attention_kernel<128><<<grid, kWarps * 32, 0, s>>>(a);
    else
        kv8_attention_kernel<256><<<grid, kWarps * 32, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace nvf
