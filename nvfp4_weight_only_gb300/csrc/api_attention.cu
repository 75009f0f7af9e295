// api_attention.cu -- the attention-side calls of the C ABI (norm, rotary
// table, cache append and read, attention): host-side argument validation and
// launch.  No arithmetic of the operators lives here.
#include <cmath>
#include <cstdint>

#include "internal.h"
#include "kv8.h"
#include "nvfp4ffn.h"

namespace {

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Whether [a, a + na) and [b, b + nb) share a byte (null shares none).
bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    if (!a || !b) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

// Overlap other than being the same buffer (elementwise calls may run in place).
bool partly(const void* a, const void* b, size_t n) { return a != b && overlap(a, n, b, n); }

nvfp4_status cuda_status(cudaError_t e) { return e == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA; }

// Bytes that T rows of `width` bf16 values, `stride` values apart, reach over.
size_t reach(int T, long long stride, size_t width) {
    return ((size_t)(T - 1) * (size_t)stride + width) * 2;
}

nvfp4_status check_cache_sizes(const kv8_cache* c) {
    if (c->pages < 1 || c->kv_heads < 1) return NVFP4_ERR_SHAPE;
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return NVFP4_ERR_SHAPE;
    if (c->page < 16 || c->page > 256 || (c->page & (c->page - 1))) return NVFP4_ERR_SHAPE;
    return NVFP4_OK;
}

nvfp4_status check_cache(const kv8_cache* c) {
    if (!c || !c->k_codes || !c->v_codes || !c->k_scales || !c->v_scales) return NVFP4_ERR_NULL;
    const nvfp4_status e = check_cache_sizes(c);
    if (e != NVFP4_OK) return e;
    if (!aligned(c->k_codes, 16) || !aligned(c->v_codes, 16) || !aligned(c->k_scales, 4) ||
        !aligned(c->v_scales, 4))
        return NVFP4_ERR_ALIGN;
    return NVFP4_OK;
}

nvfp4_status check_batch_sizes(const kv8_batch* b, const kv8_cache* c, int tokens) {
    if (b->batch < 1 || b->batch > nvf::kKv8MaxBatch || tokens < 1) return NVFP4_ERR_RANGE;
    if (b->table_width < 1 || (long long)b->table_width * c->page > 0x7fffff00LL)
        return NVFP4_ERR_SHAPE;
    return NVFP4_OK;
}

nvfp4_status check_batch(const kv8_batch* b, const kv8_cache* c, int tokens) {
    if (!b || !b->q_start || !b->kv_len || !b->page_table) return NVFP4_ERR_NULL;
    const nvfp4_status e = check_batch_sizes(b, c, tokens);
    if (e != NVFP4_OK) return e;
    if (!aligned(b->q_start, 4) || !aligned(b->kv_len, 4) || !aligned(b->page_table, 4) ||
        !aligned(b->status, 4))
        return NVFP4_ERR_ALIGN;
    return NVFP4_OK;
}

// Query heads of the call: a multiple of the cache's, and rows that the kernels count.
nvfp4_status check_heads(const kv8_cache* c, int tokens, int heads) {
    if (heads < 1 || heads % c->kv_heads != 0) return NVFP4_ERR_SHAPE;
    return (long long)tokens * (heads / c->kv_heads) > (1LL << 30) ? NVFP4_ERR_RANGE : NVFP4_OK;
}

nvf::Kv8CacheArgs cache_args(const kv8_cache* c) {
    return {reinterpret_cast<uint8_t*>(c->k_codes),
            reinterpret_cast<uint8_t*>(c->v_codes),
            c->k_scales,
            c->v_scales,
            c->pages,
            c->kv_heads,
            c->head_dim};
}

nvf::Kv8BatchArgs batch_args(const kv8_batch* b, const kv8_cache* c, int tokens) {
    int shift = 4;
    while ((1 << shift) < c->page) ++shift;
    return {b->q_start, b->kv_len,      b->page_table, b->status,           b->batch,
            b->table_width, tokens, shift,         b->table_width * c->page};
}

// Rows of `heads` heads `stride` values apart: vector loads want 16 bytes.
nvfp4_status check_rows(const void* p, int heads, long long stride, int dim) {
    if (stride < (long long)heads * dim || stride % 8 != 0 || stride > (1LL << 40))
        return NVFP4_ERR_SHAPE;
    return aligned(p, 16) ? NVFP4_OK : NVFP4_ERR_ALIGN;
}

nvfp4_status check_norm(const void* x, const void* residual, const void* weight, int M, int H,
                        float eps, const void* sum_out) {
    if (!x || !weight) return NVFP4_ERR_NULL;
    if (M < 1 || H < 16 || H % 16 != 0 || H > nvf::kNormMaxWidth) return NVFP4_ERR_SHAPE;
    if (!(eps >= 0.0f) || !std::isfinite(eps)) return NVFP4_ERR_RANGE;
    if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(weight, 16) || !aligned(sum_out, 16))
        return NVFP4_ERR_ALIGN;
    const size_t n = (size_t)M * H * 2;
    if (partly(sum_out, x, n) || partly(sum_out, residual, n) ||
        overlap(sum_out, n, weight, (size_t)H * 2))
        return NVFP4_ERR_ALIAS;
    return NVFP4_OK;
}

}  // namespace

extern "C" {

nvfp4_status add_rmsnorm_bf16(const void* x, const void* residual, const void* weight, int M,
                              int H, float eps, float weight_bias, void* sum_out, void* out,
                              cudaStream_t stream) {
    const nvfp4_status v = check_norm(x, residual, weight, M, H, eps, sum_out);
    if (!out) return NVFP4_ERR_NULL;
    if (v != NVFP4_OK) return v;
    if (!aligned(out, 16)) return NVFP4_ERR_ALIGN;
    const size_t n = (size_t)M * H * 2;
    if (partly(out, x, n) || partly(out, residual, n) || overlap(out, n, sum_out, n) ||
        overlap(out, n, weight, (size_t)H * 2))
        return NVFP4_ERR_ALIAS;
    return cuda_status(nvf::launch_add_rmsnorm(x, residual, weight, M, H, eps, weight_bias,
                                               sum_out, out, nullptr, nullptr, stream));
}

nvfp4_status add_rmsnorm_e4m3(const void* x, const void* residual, const void* weight, int M,
                              int H, float eps, float weight_bias, void* sum_out, uint8_t* codes,
                              float* scales, cudaStream_t stream) {
    const nvfp4_status v = check_norm(x, residual, weight, M, H, eps, sum_out);
    if (!codes || !scales) return NVFP4_ERR_NULL;
    if (v != NVFP4_OK) return v;
    if (!aligned(codes, 16) || !aligned(scales, 4)) return NVFP4_ERR_ALIGN;
    const size_t n = (size_t)M * H, ns = (size_t)M * ((H + 127) / 128) * 4;
    const void* in[3] = {x, residual, sum_out};
    for (const void* p : in)
        if (overlap(codes, n, p, 2 * n) || overlap(scales, ns, p, 2 * n)) return NVFP4_ERR_ALIAS;
    if (overlap(codes, n, scales, ns) || overlap(codes, n, weight, (size_t)H * 2) ||
        overlap(scales, ns, weight, (size_t)H * 2))
        return NVFP4_ERR_ALIAS;
    return cuda_status(nvf::launch_add_rmsnorm(x, residual, weight, M, H, eps, weight_bias,
                                               sum_out, nullptr, codes, scales, stream));
}

nvfp4_status rope_table(int positions, int rot_dim, double base, rope_scaling scaling,
                        double factor, double context, double slow, double fast, double magnitude,
                        float* table, cudaStream_t stream) {
    if (!table) return NVFP4_ERR_NULL;
    if (positions < 1 || rot_dim < 16 || rot_dim > 256 || rot_dim % 16 != 0)
        return NVFP4_ERR_SHAPE;
    if (!aligned(table, 16)) return NVFP4_ERR_ALIGN;
    if ((int)scaling < ROPE_PLAIN || (int)scaling > ROPE_RAMP) return NVFP4_ERR_RANGE;
    if (!(base > 1.0) || !std::isfinite(base) || !std::isfinite(magnitude))
        return NVFP4_ERR_RANGE;
    if (scaling != ROPE_PLAIN && (!(factor > 0.0) || !std::isfinite(factor)))
        return NVFP4_ERR_RANGE;
    if (scaling == ROPE_RAMP &&
        (!(context > 0.0) || !(slow >= 0.0) || !(fast > slow) || !std::isfinite(context) ||
         !std::isfinite(fast)))
        return NVFP4_ERR_RANGE;
    return cuda_status(nvf::launch_rope_table(positions, rot_dim, base, (int)scaling, factor,
                                              context, slow, fast, magnitude, table, stream));
}

nvfp4_status kv8_append(const kv8_cache* cache, const kv8_batch* batch, int tokens, const void* k,
                        int64_t k_stride, const void* v, int64_t v_stride, const void* q,
                        int64_t q_stride, int heads, void* q_out, const float* rope,
                        int rope_positions, int rot_dim, int interleaved, cudaStream_t stream) {
    nvfp4_status e = check_cache(cache);
    if (e == NVFP4_OK) e = check_batch(batch, cache, tokens);
    if (e != NVFP4_OK) return e;
    if (!k || !v || (q == nullptr) != (q_out == nullptr)) return NVFP4_ERR_NULL;
    const int dim = cache->head_dim;
    e = check_rows(k, cache->kv_heads, k_stride, dim);
    if (e == NVFP4_OK) e = check_rows(v, cache->kv_heads, v_stride, dim);
    if (e != NVFP4_OK) return e;
    if (q) {
        if (heads < 1) return NVFP4_ERR_SHAPE;
        e = check_rows(q, heads, q_stride, dim);
        if (e != NVFP4_OK) return e;
        if (!aligned(q_out, 16)) return NVFP4_ERR_ALIGN;
        const size_t qw = (size_t)heads * dim, n = (size_t)tokens * qw * 2;
        const size_t kw = (size_t)cache->kv_heads * dim;
        // in place only when q has q_out's layout
        const bool in_place = q == q_out && q_stride == (int64_t)qw;
        if ((!in_place && overlap(q_out, n, q, reach(tokens, q_stride, qw))) ||
            overlap(q_out, n, k, reach(tokens, k_stride, kw)) ||
            overlap(q_out, n, v, reach(tokens, v_stride, kw)))
            return NVFP4_ERR_ALIAS;
    }
    nvf::RopeArgs r{rope, 0x7fffffff, 0, interleaved ? 1 : 0};
    if (rope) {
        if (rope_positions < 1 || rot_dim < 16 || rot_dim % 16 != 0 || rot_dim > dim)
            return NVFP4_ERR_SHAPE;
        if (!aligned(rope, 16)) return NVFP4_ERR_ALIGN;
        r.positions = rope_positions;
        r.rot = rot_dim;
    }
    return cuda_status(nvf::launch_kv8_append(cache_args(cache), batch_args(batch, cache, tokens),
                                              k, k_stride, v, v_stride, q, q_stride, heads, q_out,
                                              r, stream));
}

nvfp4_status kv8_read(const kv8_cache* cache, const kv8_batch* batch, int tokens, void* k_out,
                      void* v_out, cudaStream_t stream) {
    nvfp4_status e = check_cache(cache);
    if (e == NVFP4_OK) e = check_batch(batch, cache, tokens);
    if (e != NVFP4_OK) return e;
    if (!k_out || !v_out) return NVFP4_ERR_NULL;
    if (!aligned(k_out, 16) || !aligned(v_out, 16)) return NVFP4_ERR_ALIGN;
    const size_t n = (size_t)tokens * cache->kv_heads * cache->head_dim * 2;
    if (overlap(k_out, n, v_out, n)) return NVFP4_ERR_ALIAS;
    return cuda_status(nvf::launch_kv8_read(cache_args(cache), batch_args(batch, cache, tokens),
                                            k_out, v_out, stream));
}

size_t kv8_attention_workspace_bytes(const kv8_cache* cache, const kv8_batch* batch, int tokens,
                                     int heads) {
    if (!cache || !batch || check_cache_sizes(cache) != NVFP4_OK ||
        check_batch_sizes(batch, cache, tokens) != NVFP4_OK ||
        check_heads(cache, tokens, heads) != NVFP4_OK)
        return 0;
    const int sms = nvf::device_sm_count();
    return nvf::kDataOffset +
           nvf::kv8_attention_data_bytes(cache->head_dim, tokens, heads / cache->kv_heads,
                                         batch->batch, sms > 0 ? sms : 160);
}

nvfp4_status kv8_attention(const void* q, int64_t q_stride, int tokens, int heads,
                           const kv8_cache* cache, const kv8_batch* batch, float softmax_scale,
                           int window, int sinks, void* out, float* lse, void* ws, size_t ws_bytes,
                           cudaStream_t stream) {
    nvfp4_status e = check_cache(cache);
    if (e == NVFP4_OK) e = check_batch(batch, cache, tokens);
    if (e != NVFP4_OK) return e;
    if (!q || !out || !ws) return NVFP4_ERR_NULL;
    const int dim = cache->head_dim;
    e = check_heads(cache, tokens, heads);
    if (e != NVFP4_OK) return e;
    if (window < 0 || sinks < 0 || !std::isfinite(softmax_scale)) return NVFP4_ERR_RANGE;
    e = check_rows(q, heads, q_stride, dim);
    if (e != NVFP4_OK) return e;
    if (!aligned(out, 16) || !aligned(lse, 4) || !aligned(ws, 16)) return NVFP4_ERR_ALIGN;
    const size_t n = (size_t)tokens * heads * dim * 2, nl = (size_t)tokens * heads * 4;
    const size_t nq = reach(tokens, q_stride, (size_t)heads * dim);
    if (overlap(out, n, q, nq) || overlap(lse, nl, q, nq) || overlap(lse, nl, out, n))
        return NVFP4_ERR_ALIAS;
    const int sms = nvf::device_sm_count();
    if (sms <= 0) return NVFP4_ERR_CUDA;
    if (ws_bytes < nvf::kDataOffset + nvf::kv8_attention_data_bytes(
                                          dim, tokens, heads / cache->kv_heads, batch->batch, sms))
        return NVFP4_ERR_WORKSPACE;
    char* w = reinterpret_cast<char*>(ws);
    return cuda_status(nvf::launch_kv8_attention(
        q, q_stride, heads, cache_args(cache), batch_args(batch, cache, tokens), softmax_scale,
        window, sinks, out, lse, reinterpret_cast<int*>(w),
        reinterpret_cast<int*>(w + nvf::kStatusBytes), w + nvf::kDataOffset, sms, stream));
}

nvfp4_status kv8_batch_status(const kv8_batch* batch, cudaStream_t stream) {
    if (!batch || !batch->status) return NVFP4_ERR_NULL;
    if (!aligned(batch->status, 4)) return NVFP4_ERR_ALIGN;
    int v = 0;
    if (cudaMemcpyAsync(&v, batch->status, 4, cudaMemcpyDeviceToHost, stream) != cudaSuccess ||
        cudaStreamSynchronize(stream) != cudaSuccess ||
        cudaMemsetAsync(batch->status, 0, 4, stream) != cudaSuccess ||
        cudaStreamSynchronize(stream) != cudaSuccess)
        return NVFP4_ERR_CUDA;
    return v == 0 ? NVFP4_OK : NVFP4_ERR_RANGE;
}

}  // extern "C"
