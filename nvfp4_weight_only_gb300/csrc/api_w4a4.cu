// api_w4a4.cu -- the calls of the C ABI on 4-bit activations (repack, quantise,
// products, FFN, experts): host-side argument validation, workspace carving and
// launch.  No arithmetic of the operators lives here.
#include <cmath>
#include <cstdint>

#include "internal.h"
#include "nvfp4ffn.h"
#include "w4a4.h"

namespace {

constexpr int kFallbackSms = 160;  // for workspace queries without a device
constexpr int kMaxChoices = 64;

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return a && b && x < y + nb && y < x + na;
}

nvfp4_status cuda_status(cudaError_t e) { return e == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA; }

size_t round256(size_t b) { return (b + 255) / 256 * 256; }

int sms_for_sizing() {
    const int n = nvf::device_sm_count();
    return n > 0 ? n : kFallbackSms;
}

bool weight_sizes(int experts, int N, int K) {
    return experts >= 1 && experts <= nvf::kW4MaxExperts && N >= 1 && N <= nvf::kW4MaxN && K >= 16 &&
           K % 16 == 0 && K <= nvf::kW4MaxK;
}

// M = 0 rows and more than the call takes are out of range.
bool row_count(long long M) { return M >= 1 && M <= nvf::kW4MaxTokens; }

nvf::W4Groups groups_of(const w4a4_groups* g) {
    if (!g) return {nullptr, 1};
    return {g->start, g->experts};
}

bool routed_sizes(int tokens, int choices, int experts) {
    return tokens >= 1 && choices >= 1 && choices <= kMaxChoices && experts >= 1 &&
           experts <= nvf::kW4MaxExperts && row_count((long long)tokens * choices);
}

nvfp4_status check_groups(const w4a4_groups* g) {
    if (!g) return NVFP4_OK;
    if (!g->start) return NVFP4_ERR_NULL;
    if (g->experts < 1 || g->experts > nvf::kW4MaxExperts) return NVFP4_ERR_RANGE;
    return aligned(g->start, 4) ? NVFP4_OK : NVFP4_ERR_ALIGN;
}

size_t rows_bytes(int M, int K, int experts) {
    return nvf::w4_rows_scale_offset(M, K, experts) + (size_t)M * 4;
}

size_t gemm_bytes(int M, int experts, int sms) {
    return nvf::kDataOffset + round256(nvf::w4_partial_bytes(M, experts, sms));
}

// What the products' entry points have in common.
struct Product {
    const void* rows;
    int M, K;
    const w4a4_groups* groups;  // null: dense
    const void* packed;
    float scale_a, scale_b;
    const float* scales_a;
    const float* scales_b;
    int N, streams, act;
    void* out;
};

nvfp4_status product(const Product& p, void* ws, size_t ws_bytes, cudaStream_t stream) {
    if (!p.rows || !p.packed || !p.out || !ws) return NVFP4_ERR_NULL;
    if (p.groups && (!p.scales_a || (p.streams == 2 && !p.scales_b))) return NVFP4_ERR_NULL;
    if (!row_count(p.M)) return NVFP4_ERR_RANGE;
    if (p.act != NVFP4_ACT_SILU && p.act != NVFP4_ACT_GELU_TANH) return NVFP4_ERR_RANGE;
    const nvfp4_status g = check_groups(p.groups);
    if (g != NVFP4_OK) return g;
    const nvf::W4Groups groups = groups_of(p.groups);
    if (!weight_sizes(groups.experts, p.N, p.K) || (p.streams == 2 && p.N % 16 != 0))
        return NVFP4_ERR_SHAPE;
    if (!aligned(p.rows, 16) || !aligned(p.packed, 16) || !aligned(p.out, 16) || !aligned(ws, 16) ||
        !aligned(p.scales_a, 4) || !aligned(p.scales_b, 4))
        return NVFP4_ERR_ALIGN;
    const size_t out_bytes = (size_t)p.M * p.N * 2, in_bytes = rows_bytes(p.M, p.K, groups.experts);
    const int sms = nvf::device_sm_count();
    if (sms <= 0) return NVFP4_ERR_CUDA;
    if (ws_bytes < gemm_bytes(p.M, groups.experts, sms)) return NVFP4_ERR_WORKSPACE;
    if (overlap(p.out, out_bytes, p.rows, in_bytes) || overlap(p.out, out_bytes, ws, ws_bytes) ||
        overlap(p.rows, in_bytes, ws, ws_bytes))
        return NVFP4_ERR_ALIAS;
    char* const w = reinterpret_cast<char*>(ws);
    const nvf::W4Product q{p.rows,    p.packed,  p.out,      p.M,        p.N,   p.K, p.streams,
                           p.act,     p.scale_a, p.scale_b,  p.scales_a, p.scales_b, groups};
    return cuda_status(nvf::launch_w4_gemm(q, reinterpret_cast<int*>(w), w + nvf::kDataOffset, sms,
                                           stream));
}

// The FFN's workspace: [status][counters][partial sums][x's rows][h][h's rows], for
// experts then [y][lists].  The products take its front as theirs.
struct FfnLayout {
    size_t front, x_rows, h, h_rows, y, start, source, place, total;
};

FfnLayout ffn_layout(int M, int H, int I, int experts, int sms) {
    FfnLayout l;
    l.front = gemm_bytes(M, experts > 0 ? experts : 1, sms);
    l.x_rows = l.front;
    l.h = l.x_rows + round256(rows_bytes(M, H, experts > 0 ? experts : 1));
    l.h_rows = l.h + round256((size_t)M * I * 2);
    l.y = l.h_rows + round256(rows_bytes(M, I, experts > 0 ? experts : 1));
    l.start = l.y + (experts > 0 ? round256((size_t)M * H * 2) : 0);
    l.source = l.start + (experts > 0 ? round256((size_t)(experts + 1) * 4) : 0);
    l.place = l.source + (experts > 0 ? round256((size_t)M * 4) : 0);
    l.total = l.place + (experts > 0 ? round256((size_t)M * 4) : 0);
    return l;
}

bool ffn_sizes(int H, int I) { return weight_sizes(1, H, I) && weight_sizes(1, I, H); }

}  // namespace

extern "C" {

size_t w4a4_repacked_bytes(int experts, int N, int K) {
    if (!weight_sizes(experts, N, K)) return 0;
    return (size_t)experts * nvf::w4_row_blocks(N, 1) * nvf::w4_k_blocks(K) * nvf::kW4Tile;
}

size_t w4a4_repacked_gate_up_bytes(int experts, int I, int H) {
    if (!weight_sizes(experts, I, H) || I % 16 != 0) return 0;
    return (size_t)experts * nvf::w4_row_blocks(I, 2) * nvf::w4_k_blocks(H) * nvf::kW4Tile;
}

nvfp4_status w4a4_repack(const uint8_t* codes, const uint8_t* scales, int experts, int N, int K,
                         void* packed, cudaStream_t stream) {
    if (!codes || !scales || !packed) return NVFP4_ERR_NULL;
    if (!weight_sizes(experts, N, K)) return NVFP4_ERR_SHAPE;
    if (!aligned(packed, 16)) return NVFP4_ERR_ALIGN;
    return cuda_status(nvf::launch_w4_repack(codes, scales, nullptr, nullptr, experts, N, K,
                                             reinterpret_cast<uint8_t*>(packed), stream));
}

nvfp4_status w4a4_repack_gate_up(const uint8_t* gate_codes, const uint8_t* gate_scales,
                                 const uint8_t* up_codes, const uint8_t* up_scales, int experts,
                                 int I, int H, void* packed, cudaStream_t stream) {
    if (!gate_codes || !gate_scales || !up_codes || !up_scales || !packed) return NVFP4_ERR_NULL;
    if (!weight_sizes(experts, I, H) || I % 16 != 0) return NVFP4_ERR_SHAPE;
    if (!aligned(packed, 16)) return NVFP4_ERR_ALIGN;
    return cuda_status(nvf::launch_w4_repack(gate_codes, gate_scales, up_codes, up_scales, experts,
                                             I, H, reinterpret_cast<uint8_t*>(packed), stream));
}

nvfp4_status w4a4_unpack(const void* packed, int experts, int N, int K, uint8_t* codes,
                         uint8_t* scales, cudaStream_t stream) {
    if (!packed || !codes || !scales) return NVFP4_ERR_NULL;
    if (!weight_sizes(experts, N, K)) return NVFP4_ERR_SHAPE;
    if (!aligned(packed, 16)) return NVFP4_ERR_ALIGN;
    return cuda_status(nvf::launch_w4_unpack(reinterpret_cast<const uint8_t*>(packed), experts, N, K,
                                             codes, scales, stream));
}

size_t w4a4_rows_bytes(int M, int K, int experts) {
    if (!row_count(M) || !weight_sizes(experts, 1, K)) return 0;
    return rows_bytes(M, K, experts);
}

nvfp4_status w4a4_quantize(const void* x, int M, int K, const w4a4_groups* groups, void* rows,
                           cudaStream_t stream) {
    if (!x || !rows) return NVFP4_ERR_NULL;
    if (!row_count(M)) return NVFP4_ERR_RANGE;
    const nvfp4_status v = check_groups(groups);
    if (v != NVFP4_OK) return v;
    const nvf::W4Groups g = groups_of(groups);
    if (!weight_sizes(1, 1, K)) return NVFP4_ERR_SHAPE;
    if (!aligned(x, 16) || !aligned(rows, 16)) return NVFP4_ERR_ALIGN;
    if (overlap(x, (size_t)M * K * 2, rows, rows_bytes(M, K, g.experts)))
        return NVFP4_ERR_ALIAS;
    return cuda_status(nvf::launch_w4_quantize(x, M, K, g, rows, stream));
}

nvfp4_status w4a4_quantize_routed(const void* x, int tokens, int K, const int* ids,
                                  const int* place, int choices, const w4a4_groups* groups,
                                  void* rows, cudaStream_t stream) {
    if (!x || !ids || !place || !groups || !rows) return NVFP4_ERR_NULL;
    if (!routed_sizes(tokens, choices, groups->experts)) return NVFP4_ERR_RANGE;
    const nvfp4_status v = check_groups(groups);
    if (v != NVFP4_OK) return v;
    if (!weight_sizes(1, 1, K)) return NVFP4_ERR_SHAPE;
    if (!aligned(x, 16) || !aligned(rows, 16) || !aligned(ids, 4) || !aligned(place, 4))
        return NVFP4_ERR_ALIGN;
    const nvf::W4Groups g = groups_of(groups);
    const size_t n = rows_bytes(tokens * choices, K, g.experts);
    const size_t lists = (size_t)tokens * choices * 4;
    if (overlap(x, (size_t)tokens * K * 2, rows, n) || overlap(ids, lists, rows, n) ||
        overlap(place, lists, rows, n))
        return NVFP4_ERR_ALIAS;
    return cuda_status(
        nvf::launch_w4_quantize_routed(x, tokens, K, ids, place, choices, g, rows, stream));
}

nvfp4_status w4a4_dequantize(const void* rows, int M, int K, const w4a4_groups* groups, void* out,
                             cudaStream_t stream) {
    if (!rows || !out) return NVFP4_ERR_NULL;
    if (!row_count(M)) return NVFP4_ERR_RANGE;
    const nvfp4_status v = check_groups(groups);
    if (v != NVFP4_OK) return v;
    const nvf::W4Groups g = groups_of(groups);
    if (!weight_sizes(1, 1, K)) return NVFP4_ERR_SHAPE;
    if (!aligned(rows, 16) || !aligned(out, 16)) return NVFP4_ERR_ALIGN;
    if (overlap(out, (size_t)M * K * 2, rows, rows_bytes(M, K, g.experts))) return NVFP4_ERR_ALIAS;
    return cuda_status(nvf::launch_w4_dequantize(rows, M, K, g, out, stream));
}

size_t w4a4_gemm_workspace_bytes(int M, int N, int K, int experts) {
    if (!row_count(M) || !weight_sizes(experts, N, K)) return 0;
    return gemm_bytes(M, experts, sms_for_sizing());
}

nvfp4_status w4a4_gemm(const void* rows, int M, int K, const void* packed_w, float scale2, int N,
                       void* y, void* ws, size_t ws_bytes, cudaStream_t stream) {
    return product({rows, M, K, nullptr, packed_w, scale2, scale2, nullptr, nullptr, N, 1, 0, y}, ws,
                   ws_bytes, stream);
}

nvfp4_status w4a4_gate_up(const void* rows, int M, int H, const void* gate_up_packed,
                          float gate_scale2, float up_scale2, int I, nvfp4_act act, void* h,
                          void* ws, size_t ws_bytes, cudaStream_t stream) {
    return product({rows, M, H, nullptr, gate_up_packed, gate_scale2, up_scale2, nullptr, nullptr, I,
                    2, (int)act, h},
                   ws, ws_bytes, stream);
}

nvfp4_status w4a4_experts_gemm(const void* rows, int M, int K, const w4a4_groups* groups,
                               const void* packed_w, const float* scale2, int N, void* y, void* ws,
                               size_t ws_bytes, cudaStream_t stream) {
    if (!groups) return NVFP4_ERR_NULL;
    return product({rows, M, K, groups, packed_w, 0.0f, 0.0f, scale2, scale2, N, 1, 0, y}, ws,
                   ws_bytes, stream);
}

nvfp4_status w4a4_experts_gate_up(const void* rows, int M, int H, const w4a4_groups* groups,
                                  const void* gate_up_packed, const float* gate_scale2,
                                  const float* up_scale2, int I, nvfp4_act act, void* h, void* ws,
                                  size_t ws_bytes, cudaStream_t stream) {
    if (!groups) return NVFP4_ERR_NULL;
    return product({rows, M, H, groups, gate_up_packed, 0.0f, 0.0f, gate_scale2, up_scale2, I, 2,
                    (int)act, h},
                   ws, ws_bytes, stream);
}

size_t ffn_swiglu_w4a4_workspace_bytes(int M, int H, int I) {
    if (!row_count(M) || !ffn_sizes(H, I)) return 0;
    return ffn_layout(M, H, I, 0, sms_for_sizing()).total;
}

nvfp4_status ffn_swiglu_w4a4(const void* x, int M, int H, int I, const void* gate_up_packed,
                             float gate_scale2, float up_scale2, const void* down_packed,
                             float down_scale2, nvfp4_act act, void* out, void* ws, size_t ws_bytes,
                             cudaStream_t stream) {
    if (!x || !gate_up_packed || !down_packed || !out || !ws) return NVFP4_ERR_NULL;
    if (!row_count(M)) return NVFP4_ERR_RANGE;
    if (act != NVFP4_ACT_SILU && act != NVFP4_ACT_GELU_TANH) return NVFP4_ERR_RANGE;
    if (!ffn_sizes(H, I)) return NVFP4_ERR_SHAPE;
    if (!aligned(x, 16) || !aligned(gate_up_packed, 16) || !aligned(down_packed, 16) ||
        !aligned(out, 16) || !aligned(ws, 16))
        return NVFP4_ERR_ALIGN;
    const int sms = nvf::device_sm_count();
    if (sms <= 0) return NVFP4_ERR_CUDA;
    const FfnLayout l = ffn_layout(M, H, I, 0, sms);
    if (ws_bytes < l.total) return NVFP4_ERR_WORKSPACE;
    const size_t n = (size_t)M * H * 2;
    if (overlap(x, n, out, n) || overlap(x, n, ws, ws_bytes) || overlap(out, n, ws, ws_bytes))
        return NVFP4_ERR_ALIAS;
    char* const w = reinterpret_cast<char*>(ws);
    nvfp4_status e = w4a4_quantize(x, M, H, nullptr, w + l.x_rows, stream);
    if (e != NVFP4_OK) return e;
    e = w4a4_gate_up(w + l.x_rows, M, H, gate_up_packed, gate_scale2, up_scale2, I, act, w + l.h, ws,
                     l.front, stream);
    if (e != NVFP4_OK) return e;
    e = w4a4_quantize(w + l.h, M, I, nullptr, w + l.h_rows, stream);
    if (e != NVFP4_OK) return e;
    return w4a4_gemm(w + l.h_rows, M, I, down_packed, down_scale2, H, out, ws, l.front, stream);
}

nvfp4_status experts_order(const int* ids, int tokens, int choices, int experts, int* start,
                           int* source, int* place, cudaStream_t stream) {
    if (!ids || !start || !source || !place) return NVFP4_ERR_NULL;
    if (!routed_sizes(tokens, choices, experts)) return NVFP4_ERR_RANGE;
    if (!aligned(ids, 4) || !aligned(start, 4) || !aligned(source, 4) || !aligned(place, 4))
        return NVFP4_ERR_ALIGN;
    const size_t n = (size_t)tokens * choices * 4, ns = (size_t)(experts + 1) * 4;
    if (overlap(ids, n, start, ns) || overlap(ids, n, source, n) || overlap(ids, n, place, n) ||
        overlap(start, ns, source, n) || overlap(start, ns, place, n) || overlap(source, n, place, n))
        return NVFP4_ERR_ALIAS;
    return cuda_status(
        nvf::launch_experts_order(ids, tokens, choices, experts, start, source, place, stream));
}

nvfp4_status experts_sum(const void* y, int rows, const int* place, const float* weights, int tokens,
                         int choices, int H, void* out, cudaStream_t stream) {
    if (!y || !place || !weights || !out) return NVFP4_ERR_NULL;
    if (!row_count(rows) || !routed_sizes(tokens, choices, 1)) return NVFP4_ERR_RANGE;
    if (H < 16 || H % 16 != 0 || H > nvf::kW4MaxK) return NVFP4_ERR_SHAPE;
    if (!aligned(y, 16) || !aligned(out, 16) || !aligned(place, 4) || !aligned(weights, 4))
        return NVFP4_ERR_ALIGN;
    const size_t n = (size_t)tokens * H * 2, lists = (size_t)tokens * choices * 4;
    if (overlap(out, n, y, (size_t)rows * H * 2) || overlap(out, n, place, lists) ||
        overlap(out, n, weights, lists))
        return NVFP4_ERR_ALIAS;
    return cuda_status(
        nvf::launch_experts_sum(y, rows, place, weights, tokens, choices, H, out, stream));
}

size_t experts_swiglu_w4a4_workspace_bytes(int tokens, int choices, int experts, int H, int I) {
    if (!routed_sizes(tokens, choices, experts) || !ffn_sizes(H, I)) return 0;
    return ffn_layout(tokens * choices, H, I, experts, sms_for_sizing()).total;
}

nvfp4_status experts_swiglu_w4a4(const void* x, int tokens, int H, int I, const int* ids,
                                 const float* weights, int choices, int experts,
                                 const void* gate_up_packed, const float* gate_scale2,
                                 const float* up_scale2, const void* down_packed,
                                 const float* down_scale2, nvfp4_act act, void* out, void* ws,
                                 size_t ws_bytes, cudaStream_t stream) {
    if (!x || !ids || !weights || !gate_up_packed || !gate_scale2 || !up_scale2 || !down_packed ||
        !down_scale2 || !out || !ws)
        return NVFP4_ERR_NULL;
    if (!routed_sizes(tokens, choices, experts)) return NVFP4_ERR_RANGE;
    if (act != NVFP4_ACT_SILU && act != NVFP4_ACT_GELU_TANH) return NVFP4_ERR_RANGE;
    if (!ffn_sizes(H, I)) return NVFP4_ERR_SHAPE;
    if (!aligned(x, 16) || !aligned(gate_up_packed, 16) || !aligned(down_packed, 16) ||
        !aligned(out, 16) || !aligned(ws, 16) || !aligned(ids, 4) || !aligned(weights, 4) ||
        !aligned(gate_scale2, 4) || !aligned(up_scale2, 4) || !aligned(down_scale2, 4))
        return NVFP4_ERR_ALIGN;
    const int sms = nvf::device_sm_count();
    if (sms <= 0) return NVFP4_ERR_CUDA;
    const int M = tokens * choices;
    const FfnLayout l = ffn_layout(M, H, I, experts, sms);
    if (ws_bytes < l.total) return NVFP4_ERR_WORKSPACE;
    const size_t n = (size_t)tokens * H * 2, lists = (size_t)M * 4;
    if (overlap(x, n, out, n) || overlap(x, n, ws, ws_bytes) || overlap(out, n, ws, ws_bytes) ||
        overlap(ids, lists, out, n) || overlap(weights, lists, out, n) ||
        overlap(ids, lists, ws, ws_bytes) || overlap(weights, lists, ws, ws_bytes))
        return NVFP4_ERR_ALIAS;
    char* const w = reinterpret_cast<char*>(ws);
    int* const start = reinterpret_cast<int*>(w + l.start);
    int* const source = reinterpret_cast<int*>(w + l.source);
    int* const place = reinterpret_cast<int*>(w + l.place);
    nvfp4_status e = experts_order(ids, tokens, choices, experts, start, source, place, stream);
    if (e != NVFP4_OK) return e;
    const w4a4_groups same{start, experts};
    e = w4a4_quantize_routed(x, tokens, H, ids, place, choices, &same, w + l.x_rows, stream);
    if (e != NVFP4_OK) return e;
    e = w4a4_experts_gate_up(w + l.x_rows, M, H, &same, gate_up_packed, gate_scale2, up_scale2, I,
                             act, w + l.h, ws, l.front, stream);
    if (e != NVFP4_OK) return e;
    e = w4a4_quantize(w + l.h, M, I, &same, w + l.h_rows, stream);
    if (e != NVFP4_OK) return e;
    e = w4a4_experts_gemm(w + l.h_rows, M, I, &same, down_packed, down_scale2, H, w + l.y, ws,
                          l.front, stream);
    if (e != NVFP4_OK) return e;
    return experts_sum(w + l.y, M, place, weights, tokens, choices, H, out, stream);
}

}  // extern "C"
