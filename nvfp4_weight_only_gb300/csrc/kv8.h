// kv8.h -- the paged E4M3 key/value cache and a batch of sequences as the
// launchers take them, and the launchers of the attention-side kernels.
#pragma once
#include <cstddef>
#include <cstdint>
#include <cuda_runtime_api.h>

namespace nvf {

// Written to a batch's status word for an index outside its buffers (the
// value of NVFP4_ERR_RANGE).
constexpr int kKv8BadIndex = 4;
// Written to a workspace's status word by an abandoned wait (NVFP4_ERR_TIMEOUT).
constexpr int kKv8Timeout = 7;
constexpr int kKv8MaxBatch = 1024;

struct Kv8CacheArgs {
    uint8_t* k_codes;  // [pages, kv_heads, page, head_dim]
    uint8_t* v_codes;
    float* k_scales;   // [pages, kv_heads]
    float* v_scales;
    int pages, kv_heads, head_dim;
};

struct Kv8BatchArgs {
    const int* q_start;     // [batch + 1]
    const int* kv_len;      // [batch]
    const int* page_table;  // [batch, table_width]
    int* status;            // one word, or null
    int batch, table_width, tokens;
    int page_shift;         // log2 of the page's tokens
    int max_kv;             // table_width pages, in tokens
};

// Most page runs (one page's share of one sequence's new tokens) that `tokens`
// new tokens of `batch` sequences can form.
inline long long kv8_max_runs(long long tokens, long long batch, int page_shift) {
    const long long n = (tokens >> page_shift) + 2 * batch;
    return n < tokens ? n : tokens;
}

struct RopeArgs {
    const float* table;  // [positions][rot / 2][2] (cos, sin), or null
    int positions;       // 2^31 - 1 without a table
    int rot;             // a multiple of 16, 0 without a table
    int interleaved;
};

// kv8_cache.cu
cudaError_t launch_rope_table(int positions, int rot, double base, int scaling, double factor,
                              double context, double slow, double fast, double magnitude,
                              float* table, cudaStream_t s);
cudaError_t launch_kv8_append(const Kv8CacheArgs& c, const Kv8BatchArgs& bt, const void* k,
                              long long k_stride, const void* v, long long v_stride,
                              const void* q, long long q_stride, int heads, void* q_out,
                              const RopeArgs& rope, cudaStream_t s);
cudaError_t launch_kv8_read(const Kv8CacheArgs& c, const Kv8BatchArgs& bt, void* k_out,
                            void* v_out, cudaStream_t s);

// kv8_attention.cu
size_t kv8_attention_data_bytes(int head_dim, long long tokens, int group, int batch,
                                int num_sms);
cudaError_t launch_kv8_attention(const void* q, long long q_stride, int heads,
                                 const Kv8CacheArgs& c, const Kv8BatchArgs& bt,
                                 float softmax_scale, int window, int sinks, void* out, float* lse,
                                 int* status, int* counters, void* partials, int num_sms,
                                 cudaStream_t s);

// rmsnorm.cu: codes null for the bf16 output, else out null; H a multiple of
// 8, at most kNormMaxWidth.
constexpr int kNormMaxWidth = 32768;
cudaError_t launch_add_rmsnorm(const void* x, const void* residual, const void* weight, int M,
                               int H, float eps, float weight_bias, void* sum_out, void* out,
                               uint8_t* codes, float* scales, cudaStream_t s);

}  // namespace nvf
