// w4a4.h -- NVFP4 operands in the tiles that the FP4 tensor cores read, and
// the launchers of the kernels on them.
//
// Both operands of the product are cut into tiles of 128 rows (of a weight, or
// tokens) by 256 K elements, each one contiguous range of kW4Tile bytes, so that a
// bulk copy brings a tile as it lies and no descriptor of the tensor is needed:
//
//   codes   128 rows of 128 bytes, canonical byte order (element 2j in the low
//           nibble of byte j), the 16-byte pieces of a row XORed with row % 8
//           (the 128-byte swizzle of the operand's shared-memory form);
//   scales  per 64 elements 512 bytes: the four E4M3 bytes of row r at
//           (r % 32) * 16 + (r / 32) * 4 (32 tensor-memory lanes of 16 bytes).
//
// Tiles of a row block follow one another along K, zero-padded (zero codes with
// zero scales contribute nothing).  A weight's row count is padded to 256, its
// experts lie one behind the other.  The gate/up pair interleaves 16 rows of gate
// with 16 of up: row r of a tile is feature 64 * tile + 16 * (r / 32) + r % 16, of
// up if r & 16, so that a warp of the epilogue reads both.
#pragma once
#include <cstddef>
#include <cstdint>
#include <cuda_runtime_api.h>

namespace nvf {

constexpr int kW4Rows = 128;
constexpr int kW4K = 256;
constexpr int kW4Codes = kW4Rows * kW4K / 2;      // 16384
constexpr int kW4Scales = kW4Rows * kW4K / 16;    // 2048
constexpr int kW4Tile = kW4Codes + kW4Scales;
constexpr int kW4MaxK = 65536;
constexpr int kW4MaxN = 1 << 20;
constexpr int kW4MaxTokens = 1 << 22;
constexpr int kW4MaxExperts = 1024;

// K blocks, and row blocks of a weight with `streams` rows per feature.
inline __host__ __device__ int w4_k_blocks(int K) { return (K + kW4K - 1) / kW4K; }
inline __host__ __device__ int w4_row_blocks(int N, int streams) {
    return (N * streams + 255) / 256 * 2;
}
// Byte of a code (row r, byte b of its 128 bytes) and of a scale (16-block c of 16).
inline __host__ __device__ int w4_code_at(int r, int b) {
    return r * 128 + ((b >> 4 ^ (r & 7)) << 4) + (b & 15);
}
inline __host__ __device__ int w4_scale_at(int r, int c) {
    return kW4Codes + (c >> 2) * 512 + (r & 31) * 16 + (r >> 5) * 4 + (c & 3);
}

// Rows that belong to experts: rows start[e] .. start[e + 1] - 1 to expert e.  The
// first tile of expert e is start[e] / 128 + e, so that a row's place needs no sum
// over the experts.  start null: one expert with all rows.
struct W4Groups {
    const int* start;  // [experts + 1]
    int experts;
};

// Quantised rows: row blocks of tiles, then one fp32 scale per row.
inline long long w4_token_blocks(int M, int experts) {
    return (M + kW4Rows - 1) / kW4Rows + (experts > 1 ? experts : 0);
}
inline size_t w4_rows_scale_offset(int M, int K, int experts) {
    return (size_t)w4_token_blocks(M, experts) * w4_k_blocks(K) * kW4Tile;
}

// w4a4_rows.cu
cudaError_t launch_w4_repack(const uint8_t* codes, const uint8_t* scales, const uint8_t* codes2,
                             const uint8_t* scales2, int experts, int N, int K, uint8_t* packed,
                             cudaStream_t s);
cudaError_t launch_w4_unpack(const uint8_t* packed, int experts, int N, int K, uint8_t* codes,
                             uint8_t* scales, cudaStream_t s);
cudaError_t launch_w4_quantize(const void* x, int M, int K, const W4Groups& g, void* rows,
                               cudaStream_t s);
// Each token's row, at the places of its choices (ids, place [tokens, choices]).
cudaError_t launch_w4_quantize_routed(const void* x, int tokens, int K, const int* ids,
                                      const int* place, int choices, const W4Groups& g, void* rows,
                                      cudaStream_t s);
cudaError_t launch_w4_dequantize(const void* rows, int M, int K, const W4Groups& g, void* out,
                                 cudaStream_t s);

// w4a4_gemm.cu: out [M, N] bf16; streams 2: the gated product of a gate/up pair
// (N features).  scales a, b: of the weight or of gate and up; lists (one per
// expert, on the device) in their place when not null.
struct W4Product {
    const void* rows;
    const void* packed;
    void* out;
    int M, N, K, streams, act;
    float scale_a, scale_b;
    const float* scales_a;
    const float* scales_b;
    W4Groups groups;
};
size_t w4_partial_bytes(int M, int experts, int num_sms);
cudaError_t launch_w4_gemm(const W4Product& p, int* status, void* partials, int num_sms,
                           cudaStream_t s);

// experts.cu
cudaError_t launch_experts_order(const int* ids, int tokens, int choices, int experts, int* start,
                                 int* source, int* place, cudaStream_t s);
cudaError_t launch_experts_sum(const void* y, int rows, const int* place, const float* weights,
                               int tokens, int choices, int H, void* out, cudaStream_t s);

}  // namespace nvf
