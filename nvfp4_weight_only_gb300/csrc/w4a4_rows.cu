// w4a4_rows.cu -- NVFP4 operands into the tiles of w4a4.h: weights once, by
// moving bytes; activation rows at every call, by quantising them.
//
// A row of x becomes r (2^e with the smallest e that keeps max|x| <= 2688 r, in
// -100..117), per 16 values s = E4M3(max|x| / 6 / r), and codes E2M1(x / (s r)).
// x / r is exact, so the two roundings are of quotients of bf16 values: by 6, and by s.
// Both are products with a rounded reciprocal, off by 2^-22 of themselves at most, which
// are then rounded to a grid that the ties of the codes lie on: a quotient that is a tie
// lands on it, and one that is not stays on its side.  For E4M3 (ties of 5 bits) max|x|
// and 6 times a tie are both 8-bit numbers, so unequal ones are 2^-8 apart; the grid has
// 13 bits.  For E2M1 (ties are multiples of 1/4 up to 5) a quotient is 2^-10 or more away
// from a tie that it is not; the grid is 2^-14 (768 is added and taken away).  So codes
// are those of the exact quotients, without a division.
#include <algorithm>

#include "internal.h"
#include "kv8.cuh"
#include "w4a4.h"

namespace nvf {

namespace {

constexpr int kThreads = 256;
constexpr int kMinExp = -100, kMaxExp = 117;
constexpr int kRowsAtOnce = 4;  // of a block, a warp each, that are short

// One thread per 16 code bytes of a tile (two scale bytes with them).
__global__ void __launch_bounds__(kThreads) repack_kernel(
    const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
    const uint8_t* __restrict__ codes2, const uint8_t* __restrict__ scales2, long long total, int N,
    int K, int row_blocks, int k_blocks, uint8_t* __restrict__ packed) {
    for (long long idx = blockIdx.x * (long long)kThreads + threadIdx.x; idx < total;
         idx += (long long)gridDim.x * kThreads) {
        const int piece = (int)(idx & 7), r = (int)(idx >> 3 & 127);
        const long long tile = idx >> 10;
        const int kb = (int)(tile % k_blocks);
        const long long rb = tile / k_blocks;
        const long long expert = rb / row_blocks;
        const int block = (int)(rb % row_blocks);
        const bool second = codes2 && (r & 16);
        const int n = codes2 ? block * 64 + (r >> 5) * 16 + (r & 15) : block * 128 + r;
        const int k = kb * kW4K + piece * 32;
        uint8_t* out = packed + tile * kW4Tile;
        uint4 w = make_uint4(0, 0, 0, 0);
        uint32_t sc = 0;
        if (n < N && k < K) {
            const long long row = expert * N + n;
            const uint8_t* c = (second ? codes2 : codes) + row * (K / 2) + k / 2;
            const uint8_t* s = (second ? scales2 : scales) + row * (K / 16) + k / 16;
            // K is a multiple of 16: 8 bytes or 16 of this piece are there
            uint32_t v[4] = {0, 0, 0, 0};
            const int have = K - k >= 32 ? 4 : 2;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < have)
                    v[i] = c[4 * i] | c[4 * i + 1] << 8 | c[4 * i + 2] << 16 |
                           (uint32_t)c[4 * i + 3] << 24;
            w = make_uint4(v[0], v[1], v[2], v[3]);
            sc = s[0] | (have == 4 ? s[1] << 8 : 0);
        }
        *reinterpret_cast<uint4*>(out + w4_code_at(r, piece * 16)) = w;
        *reinterpret_cast<uint16_t*>(out + w4_scale_at(r, piece * 2)) = (uint16_t)sc;
    }
}

__global__ void __launch_bounds__(kThreads) unpack_kernel(const uint8_t* __restrict__ packed,
                                                          long long total, int N, int K,
                                                          int row_blocks, int k_blocks,
                                                          uint8_t* __restrict__ codes,
                                                          uint8_t* __restrict__ scales) {
    const int blocks = K / 16;
    for (long long idx = blockIdx.x * (long long)kThreads + threadIdx.x; idx < total;
         idx += (long long)gridDim.x * kThreads) {
        const int b = (int)(idx % blocks);
        const long long row = idx / blocks;
        const int n = (int)(row % N);
        const uint8_t* tile =
            packed +
            ((row / N * row_blocks + n / kW4Rows) * k_blocks + b / 16) * (long long)kW4Tile;
        const int r = n % kW4Rows;
        for (int i = 0; i < 8; ++i)
            codes[row * (K / 2) + b * 8 + i] = tile[w4_code_at(r, (b % 16) * 8 + i)];
        scales[row * blocks + b] = tile[w4_scale_at(r, b % 16)];
    }
}

// The place of a row of an expert whose rows begin at `first`.
__device__ __forceinline__ void place_of(int row, int expert, int first, long long& block, int& r) {
    const int i = row - first;
    block = first / kW4Rows + expert + i / kW4Rows;
    r = i % kW4Rows;
}

// The expert of a row and its place; false for a row of none.  A whole warp calls it.
__device__ __forceinline__ bool find_place(const W4Groups& g, int row, long long& block, int& r) {
    int expert = 0, first = 0;
    if (g.start) {
        // the last expert that starts at or before the row: empty ones in front of it
        // start there too
        int before = 0;
        for (int base = 0; base < g.experts; base += 32) {
            const int e = base + (threadIdx.x & 31);
            before += __popc(__ballot_sync(0xffffffffu, e < g.experts && g.start[e] <= row));
        }
        expert = before - 1;
        if (expert < 0) return false;
        first = g.start[expert];
        if (first < 0 || first > row || row >= g.start[expert + 1]) return false;
    }
    place_of(row, expert, first, block, r);
    return true;
}

// Four pairs of quotients -> eight codes, the first in the low nibble.
__device__ __forceinline__ uint32_t e2m1x8(const float (&q)[8]) {
    uint32_t w;
    asm("{\n .reg .b8 a, b, c, d;\n"
        " cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
        " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
        " mov.b32 %0, {a, b, c, d};\n}"
        : "=r"(w)
        : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]), "f"(q[6]), "f"(q[7]));
    return w;
}

// 1 / v, off by one unit of the last place at most.
__device__ __forceinline__ float reciprocal(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// The larger magnitudes of two pairs of bf16 (of either sign), NaN if either is.
__device__ __forceinline__ uint32_t max2_abs(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// 16 values, 32 bytes; whole says that they are aligned so.
__device__ __forceinline__ void load16(const uint4* at, bool whole, uint32_t (&v)[8]) {
    if (whole) {
        asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]),
                       "=r"(v[6]), "=r"(v[7])
                     : "l"(at));
    } else {
        const uint4 a = at[0], b = at[1];
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
        v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
}

// Where a row goes: its expert's place for it, or those of a token's choices.
struct Places {
    W4Groups groups;
    const int* ids;    // routed: [tokens, choices], with each pair's row in `place`
    const int* place;
    int choices;       // 0: not routed
    int rows;
};

// A choice of a token: its expert (-1 for none, or one out of range), its row and the
// expert's first.
struct Choice {
    int expert, row, first;
};

__device__ __forceinline__ Choice choice_of(const Places& to, int token, int j) {
    const size_t at = (size_t)token * to.choices + j;
    Choice c{to.ids[at], to.place[at], 0};
    if (c.expert < 0 || c.expert >= to.groups.experts || c.row < 0 || c.row >= to.rows)
        return {-1, 0, 0};
    c.first = to.groups.start[c.expert];
    if (c.first < 0 || c.first > c.row) c.expert = -1;
    return c;
}

// One block per row of x, or one warp; a warp takes 512 values at a time, 16 per lane (a
// block with its scale), which stay in registers between the row's maximum and the codes,
// so x is read once.  A token's codes are written to the places of all of its choices.
//
// Bound by memory (4096 rows of 17408: 30.0 us, 6.1 TB/s; 16384 of 2048: 14.2, 6.1).  With
// 8 values per lane, two lanes to a scale, it issued 96 instructions for them, in two of
// three cycles, and took 35.5 and 18.5 us.  56 registers let four blocks of 9 warps share
// an SM (30.5 us without).
template <int kIter, bool kRowPerWarp>
__global__ void __maxnreg__(56)
    quantize_kernel(const uint4* __restrict__ x, int K, int k_blocks, const Places to, int count,
                    uint8_t* __restrict__ rows, float* __restrict__ row_scales) {
    // The decode products read their weights as soon as they are launched, so the next kernel
    // is launched when all kernels in front of this one are done.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31, vecs = K / 16;
    // the row's warps, and which of them this one is
    const int warps = kRowPerWarp ? 1 : blockDim.x / 32, warp = kRowPerWarp ? 0 : threadIdx.x / 32;
    const int row = kRowPerWarp ? blockIdx.x * kRowsAtOnce + threadIdx.x / 32 : blockIdx.x;
    if (row >= count) return;
    const uint4* const src = x + (size_t)row * (K / 8);
    const bool whole = (reinterpret_cast<uintptr_t>(x) & 31) == 0;
    uint32_t v[kIter][8];
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
        const int c = (warp + i * warps) * 32 + lane;
        if (c < vecs) {
            load16(src + 2 * c, whole, v[i]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = 0;
        }
    }
    // the lists are read beside x: lane j looks up choice j
    Choice choice{-1, 0, 0};
    if (lane < to.choices) choice = choice_of(to, row, lane);
    long long block = 0;
    int r = 0;
    if (to.choices == 0 && !find_place(to.groups, row, block, r)) return;
    // the largest of each block, as bf16: as integers, magnitudes keep their order, NaN on top
    uint32_t top[kIter], most = 0;
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
        const uint32_t m =
            max2_abs(max2_abs(max2_abs(v[i][0], v[i][1]), max2_abs(v[i][2], v[i][3])),
                     max2_abs(max2_abs(v[i][4], v[i][5]), max2_abs(v[i][6], v[i][7])));
        top[i] = max(m & 0x7fffu, m >> 16 & 0x7fffu);
        most = max(most, top[i]);
    }
    uint32_t amax = __reduce_max_sync(0xffffffffu, most);
    if constexpr (!kRowPerWarp) {
        __shared__ uint32_t part[32];
        if (lane == 0) part[warp] = amax;
        __syncthreads();
        amax = __reduce_max_sync(0xffffffffu, lane < warps ? part[lane] : 0);
    }
    int e = 0;  // of r
    if (amax) {
        // 2688 = 1.3125 * 2^11, and 0x3fa8 is 1.3125
        const int exponent = max((int)(amax >> 7), 1) - 127;
        e = exponent - 11 + ((amax & 0x7f) > (0x3fa8 & 0x7f) ? 1 : 0);
        e = min(max(e, kMinExp), kMaxExp);
    }
    const float scale = amax >= 0x7f80 ? __uint_as_float(0x7fffffffu)
                                       : __uint_as_float((uint32_t)(e + 127) << 23);
    const float down = __uint_as_float((uint32_t)(127 - e) << 23);  // 1 / r
    const float sixth_down = down * (1.0f / 6.0f);
    // codes in place of x, scales of 64 values in every fourth lane
    uint32_t scales[kIter];
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
        const uint32_t sixth = __float_as_uint(__uint_as_float(top[i] << 16) * sixth_down);
        // (of a row with a NaN anything without a sign)
        const uint32_t code = f32_to_e4m3(__uint_as_float((sixth + 0x400u) & ~0x7ffu)) & 0x7fu;
        const float by = code ? reciprocal(e4m3_to_f32(code)) * down : 0.0f;
        const uint64_t by2 = pair(by, by), grid = pair(768.0f, 768.0f), back = pair(-768.0f, -768.0f);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float q[8];
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                const uint32_t w = v[i][4 * h + p];
                const float2 y = unpair(add2(fma2(pair(bf16_lo(w), bf16_hi(w)), by2, grid), back));
                q[2 * p] = y.x;
                q[2 * p + 1] = y.y;
            }
            v[i][h] = e2m1x8(q);
        }
        uint32_t sc = code;
        sc |= __shfl_down_sync(0xffffffffu, sc, 1) << 8;
        sc |= __shfl_down_sync(0xffffffffu, sc, 2) << 16;
        scales[i] = sc;
    }
    auto write = [&](int at_row) {
        if (warp == 0 && lane == 0) row_scales[at_row] = scale;
        // a warp's values are those of two tiles
        const int kb0 = 2 * warp + lane / 16;
        uint8_t* tile = rows + ((size_t)block * k_blocks + kb0) * kW4Tile;
        const int code_at = w4_code_at(r, lane % 16 * 8), scale_at = w4_scale_at(r, lane % 16);
#pragma unroll
        for (int i = 0; i < kIter; ++i) {
            if (kb0 + 2 * i * warps < k_blocks) {
                *reinterpret_cast<uint2*>(tile + code_at) = make_uint2(v[i][0], v[i][1]);
                if (lane % 4 == 0) *reinterpret_cast<uint32_t*>(tile + scale_at) = scales[i];
            }
            tile += (size_t)2 * warps * kW4Tile;
        }
    };
    if (to.choices == 0) {
        write(row);
        return;
    }
    for (int j = 0; j < to.choices; ++j) {
        const Choice c = j < 32 ? choice : choice_of(to, row, j);
        const int from_lane = j < 32 ? j : lane;
        const int expert = __shfl_sync(0xffffffffu, c.expert, from_lane);
        const int at_row = __shfl_sync(0xffffffffu, c.row, from_lane);
        const int first = __shfl_sync(0xffffffffu, c.first, from_lane);
        if (expert < 0) continue;
        place_of(at_row, expert, first, block, r);
        write(at_row);
    }
}

// The values that the codes stand for: scale, block scale and code have 7 bits
// together, so bf16 holds them exactly (between its least and largest value).
__global__ void __launch_bounds__(kThreads) dequantize_kernel(const uint8_t* __restrict__ rows,
                                                              const float* __restrict__ row_scales,
                                                              int K, int k_blocks,
                                                              const W4Groups g,
                                                              uint4* __restrict__ out) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int row = blockIdx.x;
    long long block;
    int r;
    if (!find_place(g, row, block, r)) return;
    const float scale = row_scales[row];
    for (int c = threadIdx.x; c < K / 8; c += blockDim.x) {
        const uint8_t* tile = rows + ((size_t)block * k_blocks + c / 32) * kW4Tile;
        const uint32_t w = *reinterpret_cast<const uint32_t*>(tile + w4_code_at(r, c % 32 * 4));
        const float s = e4m3_to_f32(tile[w4_scale_at(r, c % 32 / 2)]);
        uint32_t h[4], o[4];
        e2m1x8_to_f16x2x4(w, h[0], h[1], h[2], h[3]);
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[p]));
            o[p] = bf16x2(f.x * s * scale, f.y * s * scale);
        }
        out[(size_t)row * (K / 8) + c] = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

template <typename... Args>
cudaError_t launch(void (*kernel)(Args...), int blocks, int threads, cudaStream_t s,
                   Args... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(threads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

int grid_of(long long work) {
    const long long want = (work + kThreads - 1) / kThreads;
    return (int)std::min(want, 16LL * std::max(1, device_sm_count()));
}

}  // namespace

cudaError_t launch_w4_repack(const uint8_t* codes, const uint8_t* scales, const uint8_t* codes2,
                             const uint8_t* scales2, int experts, int N, int K, uint8_t* packed,
                             cudaStream_t s) {
    const int row_blocks = w4_row_blocks(N, codes2 ? 2 : 1), k_blocks = w4_k_blocks(K);
    const long long total = (long long)experts * row_blocks * k_blocks * 1024;
    repack_kernel<<<grid_of(total), kThreads, 0, s>>>(codes, scales, codes2, scales2, total, N, K,
                                                      row_blocks, k_blocks, packed);
    return cudaGetLastError();
}

cudaError_t launch_w4_unpack(const uint8_t* packed, int experts, int N, int K, uint8_t* codes,
                             uint8_t* scales, cudaStream_t s) {
    const long long total = (long long)experts * N * (K / 16);
    unpack_kernel<<<grid_of(total), kThreads, 0, s>>>(packed, total, N, K, w4_row_blocks(N, 1),
                                                      w4_k_blocks(K), codes, scales);
    return cudaGetLastError();
}

namespace {

cudaError_t quantize(const void* x, int count, int M, int K, const Places& to, void* rows,
                     cudaStream_t s) {
    const int k_blocks = w4_k_blocks(K);
    // A row per warp as long as 4 passes hold it, four rows to a block, with no barrier and
    // fewer blocks to start (16384 rows of 2048 14.2 us, with a block of two warps each 17.1;
    // 8192 of 528: 3.5, 8.9).  Longer ones two warps, as long as 8 passes hold it: small
    // blocks, whose loads and stores overlap others'.  Few rows, as many as SMs, leave room
    // for eight, each with less to write (64 tokens of 4096 values for 8 experts each: 3.0
    // us, with two warps 4.1).
    const int passes = (K + 511) / 512;
    const bool few = count <= device_sm_count(), row_per_warp = passes <= 4 && !few;
    const int most = few ? 8 : row_per_warp ? 1 : 2;
    int iter = 1;
    while (iter < 4 && passes > most * iter) iter *= 2;
    const int warps = (passes + iter - 1) / iter;
    uint8_t* const base = reinterpret_cast<uint8_t*>(rows);
    float* const scales =
        reinterpret_cast<float*>(base + w4_rows_scale_offset(M, K, to.groups.experts));
    auto go = [&](auto kernel, int blocks, int threads) {
        return launch(kernel, blocks, threads, s, reinterpret_cast<const uint4*>(x), K, k_blocks, to,
                      count, base, scales);
    };
    if (row_per_warp) {
        const int blocks = (count + kRowsAtOnce - 1) / kRowsAtOnce, threads = kRowsAtOnce * 32;
        return iter == 1   ? go(quantize_kernel<1, true>, blocks, threads)
               : iter == 2 ? go(quantize_kernel<2, true>, blocks, threads)
                           : go(quantize_kernel<4, true>, blocks, threads);
    }
    return iter == 1   ? go(quantize_kernel<1, false>, count, warps * 32)
           : iter == 2 ? go(quantize_kernel<2, false>, count, warps * 32)
                       : go(quantize_kernel<4, false>, count, warps * 32);
}

}  // namespace

cudaError_t launch_w4_quantize(const void* x, int M, int K, const W4Groups& g, void* rows,
                               cudaStream_t s) {
    return quantize(x, M, M, K, Places{g, nullptr, nullptr, 0, M}, rows, s);
}

cudaError_t launch_w4_quantize_routed(const void* x, int tokens, int K, const int* ids,
                                      const int* place, int choices, const W4Groups& g, void* rows,
                                      cudaStream_t s) {
    const int M = tokens * choices;
    return quantize(x, tokens, M, K, Places{g, ids, place, choices, M}, rows, s);
}

cudaError_t launch_w4_dequantize(const void* rows, int M, int K, const W4Groups& g, void* out,
                                 cudaStream_t s) {
    const uint8_t* const base = reinterpret_cast<const uint8_t*>(rows);
    const float* const scales =
        reinterpret_cast<const float*>(base + w4_rows_scale_offset(M, K, g.experts));
    return launch(dequantize_kernel, M, kThreads, s, base, scales, K, w4_k_blocks(K), g,
                  reinterpret_cast<uint4*>(out));
}

}  // namespace nvf
