// kv8.cuh -- what the kernels on the paged E4M3 key/value cache share: the
// cache and batch descriptions as the kernels take them, the search for a
// page run or a token's sequence, and E4M3 conversions of 16 values.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "device_util.cuh"
#include "kv8.h"

namespace nvf {

// Power-of-two scales a page can get: 2^kKv8MinExp (also that of zeros) to
// 2^kKv8MaxExp.  448 * 2^119 is finite in fp32 and bf16; larger values
// saturate.
constexpr int kKv8MinExp = -60;
constexpr int kKv8MaxExp = 119;

// Sequence b's new tokens and length, with values that the buffers cannot hold
// cut off (and reported): q0..q1 inside [0, tokens], kv inside the table.
struct Kv8Seq {
    int q0, len, kv;
    bool bad;
};

__device__ __forceinline__ Kv8Seq kv8_seq(const Kv8BatchArgs& bt, int b) {
    Kv8Seq s;
    const int a0 = bt.q_start[b], a1 = bt.q_start[b + 1], kv = bt.kv_len[b];
    s.q0 = min(max(a0, 0), bt.tokens);
    s.len = min(max(a1, s.q0), bt.tokens) - s.q0;
    s.kv = min(max(kv, 0), bt.max_kv);
    s.bad = s.q0 != a0 || s.q0 + s.len != a1 || s.kv != kv || s.len > s.kv;
    return s;
}

__device__ __forceinline__ void kv8_report(const Kv8BatchArgs& bt) {
    if (bt.status) *bt.status = kKv8BadIndex;
}

// One page's share of one sequence's new tokens.
struct Kv8Run {
    int b, page_index;   // which page of sequence b
    int token;           // first token of the run in q/k/v
    int position;        // its position in the sequence
    int rows;            // tokens of the run
    int row;             // its row in the page
};

// The x-th run of the batch, in the order of the sequences and their pages;
// false when there are fewer.  One warp calls it with all its lanes: each lane
// counts the pages of one sequence, a prefix sum finds the sequence.
__device__ __forceinline__ bool kv8_find_run(const Kv8BatchArgs& bt, int x, Kv8Run& r) {
    const int lane = threadIdx.x & 31;
    int base = 0;
    for (int c = 0; c < bt.batch; c += 32) {
        Kv8Seq s{0, 0, 0, false};
        int n = 0, first = 0;
        if (c + lane < bt.batch) {
            s = kv8_seq(bt, c + lane);
            if (s.bad) kv8_report(bt);
            first = max(s.kv - s.len, 0);  // tokens in front of position 0 are left out
            if (s.len > 0 && s.kv > first)
                n = ((s.kv - 1) >> bt.page_shift) - (first >> bt.page_shift) + 1;
        }
        int sum = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, sum, d);
            if (lane >= d) sum += o;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, base + sum > x);
        if (hit) {
            const int l = __ffs(hit) - 1;
            const int before = base + __shfl_sync(0xffffffffu, sum - n, l);
            const int f = __shfl_sync(0xffffffffu, first, l);
            const int kv = __shfl_sync(0xffffffffu, s.kv, l);
            const int q0 = __shfl_sync(0xffffffffu, s.q0, l);
            const int len = __shfl_sync(0xffffffffu, s.len, l);
            r.b = c + l;
            r.page_index = (f >> bt.page_shift) + (x - before);
            const int lo = max(f, r.page_index << bt.page_shift);
            const int hi = min(kv, (r.page_index + 1) << bt.page_shift);
            r.position = lo;
            r.rows = hi - lo;
            r.row = lo & ((1 << bt.page_shift) - 1);
            r.token = q0 + lo - (kv - len);
            return true;
        }
        base += __shfl_sync(0xffffffffu, sum, 31);
    }
    return false;
}

// The page of a run, or -1 (reported) for an entry outside the cache.
__device__ __forceinline__ int kv8_page(const Kv8BatchArgs& bt, const Kv8CacheArgs& c, int b,
                                        int page_index) {
    const int p = bt.page_table[(size_t)b * bt.table_width + page_index];
    if (p >= 0 && p < c.pages) return p;
    kv8_report(bt);
    return -1;
}

// The sequence that token t belongs to (one warp, all lanes): the number of
// sequences that end at or before it; bt.batch when none holds it.
__device__ __forceinline__ int kv8_owner(const Kv8BatchArgs& bt, int t) {
    const int lane = threadIdx.x & 31;
    int b = 0;
    for (int c = 0; c < bt.batch; c += 32) {
        const bool past = c + lane < bt.batch && bt.q_start[c + lane + 1] <= t;
        const unsigned m = __ballot_sync(0xffffffffu, past);
        b += __popc(m);
        if (m != 0xffffffffu) break;
    }
    return b;
}

// Two fp32 -> two E4M3 bytes (a in the low one), to nearest even, saturated.
__device__ __forceinline__ uint32_t f32x2_to_e4m3x2(float a, float b) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ uint32_t f32x4_to_e4m3x4(float a, float b, float c, float d) {
    return f32x2_to_e4m3x2(a, b) | (f32x2_to_e4m3x2(c, d) << 16);
}

// Four E4M3 bytes -> fp32 (exact).
__device__ __forceinline__ void e4m3x4_to_f32(uint32_t w, float (&v)[4]) {
    const uint32_t lo = e4m3x2_to_f16x2(w), hi = e4m3x2_hi_to_f16x2(w);
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    v[0] = a.x;
    v[1] = a.y;
    v[2] = b.x;
    v[3] = b.y;
}

__device__ __forceinline__ uint32_t bf16x2(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// fp32 pairs: two results per instruction.
__device__ __forceinline__ uint64_t pair(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 unpair(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// bf16 pair -> fp32 (element 0 in the low half).
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

}  // namespace nvf
