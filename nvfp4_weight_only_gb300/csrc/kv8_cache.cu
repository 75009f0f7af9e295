// kv8_cache.cu -- the paged E4M3 cache: rotary positions and quantisation of
// new tokens as they are written, the same tokens read back, and the table of
// rotations (a load-time call).
//
// Write.  A run is one page's share of one sequence's new tokens; one block
// takes one run of one head of k or v, so a page's scale has one writer and
// nothing is atomic.  For the run's values x (k rotated in fp32, not rounded
// in between):
//   need   = the smallest 2^e with max |x| <= 448 * 2^e, e in -60..119
//   scale' = max(scale, need) when the page already holds rows, else need
//   old rows, when scale' != scale:  code = e4m3(code * (scale / scale'))
//   new rows:                        code = e4m3(x / scale')
// A power-of-two scale costs E4M3 no precision (its own exponent covers 2^15)
// and makes the re-scaling of old rows a shift of their exponents, exact but
// for codes that become subnormal.  max ignores NaN (kept as E4M3's NaN);
// infinities saturate.
#include "kv8.cuh"

namespace nvf {

namespace {

constexpr int kAppendThreads = 128;

struct AppendArgs {
    Kv8CacheArgs c;
    Kv8BatchArgs bt;
    RopeArgs rope;
    const __nv_bfloat16* k;
    const __nv_bfloat16* v;
    const __nv_bfloat16* q;
    __nv_bfloat16* q_out;
    long long k_stride, v_stride, q_stride;
    int heads, runs;
    int q_blocks;  // blocks of the rotation of q, after those of the cache
};

// The two vectors of 8 values that slot `slot` of a head stands for: in the
// half layout a rotated slot pairs vector `slot` with the one rot/2 values
// later; otherwise slots are 16 consecutive values.
__device__ __forceinline__ void slot_vectors(const RopeArgs& r, int slot, int& va, int& vb) {
    if (!r.interleaved && slot < r.rot / 16) {
        va = slot;
        vb = slot + r.rot / 16;
    } else {
        va = 2 * slot;
        vb = va + 1;
    }
}

// The 16 values of one slot of one head at one position, rotated.
__device__ __forceinline__ void load_slot(const RopeArgs& r, const __nv_bfloat16* head,
                                          int position, int slot, float (&a)[8], float (&b)[8]) {
    int va, vb;
    slot_vectors(r, slot, va, vb);
    const uint4 wa = reinterpret_cast<const uint4*>(head)[va];
    const uint4 wb = reinterpret_cast<const uint4*>(head)[vb];
    const uint32_t pa[4] = {wa.x, wa.y, wa.z, wa.w}, pb[4] = {wb.x, wb.y, wb.z, wb.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        a[2 * i] = bf16_lo(pa[i]);
        a[2 * i + 1] = bf16_hi(pa[i]);
        b[2 * i] = bf16_lo(pb[i]);
        b[2 * i + 1] = bf16_hi(pb[i]);
    }
    if (slot >= r.rot / 16) return;
    // (cos, sin) of the slot's 8 pairs
    const float4* t = reinterpret_cast<const float4*>(r.table + (size_t)position * r.rot) +
                      4 * slot;
    float cs[16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 w = t[i];
        cs[4 * i] = w.x;
        cs[4 * i + 1] = w.y;
        cs[4 * i + 2] = w.z;
        cs[4 * i + 3] = w.w;
    }
    if (!r.interleaved) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float x = a[i], y = b[i], c = cs[2 * i], s = cs[2 * i + 1];
            a[i] = __fsub_rn(__fmul_rn(x, c), __fmul_rn(y, s));
            b[i] = __fadd_rn(__fmul_rn(y, c), __fmul_rn(x, s));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float x = a[2 * i], y = a[2 * i + 1], c = cs[2 * i], s = cs[2 * i + 1];
            a[2 * i] = __fsub_rn(__fmul_rn(x, c), __fmul_rn(y, s));
            a[2 * i + 1] = __fadd_rn(__fmul_rn(y, c), __fmul_rn(x, s));
            const float z = b[2 * i], w = b[2 * i + 1], d = cs[8 + 2 * i], e = cs[8 + 2 * i + 1];
            b[2 * i] = __fsub_rn(__fmul_rn(z, d), __fmul_rn(w, e));
            b[2 * i + 1] = __fadd_rn(__fmul_rn(w, d), __fmul_rn(z, e));
        }
    }
}

__device__ __forceinline__ uint2 quantise8(const float (&x)[8], float inv) {
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = x[i] * inv;
    return make_uint2(f32x4_to_e4m3x4(q[0], q[1], q[2], q[3]),
                      f32x4_to_e4m3x4(q[4], q[5], q[6], q[7]));
}

__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
    return make_uint4(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]), bf16x2(v[4], v[5]),
                      bf16x2(v[6], v[7]));
}

// Exponent of the smallest power of two that holds amax: amax = m * 2^x with
// m in [1, 2) and 448 = 1.75 * 2^8, so e = x - 8, or one more when m > 1.75.
__device__ __forceinline__ int scale_exponent(float amax) {
    const uint32_t bits = __float_as_uint(amax);
    const int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    return min(max(e, kKv8MinExp), kKv8MaxExp);
}

__device__ __forceinline__ float two_to(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

__device__ __forceinline__ uint32_t rescale4(uint32_t w, float ratio) {
    float v[4];
    e4m3x4_to_f32(w, v);
    return f32x4_to_e4m3x4(v[0] * ratio, v[1] * ratio, v[2] * ratio, v[3] * ratio);
}

__device__ __forceinline__ int rope_position(const AppendArgs& a, int position) {
    if (a.rope.rot == 0 || position < a.rope.positions) return position;
    kv8_report(a.bt);
    return a.rope.positions - 1;
}

__device__ void append_run(const AppendArgs& a, int x, int head, bool is_v) {
    Kv8Run r;
    if (!kv8_find_run(a.bt, x, r)) return;
    const int page = kv8_page(a.bt, a.c, r.b, r.page_index);
    if (page < 0) return;
    const int dim = a.c.head_dim, slots = dim / 16;
    const int size = 1 << a.bt.page_shift;
    const size_t at = (size_t)page * a.c.kv_heads + head;
    uint8_t* codes = (is_v ? a.c.v_codes : a.c.k_codes) + at * size * dim;
    float* scales = (is_v ? a.c.v_scales : a.c.k_scales) + at;
    const long long stride = is_v ? a.v_stride : a.k_stride;
    const __nv_bfloat16* src = (is_v ? a.v : a.k) + r.token * stride + (size_t)head * dim;
    RopeArgs rope = a.rope;
    if (is_v) rope.rot = 0;
    const int items = r.rows * slots;
    const int tid = threadIdx.x;
    float top = 0.0f;
    for (int i = tid; i < items; i += kAppendThreads) {
        const int row = i / slots, slot = i - row * slots;
        float p[8], q[8];
        load_slot(rope, src + row * stride, is_v ? 0 : rope_position(a, r.position + row), slot, p,
                  q);
#pragma unroll
        for (int e = 0; e < 8; ++e) top = fmaxf(top, fmaxf(fabsf(p[e]), fabsf(q[e])));
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    __shared__ float part[kAppendThreads / 32];
    if ((tid & 31) == 0) part[tid >> 5] = top;
    const float before = r.row > 0 ? *scales : 0.0f;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kAppendThreads / 32; ++w) top = fmaxf(top, part[w]);
    const float need = two_to(scale_exponent(top));
    const float scale = fmaxf(before, need);
    if (r.row > 0 && scale != before) {
        const float ratio = __fdiv_rn(before, scale);
        uint4* old = reinterpret_cast<uint4*>(codes);
        for (int i = tid; i < r.row * slots; i += kAppendThreads) {
            uint4 w = old[i];
            w.x = rescale4(w.x, ratio);
            w.y = rescale4(w.y, ratio);
            w.z = rescale4(w.z, ratio);
            w.w = rescale4(w.w, ratio);
            old[i] = w;
        }
    }
    // 1 / scale is exact for a power of two; a foreign scale takes one rounding
    const float inv = __fdiv_rn(1.0f, scale);
    for (int i = tid; i < items; i += kAppendThreads) {
        const int row = i / slots, slot = i - row * slots;
        float p[8], q[8];
        load_slot(rope, src + row * stride, is_v ? 0 : rope_position(a, r.position + row), slot, p,
                  q);
        int va, vb;
        slot_vectors(rope, slot, va, vb);
        uint2* dst = reinterpret_cast<uint2*>(codes + (size_t)(r.row + row) * dim);
        dst[va] = quantise8(p, inv);
        dst[vb] = quantise8(q, inv);
    }
    if (tid == 0) *scales = scale;
}

// Rotates q of one token per warp (or copies it without a table).
__device__ void turn_q(const AppendArgs& a, int t) {
    const int b = kv8_owner(a.bt, t);
    int position = 0;
    RopeArgs rope = a.rope;
    if (b < a.bt.batch) {
        const Kv8Seq s = kv8_seq(a.bt, b);
        position = s.kv - s.len + (t - s.q0);
        if (s.bad && (threadIdx.x & 31) == 0) kv8_report(a.bt);
    } else {
        kv8_report(a.bt);
    }
    position = rope_position(a, max(position, 0));
    const int dim = a.c.head_dim, slots = dim / 16;
    for (int i = threadIdx.x & 31; i < a.heads * slots; i += 32) {
        const int head = i / slots, slot = i - head * slots;
        float p[8], r[8];
        load_slot(rope, a.q + t * a.q_stride + (size_t)head * dim, position, slot, p, r);
        int va, vb;
        slot_vectors(rope, slot, va, vb);
        uint4* dst = reinterpret_cast<uint4*>(a.q_out + ((size_t)t * a.heads + head) * dim);
        dst[va] = pack8(p);
        dst[vb] = pack8(r);
    }
}

__global__ void __launch_bounds__(kAppendThreads) kv8_append_kernel(const AppendArgs a) {
    const int per_run = 2 * a.c.kv_heads;
    const int cache_blocks = a.runs * per_run;
    const int x = blockIdx.x;
    if (x < cache_blocks) {
        const int head = x % per_run;
        append_run(a, x / per_run, head >> 1, head & 1);
    } else {
        const int t = (x - cache_blocks) * (kAppendThreads / 32) + (threadIdx.x >> 5);
        if (t < a.bt.tokens) turn_q(a, t);
    }
}

struct ReadArgs {
    Kv8CacheArgs c;
    Kv8BatchArgs bt;
    __nv_bfloat16* k_out;
    __nv_bfloat16* v_out;
    int runs;
};

__global__ void __launch_bounds__(kAppendThreads) kv8_read_kernel(const ReadArgs a) {
    const int per_run = 2 * a.c.kv_heads;
    const int head = (blockIdx.x % per_run) >> 1;
    const bool is_v = blockIdx.x & 1;
    Kv8Run r;
    if (!kv8_find_run(a.bt, blockIdx.x / per_run, r)) return;
    const int page = kv8_page(a.bt, a.c, r.b, r.page_index);
    if (page < 0) return;
    const int dim = a.c.head_dim, slots = dim / 16;
    const size_t at = (size_t)page * a.c.kv_heads + head;
    const float scale = (is_v ? a.c.v_scales : a.c.k_scales)[at];
    const uint4* codes = reinterpret_cast<const uint4*>(
        (is_v ? a.c.v_codes : a.c.k_codes) + ((at << a.bt.page_shift) + r.row) * dim);
    __nv_bfloat16* out = is_v ? a.v_out : a.k_out;
    for (int i = threadIdx.x; i < r.rows * slots; i += kAppendThreads) {
        const int row = i / slots, slot = i - row * slots;
        const uint4 w = codes[i];
        const uint32_t p[4] = {w.x, w.y, w.z, w.w};
        uint32_t o[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float v[4];
            e4m3x4_to_f32(p[e], v);
            o[2 * e] = bf16x2(v[0] * scale, v[1] * scale);
            o[2 * e + 1] = bf16x2(v[2] * scale, v[3] * scale);
        }
        uint4* dst = reinterpret_cast<uint4*>(
            out + ((size_t)(r.token + row) * a.c.kv_heads + head) * dim + slot * 16);
        dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
        dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
}

struct TableArgs {
    int positions, half, scaling;
    double base, factor, context, slow, fast, magnitude;
    float2* table;
};

// Entry (p, i): magnitude * (cos, sin)(p * f_i), in fp64 and rounded once.
// f_i = base^(-2i/rot), changed for longer contexts by
//   linear: f_i / factor
//   base:   base * factor^(rot / (rot - 2)) in place of base
//   ramp:   f_i * (g + (1 - g) / factor), g the share of the way that the
//           turns f_i makes over `context` tokens are from slow to fast
__global__ void rope_table_kernel(const TableArgs a) {
    const size_t n = (size_t)a.positions * a.half;
    const double two_pi = 6.283185307179586;
    for (size_t x = blockIdx.x * (size_t)blockDim.x + threadIdx.x; x < n;
         x += (size_t)gridDim.x * blockDim.x) {
        const int i = (int)(x % a.half);
        const double rot = 2.0 * a.half;
        double base = a.base;
        if (a.scaling == 2 && a.half > 1) base *= pow(a.factor, rot / (rot - 2.0));
        double f = pow(base, -2.0 * i / rot);
        if (a.scaling == 1) f /= a.factor;
        if (a.scaling == 3) {
            const double turns = f * a.context / two_pi;
            const double g = fmin(fmax((turns - a.slow) / (a.fast - a.slow), 0.0), 1.0);
            f *= g + (1.0 - g) / a.factor;
        }
        double s, c;
        sincos((double)(x / a.half) * f, &s, &c);
        a.table[x] = make_float2((float)(c * a.magnitude), (float)(s * a.magnitude));
    }
}

}  // namespace

cudaError_t launch_rope_table(int positions, int rot, double base, int scaling, double factor,
                              double context, double slow, double fast, double magnitude,
                              float* table, cudaStream_t s) {
    const TableArgs a{positions, rot / 2, scaling, base, factor, context, slow, fast, magnitude,
                      reinterpret_cast<float2*>(table)};
    const size_t n = (size_t)positions * a.half;
    const unsigned blocks = (unsigned)((n + 255) / 256 < 4096 ? (n + 255) / 256 : 4096);
    rope_table_kernel<<<blocks, 256, 0, s>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_kv8_append(const Kv8CacheArgs& c, const Kv8BatchArgs& bt, const void* k,
                              long long k_stride, const void* v, long long v_stride,
                              const void* q, long long q_stride, int heads, void* q_out,
                              const RopeArgs& rope, cudaStream_t s) {
    AppendArgs a;
    a.c = c;
    a.bt = bt;
    a.rope = rope;
    a.k = reinterpret_cast<const __nv_bfloat16*>(k);
    a.v = reinterpret_cast<const __nv_bfloat16*>(v);
    a.q = reinterpret_cast<const __nv_bfloat16*>(q);
    a.q_out = reinterpret_cast<__nv_bfloat16*>(q_out);
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.q_stride = q_stride;
    a.heads = heads;
    a.runs = (int)kv8_max_runs(bt.tokens, bt.batch, bt.page_shift);
    const int per = kAppendThreads / 32;
    const long long blocks = (long long)a.runs * 2 * c.kv_heads +
                             (q ? ((long long)bt.tokens + per - 1) / per : 0);
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    kv8_append_kernel<<<(unsigned)blocks, kAppendThreads, 0, s>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_kv8_read(const Kv8CacheArgs& c, const Kv8BatchArgs& bt, void* k_out,
                            void* v_out, cudaStream_t s) {
    ReadArgs a;
    a.c = c;
    a.bt = bt;
    a.k_out = reinterpret_cast<__nv_bfloat16*>(k_out);
    a.v_out = reinterpret_cast<__nv_bfloat16*>(v_out);
    a.runs = (int)kv8_max_runs(bt.tokens, bt.batch, bt.page_shift);
    const long long blocks = (long long)a.runs * 2 * c.kv_heads;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    kv8_read_kernel<<<(unsigned)blocks, kAppendThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace nvf
