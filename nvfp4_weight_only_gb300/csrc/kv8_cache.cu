// kv8_cache.cu -- the paged E4M3 cache: rotary positions and quantisation of
// new tokens as they are written, the same tokens read back, and the table of
// rotations (a load-time call).
//
// Write.  A run is one page's share of one sequence's new tokens; one warp or
// block takes one run of one head of k or v, so a page's scale has one writer and
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

constexpr int kAppendWarps = 8;
constexpr int kAppendThreads = kAppendWarps * 32;
// New tokens per sequence, on average, from which a run takes a block (8 sequences,
// 8 kv heads of 128, 40 q heads: 1 token 4.4 us against 4.8 in blocks, 8 tokens 4.5
// against 5.0, 16 tokens 5.5 against 5.1, 128 tokens 17.4 against 9.4).
constexpr int kWideRows = 16;

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
    int cache_blocks, q_blocks;  // blocks of the cache's part; those that rotate q
};

// A slot is 16 values of a head, as two vectors of 8.  In the half layout a
// rotated slot pairs vector `slot` with the one rot/2 values later; other
// vectors are paired with those half of them further, so that neighbouring
// slots' vectors lie side by side in memory.  A head has dim / 16 slots, which
// divides a warp: a lane keeps one slot, and its rotations serve every head of a
// token.
struct Slot {
    int a, b;            // vectors
    bool turn_a, turn_b;  // whether they are rotated (together in the half layout)
};

__device__ __forceinline__ Slot slot_of(const RopeArgs& r, int slot, int slots) {
    if (r.interleaved) return Slot{slot, slot + slots, slot < r.rot / 8, slot + slots < r.rot / 8};
    const int turned = r.rot / 16;
    if (slot < turned) return Slot{slot, slot + turned, true, true};
    return Slot{slot + turned, slot + slots, false, false};
}

// (cos, sin) of a slot's 8 pairs at one position (those of vectors that turn).
struct Turn {
    float cs[16];
};

__device__ __forceinline__ Turn load_turn(const RopeArgs& r, int position, const Slot& s) {
    Turn t;
    const float4* const p =
        reinterpret_cast<const float4*>(r.table + (size_t)position * r.rot);
    // the half layout's pair i is value i of both vectors; interleaved vectors
    // have 4 pairs of their own
    const int at[2] = {r.interleaved ? 2 * s.a : 4 * s.a, r.interleaved ? 2 * s.b : 4 * s.a + 2};
    const bool turns[2] = {s.turn_a, s.turn_b};
#pragma unroll
    for (int h = 0; h < 2; ++h)
        if (turns[h]) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float4 w = p[at[h] + i];
                t.cs[8 * h + 4 * i] = w.x;
                t.cs[8 * h + 4 * i + 1] = w.y;
                t.cs[8 * h + 4 * i + 2] = w.z;
                t.cs[8 * h + 4 * i + 3] = w.w;
            }
        }
    return t;
}

// The slot's raw values.
struct Raw {
    uint4 a, b;
};

__device__ __forceinline__ Raw load_raw(const __nv_bfloat16* head, const Slot& s) {
    return Raw{reinterpret_cast<const uint4*>(head)[s.a], reinterpret_cast<const uint4*>(head)[s.b]};
}

__device__ __forceinline__ void unpack8(const uint4& w, float (&v)[8]) {
    const uint32_t p[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf16_lo(p[i]);
        v[2 * i + 1] = bf16_hi(p[i]);
    }
}

__device__ __forceinline__ void turn_pair(float& x, float& y, float c, float s) {
    const float u = x, w = y;
    x = __fsub_rn(__fmul_rn(u, c), __fmul_rn(w, s));
    y = __fadd_rn(__fmul_rn(w, c), __fmul_rn(u, s));
}

// The slot's values in fp32, rotated (two rounded products and their rounded
// sum; values that do not turn pass unchanged, signs of zeros included).
__device__ __forceinline__ void values(const RopeArgs& r, const Raw& raw, const Slot& s,
                                       const Turn& t, float (&a)[8], float (&b)[8]) {
    unpack8(raw.a, a);
    unpack8(raw.b, b);
    if (!r.interleaved) {
        if (s.turn_a)
#pragma unroll
            for (int i = 0; i < 8; ++i) turn_pair(a[i], b[i], t.cs[2 * i], t.cs[2 * i + 1]);
    } else {
        if (s.turn_a)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                turn_pair(a[2 * i], a[2 * i + 1], t.cs[2 * i], t.cs[2 * i + 1]);
        if (s.turn_b)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                turn_pair(b[2 * i], b[2 * i + 1], t.cs[8 + 2 * i], t.cs[9 + 2 * i]);
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

// Finds the x-th run, without the tokens behind the rotation table (reported, and not
// written); false when nothing is left.
__device__ __forceinline__ bool find_run(const AppendArgs& a, int x, Kv8Run& r) {
    if (!kv8_find_run(a.bt, x, r)) return false;
    const int left = a.rope.positions - r.position;
    if (left < r.rows) {
        kv8_report(a.bt);
        if (left <= 0) return false;
        r.rows = left;
    }
    return true;
}

constexpr int kHeld = 2;  // items of a thread that stay in registers

// A team's part of one head of a run: kTeam threads, each with one slot of
// every (kTeam / slots)-th row.
template <bool kTurn, int kTeam>
struct RunPart {
    RopeArgs rope;
    const __nv_bfloat16* src;
    long long stride;
    int row0, step, slots;
    Slot slot;
    Raw held[kHeld];

    // Starts the loads of the first items (all of a run of a page's worth when
    // the team is a block).
    __device__ __forceinline__ RunPart(const AppendArgs& a, const Kv8Run& r, int head)
        : rope(a.rope), stride(kTurn ? a.k_stride : a.v_stride) {
        const int mate = threadIdx.x % kTeam, dim = a.c.head_dim;
        slots = dim / 16;
        step = kTeam / slots;
        row0 = mate / slots;
        if (!kTurn) rope.rot = 0;
        slot = slot_of(rope, mate % slots, slots);
        src = (kTurn ? a.k : a.v) + r.token * stride + (size_t)head * dim;
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            const int row = row0 + i * step;
            held[i] = Raw{make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
            if (row < r.rows) held[i] = load_raw(src + row * stride, slot);
        }
    }
};

// Quantises a run of one head into its page (`shared` joins the maxima of a
// block's warps).  Items beyond the held ones are read twice, the second time
// from the caches.
template <bool kTurn, int kTeam>
__device__ __forceinline__ void store_run(const AppendArgs& a, const Kv8Run& r, int page, int head,
                                          const RunPart<kTurn, kTeam>& part, float* shared,
                                          float4* kept) {
    constexpr bool is_v = !kTurn;
    const int mate = threadIdx.x % kTeam, dim = a.c.head_dim, slots = part.slots;
    const int row0 = part.row0, step = part.step;
    const Slot slot = part.slot;
    const RopeArgs& rope = part.rope;
    const long long stride = part.stride;
    const __nv_bfloat16* const src = part.src;
    const Raw(&held)[kHeld] = part.held;
    const size_t at = (size_t)page * a.c.kv_heads + head;
    uint8_t* codes = (is_v ? a.c.v_codes : a.c.k_codes) + (at << a.bt.page_shift) * dim;
    float* scales = (is_v ? a.c.v_scales : a.c.k_scales) + at;
    const float before = r.row > 0 ? *scales : 0.0f;
    auto turned = [&](const Raw& raw, int row, float (&p)[8], float (&q)[8]) {
        Turn t;
        if (kTurn && (slot.turn_a || slot.turn_b))
            t = load_turn(rope, r.position + row, slot);
        values(rope, raw, slot, t, p, q);
    };
    float top = 0.0f;
    auto measure = [&](const float (&p)[8], const float (&q)[8]) {
#pragma unroll
        for (int e = 0; e < 8; ++e) top = fmaxf(top, fmaxf(fabsf(p[e]), fabsf(q[e])));
    };
    // A block keeps rotated values in shared memory (registers are what it has too
    // few of); a warp, which has few items, rotates again.
    auto keep = [&](int i, float (&u)[8], float (&w)[8]) {
        const float4 x[4] = {make_float4(u[0], u[1], u[2], u[3]), make_float4(u[4], u[5], u[6], u[7]),
                             make_float4(w[0], w[1], w[2], w[3]), make_float4(w[4], w[5], w[6], w[7])};
#pragma unroll
        for (int e = 0; e < 4; ++e) kept[(4 * i + e) * kTeam + mate] = x[e];
    };
    auto again = [&](int i, int row, float (&u)[8], float (&w)[8]) {
        if constexpr (kTurn && kTeam > 32) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float4 x = kept[(4 * i + e) * kTeam + mate];
                float* const to = e < 2 ? u + 4 * e : w + 4 * (e - 2);
                to[0] = x.x;
                to[1] = x.y;
                to[2] = x.z;
                to[3] = x.w;
            }
        } else {
            turned(held[i], row, u, w);
        }
    };
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
        if (row0 + i * step < r.rows) {
            float u[8], w[8];
            turned(held[i], row0 + i * step, u, w);
            measure(u, w);
            if (kTurn && kTeam > 32) keep(i, u, w);
        }
#pragma unroll 1
    for (int row = row0 + kHeld * step; row < r.rows; row += step) {
        float u[8], w[8];
        turned(load_raw(src + row * stride, slot), row, u, w);
        measure(u, w);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    if constexpr (kTeam > 32) {
        if ((mate & 31) == 0) shared[mate >> 5] = top;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kTeam / 32; ++w) top = fmaxf(top, shared[w]);
    }
    const float scale = fmaxf(before, two_to(scale_exponent(top)));
    if (r.row > 0 && scale != before) {
        const float ratio = __fdiv_rn(before, scale);
        uint4* old = reinterpret_cast<uint4*>(codes);
        for (int i = mate; i < r.row * slots; i += kTeam) {
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
    auto write = [&](const float (&u)[8], const float (&w)[8], int row) {
        uint2* dst = reinterpret_cast<uint2*>(codes + (size_t)(r.row + row) * dim);
        dst[slot.a] = quantise8(u, inv);
        dst[slot.b] = quantise8(w, inv);
    };
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
        if (row0 + i * step < r.rows) {
            float u[8], w[8];
            again(i, row0 + i * step, u, w);
            write(u, w, row0 + i * step);
        }
#pragma unroll 1
    for (int row = row0 + kHeld * step; row < r.rows; row += step) {
        float u[8], w[8];
        turned(load_raw(src + row * stride, slot), row, u, w);
        write(u, w, row);
    }
    if (mate == 0) *scales = scale;  // read by all before the maxima were joined
}

// Rotates q of one token that has a position (or copies it without a table), by one
// warp.  The first
// heads are on their way while the token's position is looked up.
template <int kAhead>
__device__ __forceinline__ void turn_q(const AppendArgs& a, int t) {
    const int lane = threadIdx.x & 31;
    const int dim = a.c.head_dim, slots = dim / 16, step = 32 / slots;
    const Slot slot = slot_of(a.rope, lane % slots, slots);
    const __nv_bfloat16* src = a.q + t * a.q_stride;
    __nv_bfloat16* dst = a.q_out + (size_t)t * a.heads * dim;
    const int head0 = lane / slots;
    Raw raw[kAhead];
    auto load = [&](int first) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int head = first + i * step;
            if (head < a.heads) raw[i] = load_raw(src + (size_t)head * dim, slot);
        }
    };
    load(head0);
    const int b = kv8_owner(a.bt, t);
    if (b >= a.bt.batch) return;  // the token belongs to no sequence
    const Kv8Seq s = kv8_seq(a.bt, b);
    if (s.bad) kv8_report(a.bt);
    const int i = t - s.q0, position = s.kv - s.len + i;
    if (i < 0 || i >= s.len || position < 0) return;
    if (position >= a.rope.positions) {
        kv8_report(a.bt);
        return;
    }
    Turn turn;
    if (slot.turn_a || slot.turn_b) turn = load_turn(a.rope, position, slot);
#pragma unroll 1
    for (int first = head0; first < a.heads;) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int head = first + i * step;
            if (head >= a.heads) break;
            float p[8], r[8];
            values(a.rope, raw[i], slot, turn, p, r);
            uint4* to = reinterpret_cast<uint4*>(dst + (size_t)head * dim);
            to[slot.a] = pack8(p);
            to[slot.b] = pack8(r);
        }
        first += kAhead * step;
        load(first);
    }
}

// One token per sequence, or few: a warp per run and head of k or v (a block's
// warps take neighbouring heads, which share the run's rotations in L1), then q,
// a warp per token.  Latency bounds it: list, table and page are found one
// after the other (3.2 us for one token of 40 heads on 8).
__global__ void __launch_bounds__(kAppendThreads) kv8_append_kernel(const AppendArgs a) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if ((int)blockIdx.x < a.cache_blocks) {
        const int per_run = 2 * a.c.kv_heads;
        const int x = blockIdx.x * kAppendWarps + (threadIdx.x >> 5);
        const int run = x / per_run, part = x - run * per_run;
        Kv8Run r;
        if (run >= a.runs || !find_run(a, run, r)) return;
        const bool is_k = part < a.c.kv_heads;
        const int head = is_k ? part : part - a.c.kv_heads;
        if (is_k) {
            const RunPart<true, 32> k(a, r, head);
            const int page = kv8_page(a.bt, a.c, r.b, r.page_index);
            if (page >= 0) store_run(a, r, page, head, k, nullptr, nullptr);
        } else {
            const RunPart<false, 32> v(a, r, head);
            const int page = kv8_page(a.bt, a.c, r.b, r.page_index);
            if (page >= 0) store_run(a, r, page, head, v, nullptr, nullptr);
        }
    } else {
        const int t = (blockIdx.x - a.cache_blocks) * kAppendWarps + (threadIdx.x >> 5);
        if (t < a.bt.tokens) turn_q<4>(a, t);
    }
}

// Prompts: a block per run and head, k and v, so that both are on their way
// while the run and its page are looked up and k is worked on.  Memory bounds it: a
// run's rows stay on chip between the maximum and the codes, so they are read once
// (up to 3001 tokens of 5 sequences, 32 heads on 16, with q: 82 us for 436 MB, 5.4 TB/s).
// A block waits for its run's table, rows and sum one after the other and then has
// much to compute; q's warps mostly wait for memory: mixed, they fill each other's gaps
// (99 us in two launches).
__global__ void __launch_bounds__(kAppendThreads, 4) kv8_append_rows_kernel(const AppendArgs a) {
    __shared__ float tops[2][kAppendWarps];
    __shared__ float4 kept[kHeld * 4 * kAppendThreads];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // q's blocks lie evenly among the others
    const unsigned q_before =
        (unsigned)((unsigned long long)blockIdx.x * a.q_blocks / gridDim.x);
    if ((unsigned)((unsigned long long)(blockIdx.x + 1) * a.q_blocks / gridDim.x) != q_before) {
        const int t = q_before * kAppendWarps + (threadIdx.x >> 5);
        if (t < a.bt.tokens) turn_q<2>(a, t);
        return;
    }
    const int x = blockIdx.x - q_before;
    const int run = x / a.c.kv_heads, head = x - run * a.c.kv_heads;
    Kv8Run r;
    if (!find_run(a, run, r)) return;
    const RunPart<true, kAppendThreads> k(a, r, head);
    const RunPart<false, kAppendThreads> v(a, r, head);
    const int page = kv8_page(a.bt, a.c, r.b, r.page_index);
    if (page < 0) return;
    store_run(a, r, page, head, k, tops[0], kept);
    store_run(a, r, page, head, v, tops[1], nullptr);
}

struct ReadArgs {
    Kv8CacheArgs c;
    Kv8BatchArgs bt;
    __nv_bfloat16* k_out;
    __nv_bfloat16* v_out;
    int runs;
};

constexpr int kReadThreads = 128;

// One run of one head of k or v per block; memory bounds it (93 us for 587 MB, 6.3
// TB/s of 6.8 that a copy reaches).
__global__ void __launch_bounds__(kReadThreads) kv8_read_kernel(const ReadArgs a) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
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
#pragma unroll 4
    for (int i = threadIdx.x; i < r.rows * slots; i += kReadThreads) {
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

// A launch that may begin while the preceding kernel on the stream finishes;
// the kernel waits for that one before it reads or writes anything.
template <typename Args>
cudaError_t launch_after(void (*kernel)(Args), unsigned blocks, int threads, cudaStream_t s,
                         const Args& a) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(threads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
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
    const long long runs = a.runs;
    const long long q_blocks = q ? ((long long)bt.tokens + kAppendWarps - 1) / kAppendWarps : 0;
    const long long cache_blocks = (runs * 2 * c.kv_heads + kAppendWarps - 1) / kAppendWarps;
    if (runs * 2 * c.kv_heads + q_blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    a.cache_blocks = (int)cache_blocks;
    a.q_blocks = (int)q_blocks;
    if (bt.tokens < kWideRows * bt.batch)
        return launch_after(kv8_append_kernel, (unsigned)(cache_blocks + q_blocks), kAppendThreads,
                            s, a);
    a.cache_blocks = (int)(runs * c.kv_heads);
    return launch_after(kv8_append_rows_kernel, (unsigned)(a.cache_blocks + q_blocks),
                        kAppendThreads, s, a);
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
    return launch_after(kv8_read_kernel, (unsigned)blocks, kReadThreads, s, a);
}

}  // namespace nvf
