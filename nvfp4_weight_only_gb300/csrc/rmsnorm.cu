// rmsnorm.cu -- root-mean-square norm of x + residual, in one pass:
//   r = x + residual (fp32),  sum = bf16(r)
//   y = r * (mean(r^2) + eps)^(-1/2) * (weight + weight_bias)
// stored as bf16(y), or as E4M3 codes with one fp32 scale per row and 128
// columns: scale = max(amax / 448, 2^-126) (1 for a group of zeros),
// code = e4m3(y / scale), the quotient rounded to fp32, which saturates and keeps NaN.
//
// One block per row; a thread holds its 8-column vectors of r in registers
// between the sum of squares and the output, so x and the residual are read
// once.  The sum, the norm and y stay in fp32 (the residual stream's rounding
// to bf16 does not enter the norm).
//
// Memory bounds many rows (4096 x 5376 with residual, into E4M3: 25.3 us for 155 MB,
// 6.1 TB/s; the block's sum is a wait that other blocks of the SM have to fill),
// one row the launch (1.8 us).  Arithmetic on pairs halves its instructions, which
// took 63% of the issue slots (29.5 us before).
#include "kv8.cuh"

namespace nvf {

namespace {

struct NormArgs {
    const uint4* x;
    const uint4* residual;  // or null
    const uint4* weight;
    uint4* sum_out;         // or null
    uint4* out;             // bf16 output, or null
    uint2* codes;           // E4M3 output, or null
    float* scales;
    int vecs;               // H / 8
    int groups;             // ceil(H / 128)
    float inv_h, eps, weight_bias;
};

// 8 bf16 values as pairs of fp32.
__device__ __forceinline__ void unpack8(const uint4& w, uint64_t (&v)[4]) {
    const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = pair(bf16_lo(a[i]), bf16_hi(a[i]));
}

__device__ __forceinline__ uint4 pack8(const uint64_t (&v)[4]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 p = unpair(v[i]);
        w[i] = bf16x2(p.x, p.y);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

constexpr int kManyRows = 256;

// kVecs: vectors per thread.  The vectors of a warp are consecutive, so 16
// lanes hold one group of 128 columns.
// Registers are given out by eights: 40 per thread let one block more onto an SM
// than the 42 that the compiler would take (4096 x 5376 into E4M3, 352 threads: 25.1
// us against 28.0; 28.4 with 32, which spill).  Blocks have up to 1024 threads.
template <int kVecs>
__global__ void __maxnreg__(kVecs == 1 ? 32 : kVecs == 2 ? 40 : 64) add_rmsnorm_kernel(const NormArgs a) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const size_t row = blockIdx.x;
    const uint4* x = a.x + row * a.vecs;
    // everything the row needs is asked for at once
    uint4 in[kVecs], more[kVecs], w[kVecs];
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const int c = tid + i * blockDim.x;
        in[i] = more[i] = w[i] = make_uint4(0, 0, 0, 0);
        if (c < a.vecs) {
            in[i] = x[c];
            if (a.residual) more[i] = a.residual[row * a.vecs + c];
            w[i] = a.weight[c];
        }
    }
    uint64_t r[kVecs][4], squares = pair(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const int c = tid + i * blockDim.x;
        unpack8(in[i], r[i]);
        if (a.residual) {
            uint64_t o[4];
            unpack8(more[i], o);
#pragma unroll
            for (int e = 0; e < 4; ++e) r[i][e] = add2(r[i][e], o[e]);
        }
        if (a.sum_out && c < a.vecs) a.sum_out[row * a.vecs + c] = pack8(r[i]);
#pragma unroll
        for (int e = 0; e < 4; ++e) squares = fma2(r[i][e], r[i][e], squares);
    }
    float ss = unpair(squares).x + unpair(squares).y;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
    __shared__ float part[32];
    if (lane == 0) part[warp] = ss;
    __syncthreads();
    float total = lane < (int)(blockDim.x >> 5) ? part[lane] : 0.0f;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) total += __shfl_xor_sync(0xffffffffu, total, d);
    const float inv = rsqrtf(total * a.inv_h + a.eps);
    const uint64_t by_inv = pair(inv, inv), bias = pair(a.weight_bias, a.weight_bias);
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const int c = tid + i * blockDim.x;
        const bool live = c < a.vecs;
        uint64_t y[4];
        unpack8(w[i], y);
        // beyond the row 0, or NaN when the norm is not finite: neither enters a maximum
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = mul2(mul2(r[i][e], by_inv), add2(y[e], bias));
        if (a.out) {
            if (live) a.out[row * a.vecs + c] = pack8(y);
            continue;
        }
        float top = 0.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            top = fmaxf(top, fmaxf(fabsf(unpair(y[e]).x), fabsf(unpair(y[e]).y)));
#pragma unroll
        for (int d = 8; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        const float scale = top == 0.0f ? 1.0f : fmaxf(__fdiv_rn(top, 448.0f), 1.17549435e-38f);
        if (live) {
            // y / scale, rounded once, through the reciprocal as a sum of two floats: by,
            // not above it, and rest = (1 - scale * by) * by, which is exact to 2^-24 of
            // itself, so that y * by + y * rest is off by 2^-47 of the quotient before its
            // one rounding.  (rest is not negative: a zero keeps its sign.)  With by alone,
            // rounded to nearest, codes beside a tie fall to the wrong side (4096 x 5376:
            // 25.0 us against 25.3; 29.2 with a division per value).
            const float by = __frcp_rd(scale);
            const float rest = by == 0.0f ? 0.0f : __fmaf_rn(-scale, by, 1.0f) * by;
            float2 q[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                q[e] = unpair(fma2(y[e], pair(by, by), mul2(y[e], pair(rest, rest))));
            a.codes[row * a.vecs + c] =
                make_uint2(f32x4_to_e4m3x4(q[0].x, q[0].y, q[1].x, q[1].y),
                           f32x4_to_e4m3x4(q[2].x, q[2].y, q[3].x, q[3].y));
            if ((c & 15) == 0) a.scales[row * a.groups + (c >> 4)] = scale;
        }
    }
}

}  // namespace

cudaError_t launch_add_rmsnorm(const void* x, const void* residual, const void* weight, int M,
                               int H, float eps, float weight_bias, void* sum_out, void* out,
                               uint8_t* codes, float* scales, cudaStream_t s) {
    NormArgs a;
    a.x = reinterpret_cast<const uint4*>(x);
    a.residual = reinterpret_cast<const uint4*>(residual);
    a.weight = reinterpret_cast<const uint4*>(weight);
    a.sum_out = reinterpret_cast<uint4*>(sum_out);
    a.out = reinterpret_cast<uint4*>(out);
    a.codes = reinterpret_cast<uint2*>(codes);
    a.scales = scales;
    a.vecs = H / 8;
    a.groups = (H + 127) / 128;
    a.inv_h = 1.0f / (float)H;
    a.eps = eps;
    a.weight_bias = weight_bias;
    const int per = (a.vecs + 1023) / 1024;
    if (per > 4) return cudaErrorInvalidValue;
    // One vector per thread is the shortest chain for a few rows (H = 5120 into bf16: 1
    // row 1.9 us against 2.0 with two, 256 rows 3.0 against 3.1); many rows want small
    // blocks, whose loads and stores overlap others' (512 rows 3.9 against 3.5 with
    // two, 4096 rows 26.8 against 25.8).  Four are for rows that 1024 threads with two
    // do not hold.
    const int kv = per <= 1 ? (M > kManyRows ? 2 : 1) : per <= 2 ? 2 : 4;
    const int threads = ((a.vecs + kv - 1) / kv + 31) / 32 * 32;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(M);
    cfg.blockDim = dim3(threads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg,
                              kv == 1   ? add_rmsnorm_kernel<1>
                              : kv == 2 ? add_rmsnorm_kernel<2>
                                        : add_rmsnorm_kernel<4>,
                              a);
}

}  // namespace nvf
