// rmsnorm.cu -- root-mean-square norm of x + residual, in one pass:
//   r = x + residual (fp32),  sum = bf16(r)
//   y = r * (mean(r^2) + eps)^(-1/2) * (weight + weight_bias)
// stored as bf16(y), or as E4M3 codes with one fp32 scale per row and 128
// columns: scale = max(amax / 448, 2^-126) (1 for a group of zeros),
// code = e4m3(y / scale), which saturates and keeps NaN (the quotient is off by
// at most 2^-22 of itself).
//
// One block per row; a thread holds its 8-column vectors of r in registers
// between the sum of squares and the output, so x and the residual are read
// once.  The sum, the norm and y stay in fp32 (the residual stream's rounding
// to bf16 does not enter the norm).
//
// Memory bounds many rows (4096 x 5376 with residual, into E4M3: 29.5 us for 155 MB,
// 5.2 TB/s; the block's sum is a wait that other blocks of the SM fill only in part),
// one row the launch (1.8 us).
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

__device__ __forceinline__ void unpack8(const uint4& w, float (&v)[8]) {
    const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf16_lo(a[i]);
        v[2 * i + 1] = bf16_hi(a[i]);
    }
}

__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
    return make_uint4(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]), bf16x2(v[4], v[5]),
                      bf16x2(v[6], v[7]));
}

constexpr int kManyRows = 256;

// kVecs: vectors per thread.  The vectors of a warp are consecutive, so 16
// lanes hold one group of 128 columns.
template <int kVecs>
__global__ void __launch_bounds__(1024) add_rmsnorm_kernel(const NormArgs a) {
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
    float r[kVecs][8];
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const int c = tid + i * blockDim.x;
        unpack8(in[i], r[i]);
        if (a.residual) {
            float o[8];
            unpack8(more[i], o);
#pragma unroll
            for (int e = 0; e < 8; ++e) r[i][e] += o[e];
        }
        if (a.sum_out && c < a.vecs) a.sum_out[row * a.vecs + c] = pack8(r[i]);
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(r[i][e], r[i][e], ss);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
    __shared__ float part[32];
    if (lane == 0) part[warp] = ss;
    __syncthreads();
    float total = lane < (int)(blockDim.x >> 5) ? part[lane] : 0.0f;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) total += __shfl_xor_sync(0xffffffffu, total, d);
    const float inv = rsqrtf(total * a.inv_h + a.eps);
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const int c = tid + i * blockDim.x;
        const bool live = c < a.vecs;
        float y[8];
        unpack8(w[i], y);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = live ? r[i][e] * inv * (y[e] + a.weight_bias) : 0.0f;
        if (a.out) {
            if (live) a.out[row * a.vecs + c] = pack8(y);
            continue;
        }
        float top = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(y[e]));
#pragma unroll
        for (int d = 8; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        const float scale = top == 0.0f ? 1.0f : fmaxf(__fdiv_rn(top, 448.0f), 1.17549435e-38f);
        if (live) {
            // y / scale through the reciprocal: off by at most 2^-22 of itself
            const float by = __frcp_rn(scale);
            float q[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) q[e] = y[e] * by;
            a.codes[row * a.vecs + c] = make_uint2(f32x4_to_e4m3x4(q[0], q[1], q[2], q[3]),
                                                   f32x4_to_e4m3x4(q[4], q[5], q[6], q[7]));
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
    // One vector per thread is the shortest chain for a few rows (H = 5120: 1 row 1.9
    // us both ways, 256 rows 3.1 against 3.2 with two); many rows want small blocks,
    // whose loads and stores overlap others' (512 rows 4.0 against 3.6 with two; 4096
    // rows of 5376 into E4M3 33.3, two 29.8, four 35.7).
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
