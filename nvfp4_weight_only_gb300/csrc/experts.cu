// experts.cu -- a routed batch's lists and its sums.
//
// Order: ids [tokens, choices] sorted by expert, stable, from which come each
// expert's first row, each row's token and each pair's row.  One block per expert
// goes through all ids (they stay in L2): it counts those of lower experts, which
// gives its first row, and its own, which a prefix sum over the block puts in order.
// No block needs another's result, so one launch does it, at a cost of experts * ids
// compares.  One more block has the ids of no expert and the rows behind the last.
//
// Sum: out[t] = bf16(sum_j weights[t][j] * y[place[t][j]]), fp32, in the order of j.
// Bound by memory: every thread has 8 columns of a token and asks for all of its
// rows at once.
#include "kv8.cuh"
#include "w4a4.h"

namespace nvf {

namespace {

constexpr int kOrderThreads = 1024;
constexpr int kSumThreads = 256;
constexpr int kAhead = 8;  // rows of a token asked for at once

// Ids base + 4 lane .. + 3 of a warp's 128, -1 beyond the end.
__device__ __forceinline__ void load4(const int* ids, long long at, long long end, int (&v)[4]) {
    if (at + 4 <= end && (reinterpret_cast<uintptr_t>(ids + at) & 15) == 0) {
        const int4 q = __ldg(reinterpret_cast<const int4*>(ids + at));
        v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = at + i < end ? __ldg(ids + at + i) : -1;
    }
}

__global__ void __launch_bounds__(kOrderThreads) order_kernel(const int* __restrict__ ids, int pairs,
                                                              int choices, int experts,
                                                              int* __restrict__ start,
                                                              int* __restrict__ source,
                                                              int* __restrict__ place) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const unsigned expert = blockIdx.x;
    const bool rest = (int)expert == experts;
    // each warp has a run of whole groups of 128 ids
    const int groups = (pairs + 127) / 128, per = (groups + warps - 1) / warps;
    const long long begin = (long long)warp * per * 128;
    const long long end = min((long long)pairs, begin + (long long)per * 128);
    int less = 0, mine = 0;
    for (long long at = begin + 4 * lane; at - 4 * lane < end; at += 128) {
        int v[4];
        load4(ids, at, end, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            less += (unsigned)v[i] < expert;
            mine += (unsigned)v[i] == expert;
        }
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        less += __shfl_xor_sync(0xffffffffu, less, d);
        mine += __shfl_xor_sync(0xffffffffu, mine, d);
    }
    __shared__ int part[2][32];
    if (lane == 0) {
        part[0][warp] = less;
        part[1][warp] = rest ? 0 : mine;
    }
    __syncthreads();
    int all = lane < warps ? part[0][lane] : 0, before = lane < warp ? part[1][lane] : 0;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        all += __shfl_xor_sync(0xffffffffu, all, d);
        before += __shfl_xor_sync(0xffffffffu, before, d);
    }
    if (threadIdx.x == 0) start[expert] = all;
    if (rest) {
        for (int r = all + threadIdx.x; r < pairs; r += blockDim.x) source[r] = -1;
        for (int i = threadIdx.x; i < pairs; i += blockDim.x)
            if ((unsigned)ids[i] >= (unsigned)experts) place[i] = -1;
        return;
    }
    if (mine == 0) return;
    int row = all + before;
    const unsigned below = (1u << lane) - 1;
    for (long long at = begin + 4 * lane; at - 4 * lane < end; at += 128) {
        int v[4];
        load4(ids, at, end, v);
        // rows of a group: lanes in order, each with its four
        int own = 0, ahead = 0, sum = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const unsigned b = __ballot_sync(0xffffffffu, (unsigned)v[i] == expert);
            ahead += __popc(b & below);
            sum += __popc(b);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if ((unsigned)v[i] == expert) {
                const int r = row + ahead + own++;
                source[r] = (int)(at + i) / choices;
                place[at + i] = r;
            }
        row += sum;
    }
}

__global__ void __launch_bounds__(kSumThreads) sum_kernel(const uint4* __restrict__ y, int rows,
                                                          const int* __restrict__ place,
                                                          const float* __restrict__ weights,
                                                          long long vectors, int choices, int vecs,
                                                          uint4* __restrict__ out) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const long long at = blockIdx.x * (long long)kSumThreads + threadIdx.x;
    if (at >= vectors) return;
    const long long token = at / vecs;
    const int c = (int)(at - token * vecs);
    float sum[8] = {};
    for (int base = 0; base < choices; base += kAhead) {
        uint4 v[kAhead];
        float w[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            v[j] = make_uint4(0, 0, 0, 0);
            w[j] = 0.0f;
            if (base + j < choices) {
                const int p = place[token * choices + base + j];
                if (p >= 0 && p < rows) {
                    w[j] = weights[token * choices + base + j];
                    v[j] = y[(size_t)p * vecs + c];
                }
            }
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const uint32_t u[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                sum[2 * i] = fmaf(w[j], bf16_lo(u[i]), sum[2 * i]);
                sum[2 * i + 1] = fmaf(w[j], bf16_hi(u[i]), sum[2 * i + 1]);
            }
        }
    }
    out[at] = make_uint4(bf16x2(sum[0], sum[1]), bf16x2(sum[2], sum[3]), bf16x2(sum[4], sum[5]),
                         bf16x2(sum[6], sum[7]));
}

template <typename... Args>
cudaError_t launch(void (*kernel)(Args...), unsigned blocks, int threads, cudaStream_t s,
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

}  // namespace

cudaError_t launch_experts_order(const int* ids, int tokens, int choices, int experts, int* start,
                                 int* source, int* place, cudaStream_t s) {
    const int pairs = tokens * choices, groups = (pairs + 127) / 128;
    const int threads = groups < kOrderThreads / 32 ? groups * 32 : kOrderThreads;
    return launch(order_kernel, (unsigned)experts + 1, threads, s, ids, pairs, choices, experts,
                  start, source, place);
}

cudaError_t launch_experts_sum(const void* y, int rows, const int* place, const float* weights,
                               int tokens, int choices, int H, void* out, cudaStream_t s) {
    const long long vectors = (long long)tokens * (H / 8);
    return launch(sum_kernel, (unsigned)((vectors + kSumThreads - 1) / kSumThreads), kSumThreads, s,
                  reinterpret_cast<const uint4*>(y), rows, place, weights, vectors, choices, H / 8,
                  reinterpret_cast<uint4*>(out));
}

}  // namespace nvf
