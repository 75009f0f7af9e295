// experts.cu -- a routed batch's lists and its sums.
//
// Order: ids [tokens, choices] sorted by expert, stable, from which come each
// expert's first row, each row's token and each pair's row.  One block per expert
// goes through all ids (they stay in L2): it counts those of lower experts, which
// gives its first row, and its own, which a prefix sum over the block puts in order.
// No block needs another's result, so one launch does it, at a cost of experts * ids
// compares.  One more block has the ids of no expert and the rows behind the last.
// Long lists are cut into chunks of 1024 ids instead, in three launches: each chunk's
// count by expert, first rows from the sums of these over chunks and experts, and each
// chunk's rows.  The counts lie in the chunk's own part of `place`, which only the last
// launch's block of that chunk reads, and then writes.
//
// Sum: out[t] = bf16(sum_j weights[t][j] * y[place[t][j]]), fp32, in the order of j.
// Bound by memory: every thread has 8 columns of a token and asks for its rows four or
// eight at once (8192 tokens of 8 rows of 4096: 91 us, 6.6 TB/s; 4096 of 4: 27.4 us, 6.1,
// with eight asked for there too 33.6).
#include <atomic>

#include "kv8.cuh"
#include "w4a4.h"

namespace nvf {

namespace {

constexpr int kOrderThreads = 1024;
constexpr int kManyPairs = 24576;
constexpr long long kManyCompares = 1 << 20;
constexpr int kSumThreads = 256;

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
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
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
            const unsigned same = __ballot_sync(0xffffffffu, (unsigned)v[i] == expert);
            ahead += __popc(same & below);
            sum += __popc(same);
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

// Chunk c of a long list: ids c * kChunk on, the last one with what is left (up to
// 2 * kChunk - 1), so that each has at least as many ids as there may be experts.
constexpr int kChunk = 1024;
static_assert(kW4MaxExperts <= kChunk, "counts lie in the chunk's places");

__device__ __forceinline__ int chunk_end(int chunk, int chunks, int pairs) {
    return chunk + 1 < chunks ? (chunk + 1) * kChunk : pairs;
}

__global__ void __launch_bounds__(kChunk) chunk_count_kernel(const int* __restrict__ ids, int pairs,
                                                             int experts, int* __restrict__ place) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __shared__ int counts[kW4MaxExperts];
    const int tid = threadIdx.x, begin = blockIdx.x * kChunk;
    const int end = chunk_end(blockIdx.x, gridDim.x, pairs);
    if (tid < experts) counts[tid] = 0;
    __syncthreads();
    for (int i = begin + tid; i < end; i += kChunk) {
        const int id = ids[i];
        if ((unsigned)id < (unsigned)experts) atomicAdd(&counts[id], 1);
    }
    __syncthreads();
    if (tid < experts) place[begin + tid] = counts[tid];
}

// Turns the chunks' counts into their rows: sums over the experts and chunks in front.
// One block, in which several threads share the chunks of an expert.
__global__ void __launch_bounds__(1024) chunk_sum_kernel(int chunks, int experts,
                                                         int* __restrict__ start,
                                                         int* __restrict__ place) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __shared__ int total[kW4MaxExperts], part[32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int e = tid; e < experts; e += 1024) total[e] = 0;
    __syncthreads();
    // neighbouring threads take neighbouring experts; 1024 / group of them share one
    const int group = (experts + 31) / 32 * 32, sharers = 1024 / group;
    const int e = tid % group, share = tid / group;
    const int per = (chunks + sharers - 1) / sharers;
    const int c0 = min(share * per, chunks), c1 = min(c0 + per, chunks);
    __shared__ int front[1024];
    int sum = 0;
    if (e < experts && share < sharers)
#pragma unroll 8
        for (int c = c0; c < c1; ++c) sum += place[(size_t)c * kChunk + e];
    front[tid] = sum;
    __syncthreads();
    int before = 0, all = 0;
    if (e < experts && share < sharers) {
        for (int s = 0; s < sharers; ++s) {
            const int n = front[s * group + e];
            if (s < share) before += n;
            all += n;
        }
        if (share == 0) total[e] = all;
    }
    __syncthreads();
    // first rows: a sum over the experts in front (thread t has expert t)
    int mine = tid < experts ? total[tid] : 0, upto = mine;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const int o = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d) upto += o;
    }
    if (lane == 31) part[warp] = upto;
    __syncthreads();
    int warps_before = lane < warp ? part[lane] : 0;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        warps_before += __shfl_xor_sync(0xffffffffu, warps_before, d);
    upto += warps_before;
    __syncthreads();
    if (tid < experts) {
        start[tid] = upto - mine;
        total[tid] = upto - mine;
        if (tid == experts - 1) start[experts] = upto;
    }
    __syncthreads();
    if (e < experts && share < sharers) {
        int row = total[e] + before;
#pragma unroll 8
        for (int c = c0; c < c1; ++c) {
            const int n = place[(size_t)c * kChunk + e];
            place[(size_t)c * kChunk + e] = row;
            row += n;
        }
    }
}

// A chunk's rows: each warp's 32 ids are ranked among themselves, its counts by expert
// summed over the warps in front.  counts: [32 warps][experts].
__global__ void __launch_bounds__(kChunk) chunk_place_kernel(const int* __restrict__ ids, int pairs,
                                                             int choices, int experts,
                                                             const int* __restrict__ start,
                                                             int* __restrict__ source,
                                                             int* __restrict__ place) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    extern __shared__ int counts[];
    __shared__ int first[kW4MaxExperts];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int begin = blockIdx.x * kChunk, end = chunk_end(blockIdx.x, gridDim.x, pairs);
    if (tid < experts) first[tid] = place[begin + tid];
    for (int at = begin; at < end; at += kChunk) {
        for (int i = tid; i < 32 * experts; i += kChunk) counts[i] = 0;
        __syncthreads();
        const int i = at + tid;
        int id = i < end ? ids[i] : -1;
        if ((unsigned)id >= (unsigned)experts) id = -1;
        const unsigned same = __match_any_sync(0xffffffffu, id);
        if (id >= 0 && lane == __ffs(same) - 1) counts[warp * experts + id] = __popc(same);
        __syncthreads();
        if (tid < experts) {
            int row = first[tid];
#pragma unroll 8
            for (int w = 0; w < 32; ++w) {
                const int n = counts[w * experts + tid];
                counts[w * experts + tid] = row;
                row += n;
            }
            first[tid] = row;
        }
        __syncthreads();
        int row = -1;
        if (id >= 0) {
            row = counts[warp * experts + id] + __popc(same & ((1u << lane) - 1));
            source[row] = i / choices;
        }
        if (i < end) place[i] = row;
        __syncthreads();
    }
    // rows behind the last expert's
    for (long long r = start[experts] + (long long)blockIdx.x * kChunk + tid; r < pairs;
         r += (long long)gridDim.x * kChunk)
        source[r] = -1;
}

// `share` threads, a power of two, have a token's next 8 * share columns.
template <int kAhead>
__global__ void __launch_bounds__(kSumThreads) sum_kernel(const uint4* __restrict__ y, int rows,
                                                          const int* __restrict__ place,
                                                          const float* __restrict__ weights,
                                                          int tokens, int choices, int vecs,
                                                          int share, uint4* __restrict__ out) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int token = blockIdx.x * (kSumThreads / share) + threadIdx.x / share;
    const int c = blockIdx.y * share + threadIdx.x % share;
    if (token >= tokens || c >= vecs) return;
    place += (size_t)token * choices;
    weights += (size_t)token * choices;
    uint64_t sum[4] = {};  // pairs
    for (int base = 0; base < choices; base += kAhead) {
        uint4 v[kAhead];
        float w[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            v[j] = make_uint4(0, 0, 0, 0);
            w[j] = 0.0f;
            if (base + j < choices) {
                const int p = place[base + j];
                if (p >= 0 && p < rows) {
                    w[j] = weights[base + j];
                    v[j] = y[(size_t)p * vecs + c];
                }
            }
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const uint32_t u[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
            const uint64_t w2 = pair(w[j], w[j]);
#pragma unroll
            for (int i = 0; i < 4; ++i) sum[i] = fma2(w2, pair(bf16_lo(u[i]), bf16_hi(u[i])), sum[i]);
        }
    }
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 s = unpair(sum[i]);
        o[i] = bf16x2(s.x, s.y);
    }
    out[(size_t)token * vecs + c] = make_uint4(o[0], o[1], o[2], o[3]);
}

template <typename... Args>
cudaError_t launch(void (*kernel)(Args...), dim3 blocks, int threads, size_t shared,
                   cudaStream_t s, Args... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = blocks;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = shared;
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
    if (pairs >= kManyPairs && (long long)pairs * experts >= kManyCompares) {
        static std::atomic<bool> allowed[64];  // per device: the shared memory limit is set
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        if (dev >= 64 || !allowed[dev].load(std::memory_order_acquire)) {
            e = cudaFuncSetAttribute(chunk_place_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     32 * kW4MaxExperts * (int)sizeof(int));
            if (e != cudaSuccess) return e;
            if (dev < 64) allowed[dev].store(true, std::memory_order_release);
        }
        const int chunks = pairs / kChunk;
        e = launch(chunk_count_kernel, dim3(chunks), kChunk, 0, s, ids, pairs, experts, place);
        if (e != cudaSuccess) return e;
        e = launch(chunk_sum_kernel, dim3(1), 1024, 0, s, chunks, experts, start, place);
        if (e != cudaSuccess) return e;
        return launch(chunk_place_kernel, dim3(chunks), kChunk, 32 * experts * sizeof(int), s,
                      ids, pairs, choices, experts, (const int*)start, source, place);
    }
    const int threads = groups < kOrderThreads / 32 ? groups * 32 : kOrderThreads;
    return launch(order_kernel, dim3(experts + 1), threads, 0, s, ids, pairs, choices, experts,
                  start, source, place);
}

cudaError_t launch_experts_sum(const void* y, int rows, const int* place, const float* weights,
                               int tokens, int choices, int H, void* out, cudaStream_t s) {
    const int vecs = H / 8;
    // as many threads as leave an eighth of them idle at most (rows of 250 vectors: 256
    // threads; 672: 64), or a warp of them, and of a short row what it takes
    int share = kSumThreads;
    while (share > 32 && (vecs + share - 1) / share * share - vecs > vecs / 8) share /= 2;
    while (share / 2 >= vecs) share /= 2;
    const int at_once = kSumThreads / share;
    const dim3 grid((tokens + at_once - 1) / at_once, (vecs + share - 1) / share);
    return launch(choices <= 4 ? sum_kernel<4> : sum_kernel<8>, grid, kSumThreads, 0, s,
                  reinterpret_cast<const uint4*>(y), rows, place, weights, tokens, choices, vecs,
                  share, reinterpret_cast<uint4*>(out));
}

}  // namespace nvf
