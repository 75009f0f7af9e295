// w4a4_gemm.cu -- products of NVFP4 rows with NVFP4 weights on the FP4 tensor
// cores (tcgen05, block-scaled), dense or grouped by expert:
//
//   out[m][n] = bf16(r_m * (scale2 * sum_k x[m][k] w[n][k]))
//   or, of a gate/up pair, bf16(act(g) * u) with g and u such sums in bf16.
//
// The weight's rows are the 128 lanes of an accumulator, tokens its columns, up to
// kTokens of them, so that a few tokens cost few columns and a tile of the weight
// is read once for all of them.  One thread copies tiles into a ring of stages (a
// bulk copy each, see w4a4.h), one issues products: per stage the scales go to
// tensor memory (the tensor cores read them there) and four products of 64 elements
// follow.  Eight warps read the sums out, a weight row per lane.  They pack them to
// bf16 and give the accumulator back before they store, so a tile's stores run
// beside the next one's products.
//
// Work: whole tiles in turn, then the tiles that are left over (fewer than blocks)
// are cut along K into equal ranges, one per block.  A range that is not all of its
// tile leaves its sums in the workspace; the block that comes last adds all parts
// up in the order of their ranges, so results do not depend on timing, and no block
// waits for another.
#include <atomic>

#include "internal.h"
#include "kv8.cuh"
#include "tmem.cuh"
#include "w4a4.h"

namespace nvf {

namespace {

constexpr int kEpilogueWarps = 8;
constexpr int kThreads = (2 + kEpilogueWarps) * 32;
constexpr int kEpilogueThreads = kEpilogueWarps * 32;
// Token tiles that take turns with one weight tile before the next one: their tiles
// (16 x 256 tokens of K = 17408: 40 MB) stay in L2 for it.
constexpr int kSuper = 16;
// K blocks that a range of a cut tile has at least.
constexpr int kLeastRange = 2;

template <int kTokens>
struct Shape {
    static constexpr int kStages = kTokens == 256 ? 4 : 6;
    static constexpr int kSums = kTokens == 256 ? 1 : 2;  // accumulators in turn
    static constexpr int kBAt = kW4Tile;                  // tokens' codes in a stage
    static constexpr int kBScalesAt = kBAt + kTokens * 128;
    static constexpr int kStageBytes = kBScalesAt + kTokens * 16;
    static constexpr int kShared = 1024 + kStages * kStageBytes;
    // tensor memory: accumulators, then each stage's scales
    static constexpr int kScalesAt = kTokens * kSums;
    static constexpr int kScaleColumns = 16 + kTokens / 8;  // per stage
    static_assert(kScalesAt + kStages * kScaleColumns <= 512, "tensor memory");
    static constexpr int kPartial = kW4Rows * kTokens;  // floats
};

struct Args {
    const uint8_t* rows;
    const float* row_scales;
    const uint8_t* packed;
    __nv_bfloat16* out;
    const int* start;
    const float* scales_a;
    const float* scales_b;
    float scale_a, scale_b;
    int M, N, k_blocks, row_blocks, experts, act;
    int* status;
    int* counters;
    float* partials;
    unsigned long long wait_ns;
    int stall;
};

// A range of K blocks of one tile.
struct Item {
    int expert, weight, token0, tokens;  // row block of the weight; first row, rows
    long long block;                     // first tile of the rows
    int kb0, kb1;
    int parts, first_part, left_over;    // parts > 1: blocks first_part .. + parts - 1
};

// The block's list of work.  prefix[e]: token tiles of the experts in front of e.
template <int kTokens>
struct Schedule {
    const Args& a;
    const int* prefix;
    int tiles, whole, sharers;
    long long left;  // K blocks of the tiles that are left over
    int next, range0, range1;

    __device__ Schedule(const Args& args, const int* tile_prefix) : a(args), prefix(tile_prefix) {
        const int P = gridDim.x;
        tiles = prefix[a.experts] * a.row_blocks;
        whole = tiles / P * P;
        left = (long long)(tiles - whole) * a.k_blocks;
        const long long most = left / min(kLeastRange, a.k_blocks);
        sharers = most < P ? (most > 0 ? (int)most : (left > 0 ? 1 : 0)) : P;
        next = blockIdx.x;
        range0 = range1 = 0;
        if ((int)blockIdx.x < sharers) {
            range0 = (int)(left * blockIdx.x / sharers);
            range1 = (int)(left * (blockIdx.x + 1) / sharers);
        }
    }

    // The sharer whose range holds K block p of the left-over tiles.
    __device__ int sharer(int p) const {
        return (int)(((long long)(p + 1) * sharers + left - 1) / left) - 1;
    }

    __device__ void place(int tile, Item& it) const {
        // the last expert with prefix * row_blocks <= tile
        int lo = 0, hi = a.experts - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (prefix[mid] * a.row_blocks <= tile) lo = mid;
            else hi = mid - 1;
        }
        const int of_expert = prefix[lo + 1] - prefix[lo];
        int at = tile - prefix[lo] * a.row_blocks;
        const int super = at / (kSuper * a.row_blocks);
        at -= super * kSuper * a.row_blocks;
        const int width = min(kSuper, of_expert - super * kSuper);
        const int t = super * kSuper + at % width;
        it.expert = lo;
        it.weight = at / width;
        const int first = a.start ? a.start[lo] : 0, end = a.start ? a.start[lo + 1] : a.M;
        it.token0 = first + t * kTokens;
        it.tokens = min(kTokens, end - it.token0);
        it.block = first / kW4Rows + lo + (long long)t * (kTokens / kW4Rows);
    }

    // Where a block's sums of a cut tile lie.  Of a block's ranges only the first and
    // the last can be parts of tiles; the last begins in front of its tile's share.
    __device__ float4* part(int block, const Item& it) const {
        const int begin = it.left_over * a.k_blocks;
        const bool second = (int)(left * block / sharers) < begin;
        return reinterpret_cast<float4*>(a.partials +
                                         ((size_t)block * 2 + second) * Shape<kTokens>::kPartial);
    }

    __device__ bool take(Item& it) {
        it.parts = 1;
        if (next < whole) {
            place(next, it);
            it.kb0 = 0;
            it.kb1 = a.k_blocks;
            next += gridDim.x;
            return true;
        }
        if (range0 >= range1) return false;
        const int tile = range0 / a.k_blocks, begin = tile * a.k_blocks, end = begin + a.k_blocks;
        place(whole + tile, it);
        it.kb0 = range0 - begin;
        it.kb1 = min(range1, end) - begin;
        it.left_over = tile;
        it.first_part = sharer(begin);
        it.parts = sharer(end - 1) - it.first_part + 1;
        range0 = min(range1, end);
        return true;
    }
};

// kind::mxf4nvf4: E2M1 by E2M1, E4M3 scales, fp32 sums, 128 rows, n columns, 64 deep.
__device__ __forceinline__ constexpr uint32_t instruction(int n) {
    return 1u << 7 | 1u << 10 | (uint32_t)(n / 8) << 17 | (uint32_t)(128 / 128) << 27;
}

// Shared-memory descriptors: rows of 128 bytes in the 128-byte swizzle, eight to a
// kilobyte; and 32 rows of 16 bytes, plain, eight to 128 bytes.
__device__ __forceinline__ uint64_t operand(uint32_t at) {
    return (uint64_t)((at & 0x3ffffu) >> 4) | (uint64_t)(1024 >> 4) << 32 | 1ull << 46 | 2ull << 61;
}
__device__ __forceinline__ uint64_t scale_operand(uint32_t at) {
    return (uint64_t)((at & 0x3ffffu) >> 4) | (uint64_t)(128 >> 4) << 32 | 1ull << 46;
}

__device__ __forceinline__ void copy_scales(uint32_t columns, uint64_t from) {
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(columns), "l"(from)
                 : "memory");
}

__device__ __forceinline__ void multiply(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                         uint32_t scales_a, uint32_t scales_b, bool add) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
        " tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, "
        "[%4], [%5], p;\n}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(scales_a), "r"(scales_b), "r"(add ? 1 : 0)
        : "memory");
}

// `bar` completes when all products issued so far have.
__device__ __forceinline__ void commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                     bar)
                 : "memory");
}

// act(g) * u for g and u in bf16: act(g) = g * sigmoid(y), y = g or the argument of GeLU's
// tanh, doubled.  g * u is exact in fp32, and for y > 0 what sigmoid takes away from
// it is subtracted, with one rounding.  Where that is too little for fp32, g * u itself
// may be a tie of bf16 (it has 16 bits); the result is below it, so it goes towards 0.
__device__ __forceinline__ float gated(int act, float g, float u) {
    const float y = act == 0 ? g : 1.5957691216057308f * (g + 0.044715f * g * g * g);
    const float e = __expf(-fabsf(y)), s = __fdividef(e, 1.0f + e);  // sigmoid(-|y|)
    if (!(y > 0.0f)) return g * s * u;
    const float t = g * u;
    const float p = fabsf(t) < INFINITY ? fmaf(-t, s, t) : t;
    const uint32_t bits = __float_as_uint(p);
    return p == t && (bits & 0xffffu) == 0x8000u ? __uint_as_float(bits - 1) : p;
}

struct Barriers {
    uint64_t full[8], empty[8];        // stages
    uint64_t sums_full[2], sums_empty[2];
    uint64_t drained;                  // after a wait that ran out
};

template <int kTokens, bool kGated>
__global__ void __launch_bounds__(kThreads, 1) w4a4_gemm_kernel(const Args a) {
    using S = Shape<kTokens>;
    extern __shared__ __align__(1024) uint8_t dynamic[];
    // the swizzle goes by address: stages begin on multiples of 1024
    uint8_t* const shared = dynamic + (-smem_addr(dynamic) & 1023u);
    __shared__ Barriers bars;
    __shared__ int prefix[kW4MaxExperts + 1];
    __shared__ alignas(16) float row_scale[2][kTokens];  // of two tiles in turn, read in pairs
    __shared__ int last_part;
    __shared__ volatile int abort;
    __shared__ uint32_t tmem_at;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t smem = smem_addr(shared);
    constexpr int kCopyWarp = 0, kIssueWarp = 1;

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (warp == kIssueWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                         smem_addr(&tmem_at))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (tid == 0) {
        for (int i = 0; i < S::kStages; ++i) {
            mbar_init(smem_addr(&bars.full[i]), 1);
            mbar_init(smem_addr(&bars.empty[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_addr(&bars.sums_full[i]), 1);
            mbar_init(smem_addr(&bars.sums_empty[i]), kEpilogueWarps);
        }
        mbar_init(smem_addr(&bars.drained), 1);
        abort = 0;
        fence_mbar_init();
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // token tiles of each expert; one whose rows are not all inside has none
    if (tid == 0) prefix[0] = 0;
    for (int e = tid; e < a.experts; e += kThreads) {
        const int first = a.start ? a.start[e] : 0, end = a.start ? a.start[e + 1] : a.M;
        prefix[e + 1] = first >= 0 && end <= a.M && end > first
                            ? (end - first + kTokens - 1) / kTokens
                            : 0;
    }
    __syncthreads();
    if (warp == 2 && a.experts > 1) {
        int sum = 0;
        for (int base = 1; base <= a.experts; base += 32) {
            int v = base + lane <= a.experts ? prefix[base + lane] : 0;
#pragma unroll
            for (int d = 1; d < 32; d *= 2) {
                const int o = __shfl_up_sync(0xffffffffu, v, d);
                if (lane >= d) v += o;
            }
            if (base + lane <= a.experts) prefix[base + lane] = sum + v;
            sum += __shfl_sync(0xffffffffu, v, 31);
        }
    }
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = tmem_at;

    // Waits for a barrier's completion number `uses` (from 0); false, with the status
    // set, when it does not come in time.
    auto wait_lane = [&](uint64_t& bar, unsigned uses) {
        if (mbar_wait_bounded(smem_addr(&bar), uses & 1, &abort, a.wait_ns)) return true;
        abort = 1;
        *a.status = kKv8Timeout;
        return false;
    };

    Schedule<kTokens> schedule(a, prefix);
    Item it;
    if (warp == kCopyWarp && lane == 0) {
        unsigned n = 0;  // stages filled
        bool ok = true;
        while (ok && schedule.take(it)) {
            const uint8_t* w = a.packed + ((size_t)it.expert * a.row_blocks + it.weight) *
                                              a.k_blocks * kW4Tile;
            const uint8_t* x = a.rows + (size_t)it.block * a.k_blocks * kW4Tile;
            const size_t block_bytes = (size_t)a.k_blocks * kW4Tile;
            // eight rows of 128 bytes at a time
            const uint32_t codes0 = (uint32_t)((min(it.tokens, 128) + 15) / 16 * 2048);
            const uint32_t codes1 = (uint32_t)((max(it.tokens - 128, 0) + 15) / 16 * 2048);
            const uint32_t bytes = kW4Tile + codes0 + kW4Scales + (codes1 ? codes1 + kW4Scales : 0);
            for (int kb = it.kb0; kb < it.kb1; ++kb, ++n) {
                const int stage = n % S::kStages;
                if (n >= S::kStages) {
                    ok = wait_lane(bars.empty[stage], n / S::kStages - 1);
                    if (!ok) break;
                }
                if (a.stall && n >= 1) {  // testing: nothing comes any more
                    wait_lane(bars.drained, 0);
                    ok = false;
                    break;
                }
                const uint32_t bar = smem_addr(&bars.full[stage]);
                const uint32_t at = smem + stage * S::kStageBytes;
                mbar_arrive_expect_tx(bar, bytes);
                bulk_copy_g2s(at, w + (size_t)kb * kW4Tile, kW4Tile, bar);
                const uint8_t* t = x + (size_t)kb * kW4Tile;
                bulk_copy_g2s(at + S::kBAt, t, codes0, bar);
                bulk_copy_g2s(at + S::kBScalesAt, t + kW4Codes, kW4Scales, bar);
                if (codes1) {
                    t += block_bytes;
                    bulk_copy_g2s(at + S::kBAt + kW4Codes, t, codes1, bar);
                    bulk_copy_g2s(at + S::kBScalesAt + kW4Scales, t + kW4Codes, kW4Scales, bar);
                }
            }
        }
        if (abort) {
            // copies under way end before the memory that they write is left; these waits
            // heed nobody's
            const int none = 0;
            for (unsigned i = n > S::kStages ? n - S::kStages : 0; i < n; ++i)
                mbar_wait_bounded(smem_addr(&bars.full[i % S::kStages]), i / S::kStages & 1, &none);
        }
    } else if (warp == kIssueWarp && lane == 0) {
        unsigned n = 0, items = 0;
        bool ok = true;
        while (ok && schedule.take(it)) {
            const unsigned sums = items % S::kSums;
            if (items >= S::kSums) {
                ok = wait_lane(bars.sums_empty[sums], items / S::kSums - 1);
                if (!ok) break;
            }
            tmem_fence_after();
            const uint32_t d = tmem + sums * kTokens;
            const int columns = (it.tokens + 15) / 16 * 16;
            const uint32_t idesc = instruction(columns);
            for (int kb = it.kb0; kb < it.kb1; ++kb, ++n) {
                const int stage = n % S::kStages;
                ok = wait_lane(bars.full[stage], n / S::kStages);
                if (!ok) break;
                const uint32_t at = smem + stage * S::kStageBytes;
                // the stage's own columns: what read them last has completed, as the
                // stage was filled again
                const uint32_t scales_a = tmem + S::kScalesAt + stage * S::kScaleColumns;
                const uint32_t scales_b = scales_a + 16;
                const uint64_t from_a = scale_operand(at + kW4Codes);
                const uint64_t from_b = scale_operand(at + S::kBScalesAt);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    copy_scales(scales_a + 4 * j, from_a + j * (512 >> 4));
                    copy_scales(scales_b + j * (kTokens / 32), from_b + j * (512 >> 4));
                    if (kTokens == 256 && columns > 128)
                        copy_scales(scales_b + j * (kTokens / 32) + 4,
                                    from_b + (kW4Scales >> 4) + j * (512 >> 4));
                }
                const uint64_t op_a = operand(at), op_b = operand(at + S::kBAt);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    multiply(d, op_a + j * 2, op_b + j * 2, idesc, scales_a + 4 * j,
                             scales_b + j * (kTokens / 32), kb > it.kb0 || j > 0);
                commit(smem_addr(&bars.empty[stage]));
            }
            if (!ok) break;
            commit(smem_addr(&bars.sums_full[sums]));
            ++items;
        }
        if (abort) {
            // products under way end before the memory that they read is left
            const int none = 0;
            commit(smem_addr(&bars.drained));
            mbar_wait_bounded(smem_addr(&bars.drained), 0, &none);
        }
    } else if (warp >= 2) {
        const int quadrant = warp & 3, half = (warp - 2) >> 2, eid = tid - 64;
        constexpr int kHalf = kTokens / 2, kChunks = kHalf / 32;
        const int row = quadrant * 32 + lane;  // of the weight's tile
        const uint32_t lanes = tmem + ((uint32_t)(quadrant * 32) << 16);
        bool ok = true;
        for (unsigned items = 0; schedule.take(it); ++items) {
            const unsigned sums = items % S::kSums;
            // chunks of 32 tokens that this warp has
            const int mine = min(max((it.tokens - half * kHalf + 31) / 32, 0), kChunks);
            float* const scales = row_scale[items & 1];
            ok = ok && __all_sync(0xffffffffu, wait_lane(bars.sums_full[sums], items / S::kSums));
            if (ok && eid < kTokens)
                scales[eid] = eid < it.tokens ? a.row_scales[it.token0 + eid] : 0.0f;
            tmem_fence_after();
            const uint32_t from = lanes + sums * kTokens + half * kHalf;
            const bool up = kGated && lane >= 16;
            const float scale = up ? (a.scales_b ? a.scales_b[it.expert] : a.scale_b)
                                   : (a.scales_a ? a.scales_a[it.expert] : a.scale_a);
            named_barrier_sync(1, kEpilogueThreads);  // row scales are there
            uint32_t p[kChunks][16];  // pairs of tokens, bf16
            auto pack = [&](int c, const float(&x)[32]) {
                const float2* r = reinterpret_cast<const float2*>(scales + half * kHalf + 32 * c);
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    p[c][j] = bf16x2(x[2 * j] * scale * r[j].x, x[2 * j + 1] * scale * r[j].y);
            };
            auto give_back = [&] {
                tmem_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&bars.sums_empty[sums]));
            };
            bool store = ok;
            if (it.parts == 1) {
                if (ok) {
#pragma unroll
                    for (int c = 0; c < kChunks; ++c)
                        if (c < mine) {
                            float x[32];
                            tmem_load32(from + 32 * c, x);
                            tmem_wait_load(x);
                            pack(c, x);
                        }
                }
                give_back();
            } else {
                float4* to = schedule.part(blockIdx.x, it) + half * (kHalf / 4) * kW4Rows + row;
                if (ok) {
#pragma unroll
                    for (int c = 0; c < kChunks; ++c)
                        if (c < mine) {
                            float x[32];
                            tmem_load32(from + 32 * c, x);
                            tmem_wait_load(x);
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                to[(8 * c + j) * kW4Rows] =
                                    make_float4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]);
                        }
                }
                give_back();
                __threadfence();
                named_barrier_sync(1, kEpilogueThreads);
                // an abandoned range is counted too: the counter is left at 0 all the same
                if (eid == 0) {
                    int* const counter = a.counters + it.left_over;
                    const bool last = atom_add_acq_rel_gpu(counter, 1) == it.parts - 1;
                    if (last) *counter = 0;
                    last_part = last;
                }
                named_barrier_sync(1, kEpilogueThreads);
                store = ok && last_part;
                if (store) {
                    __threadfence();
#pragma unroll
                    for (int c = 0; c < kChunks; ++c)
                        if (c < mine) {
                            float x[32];
#pragma unroll
                            for (int j = 0; j < 32; ++j) x[j] = 0.0f;
                            for (int i = 0; i < it.parts; ++i) {
                                const float4* part = schedule.part(it.first_part + i, it) +
                                                     half * (kHalf / 4) * kW4Rows + row;
#pragma unroll
                                for (int j = 0; j < 8; ++j) {
                                    const float4 y = __ldcg(part + (8 * c + j) * kW4Rows);
                                    x[4 * j] += y.x;
                                    x[4 * j + 1] += y.y;
                                    x[4 * j + 2] += y.z;
                                    x[4 * j + 3] += y.w;
                                }
                            }
                            pack(c, x);
                        }
                }
            }
            if (!store) continue;
            const int t0 = half * kHalf;
            if (kGated) {
                // 16 lanes have gate, 16 up, of the same features: the first take the even
                // tokens, the others the odd ones, then neighbours trade for two features
                const int feature = it.weight * 64 + quadrant * 16 + (lane & 14);
                if (feature < a.N) {
                    __nv_bfloat16* const out = a.out + (size_t)it.token0 * a.N + feature;
#pragma unroll
                    for (int c = 0; c < kChunks; ++c)
                        if (c < mine) {
#pragma unroll
                            for (int j = 0; j < 16; j += 2) {
                                float h[2];
#pragma unroll
                                for (int k = 0; k < 2; ++k) {
                                    const uint32_t v = p[c][j + k];
                                    const uint32_t o = __shfl_xor_sync(0xffffffffu, v, 16);
                                    h[k] = gated(a.act, up ? bf16_hi(o) : bf16_lo(v),
                                                 up ? bf16_hi(v) : bf16_lo(o));
                                }
                                const uint32_t v = bf16x2(h[0], h[1]);
                                const uint32_t o = __shfl_xor_sync(0xffffffffu, v, 1);
                                const uint32_t w =
                                    lane & 1 ? prmt(o, v, 0x7632) : prmt(v, o, 0x5410);
                                const int token =
                                    t0 + 32 * c + 2 * j + (up ? 1 : 0) + 2 * (lane & 1);
                                if (token < it.tokens)
                                    *reinterpret_cast<uint32_t*>(out + (size_t)token * a.N) = w;
                            }
                        }
                }
            } else {
                const int feature = it.weight * kW4Rows + row;
                __nv_bfloat16* const out = a.out + (size_t)it.token0 * a.N + feature;
                if (a.N & 1) {
#pragma unroll
                    for (int c = 0; c < kChunks; ++c)
                        if (c < mine && feature < a.N) {
#pragma unroll
                            for (int j = 0; j < 32; ++j) {
                                const int token = t0 + 32 * c + j;
                                const uint32_t v = p[c][j / 2];
                                if (token < it.tokens)
                                    *reinterpret_cast<uint16_t*>(out + (size_t)token * a.N) =
                                        (uint16_t)(j & 1 ? v >> 16 : v);
                            }
                        }
                } else {
                    // neighbours trade: an even lane has both features of an even token
#pragma unroll
                    for (int c = 0; c < kChunks; ++c)
                        if (c < mine) {
#pragma unroll
                            for (int j = 0; j < 16; ++j) {
                                const uint32_t v = p[c][j];
                                const uint32_t o = __shfl_xor_sync(0xffffffffu, v, 1);
                                const uint32_t w =
                                    lane & 1 ? prmt(o, v, 0x7632) : prmt(v, o, 0x5410);
                                const int token = t0 + 32 * c + 2 * j + (lane & 1);
                                if (token < it.tokens && feature < a.N)
                                    *reinterpret_cast<uint32_t*>(out + (size_t)token * a.N -
                                                                 (lane & 1)) = w;
                            }
                        }
                }
            }
        }
    }
    tmem_fence_before();
    __syncthreads();
    if (warp == kIssueWarp)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem)
                     : "memory");
}

template <int kTokens, bool kGated>
cudaError_t launch(const Args& a, int num_sms, cudaStream_t s) {
    static std::atomic<bool> allowed[64];  // per device: the kernel's shared memory limit is set
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !allowed[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(w4a4_gemm_kernel<kTokens, kGated>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 Shape<kTokens>::kShared);
        if (e != cudaSuccess) return e;
        if (dev < 64) allowed[dev].store(true, std::memory_order_release);
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(num_sms);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Shape<kTokens>::kShared;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, w4a4_gemm_kernel<kTokens, kGated>, a);
}

// Tokens per tile: rows of an expert on average, as far as the host knows them.
bool wide(int M, int experts) { return M > 128LL * experts; }

}  // namespace

size_t w4_partial_bytes(int M, int experts, int num_sms) {
    return (size_t)num_sms * 2 * kW4Rows * (wide(M, experts) ? 256 : 128) * sizeof(float);
}

cudaError_t launch_w4_gemm(const W4Product& p, int* status, int* counters, void* partials,
                           int num_sms, cudaStream_t s) {
    const uint8_t* const rows = reinterpret_cast<const uint8_t*>(p.rows);
    Args a;
    a.rows = rows;
    a.row_scales = reinterpret_cast<const float*>(
        rows + w4_rows_scale_offset(p.M, p.K, p.groups.experts));
    a.packed = reinterpret_cast<const uint8_t*>(p.packed);
    a.out = reinterpret_cast<__nv_bfloat16*>(p.out);
    a.start = p.groups.start;
    a.scales_a = p.scales_a;
    a.scales_b = p.scales_b;
    a.scale_a = p.scale_a;
    a.scale_b = p.scale_b;
    a.M = p.M;
    a.N = p.N;
    a.k_blocks = w4_k_blocks(p.K);
    a.row_blocks = w4_row_blocks(p.N, p.streams);
    a.experts = p.groups.experts;
    a.act = p.act;
    a.status = status;
    a.counters = counters;
    a.partials = reinterpret_cast<float*>(partials);
    a.wait_ns = test_wait_ns();
    a.stall = test_stall();
    if (wide(p.M, p.groups.experts))
        return p.streams == 2 ? launch<256, true>(a, num_sms, s) : launch<256, false>(a, num_sms, s);
    return p.streams == 2 ? launch<128, true>(a, num_sms, s) : launch<128, false>(a, num_sms, s);
}

}  // namespace nvf
