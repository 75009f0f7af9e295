// w4a4_gemm.cu -- products of NVFP4 rows with NVFP4 weights on the FP4 tensor
// cores (tcgen05, block-scaled), dense or grouped by expert:
//
//   out[m][n] = bf16(r_m * (scale2 * sum_k x[m][k] w[n][k]))
//   or, of a gate/up pair, bf16(act(g) * u) with g and u such sums in bf16.
//
// Two shapes, by the rows of an expert (of the call, without experts) on average.
//
// Up to 128, or tiles that fit in one turn: a block has 128 rows of the weight as the lanes
// of its accumulators and the tokens as columns, as many as there are, so a few tokens cost
// few columns.  Bound by the weight's bytes; two accumulators take turns.
//
// More: a pair of blocks (two SMs, one product of 256 x 256 x 64 at a time) has tokens as
// lanes, so that the epilogue stores 32 bytes of a token's features per lane; with
// features as lanes, 64 bytes per warp, its stores took 3.8 us a tile.  Each block copies
// half of either operand.  Bound by what an SM takes in: a K block of 256 takes the
// tensor cores 264 ns, and its 38 KB, out of L2, 333 (59 bytes a cycle); without the rows'
// 18 it took 290, with a sixth stage as long.  Tiles of 256 x 384, which need fewer bytes
// per product, came to 6.0 Pflop/s against 6.7: their 48 KB took 500 ns without the third
// 128 columns' products, 570 with them.  Between tiles the accumulator is idle for about
// 950 ns: the products' completion, the epilogue's reads, word of them to the first block,
// copies that compete with the stores of the tile before.  A second accumulator would need
// half of the columns.
//
// Both: two warps copy tiles into a ring of stages (a bulk copy or a box each, see
// w4a4.h), one issues products: per stage the scales go to tensor memory, into columns of
// that stage, and four products of 64 elements follow.  Sixteen warps read the sums out.
//
// Work: whole tiles in turn, then the tiles that are left over (fewer than blocks), which
// a dense product may cut along K: a range that is not all of its tile leaves its sums in
// the workspace, and a second launch adds them up in the order of the ranges.  So results
// do not depend on timing, and no block waits for one that is not of its pair.
//
// Measured (us, of it the rate): 4096 x 17408 x 5120 111 (6.6 Pflop/s), 2048 x 5120 x
// 34816 with SiLU 119 (6.1), 59 rows of 64 experts, 4096 x 4096 with SiLU 83.5 (7.2 TB/s
// of weights), 1 x 5120 x 7168 with the weight in L2 7.9 (2.6 TB/s: start, first copies and
// end take 6 of it), out of memory 8.8.
#include <cuda.h>

#include <algorithm>
#include <atomic>

#include "internal.h"
#include "kv8.cuh"
#include "tmem.cuh"
#include "w4a4.h"

namespace nvf {

namespace {

constexpr int kEpilogueWarps = 16;
// K blocks that a cut has to save for its join (8 rows of 4096 x 4096, which it would save
// 10: cut 7.9 us, whole 7.3; 1 row of 17408 x 5120, 53: 14.7, 23.5; 300 rows of 8192 x
// 4096, 16: 18.9, 14.9; 2048 rows of 17408 x 5120, 51: 66.8, 71.0).
constexpr int kJoinCost = 16;
constexpr int kJoin = 4;  // parts of a cut tile that are asked for at a time
constexpr int kThreads = (3 + kEpilogueWarps) * 32;
constexpr int kEpilogueThreads = kEpilogueWarps * 32;
// Token tiles that take turns with one weight tile before the next one: their tiles
// (16 x 256 tokens of K = 17408: 40 MB) stay in L2 for it.
constexpr int kSuper = 16;

template <int kTokens>
struct Shape {
    // Blocks that share a tile.  One alone has 128 rows of the weight as lanes and tokens as
    // columns, as many as there are.  A pair has 256 tokens by 256 rows of the weight: each
    // block copies its 128 tokens, the lanes of its accumulator, and half of the weight's
    // rows, the columns; the tensor cores of both read both halves.
    static constexpr int kBlocks = kTokens == 256 ? 2 : 1;
    static constexpr int kStages = kTokens == 256 ? 5 : 6;
    static constexpr int kSums = kTokens == 256 ? 1 : 2;  // accumulators in turn
    static constexpr int kBAt = kW4Tile;                  // the columns' codes in a stage
    static constexpr int kBScalesAt = kBAt + kTokens / kBlocks * 128;
    static constexpr int kStageBytes = kBScalesAt + kTokens * 16;
    static constexpr int kShared = 1024 + kStages * kStageBytes;
    // tensor memory: accumulators, then each stage's scales
    static constexpr int kScalesAt = kTokens * kSums;
    static constexpr int kScaleColumns = 16 + kTokens / 8;  // per stage
    static_assert(kScalesAt + kStages * kScaleColumns <= 512, "tensor memory");
    static constexpr int kPartial = kW4Rows * kTokens;  // floats
    // K blocks that a range of a cut tile has at least.
    static constexpr int kLeastRange = kBlocks > 1 ? 8 : 2;
    // Columns of a tile's products.
    static __device__ __forceinline__ int columns(int tokens) {
        return kBlocks == 1 ? (tokens + 15) / 16 * 16 : 256;
    }
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
    int M, N, k_blocks, row_blocks, experts, act;  // row_blocks: of a tile's rows
    int cut;     // K blocks of a tile that may be cut, 0 for none
    int vector;  // bytes that 16 features of a row may be stored by: 32, 16, or 2
    int* status;
    float* partials;
    unsigned long long wait_ns;
    int stall;
};

// Tiles as tensors of kilobytes, [block][K block][18][256 x 4 bytes], for the copies of
// pairs: what one block copies is reported to the other's barrier, which the plain bulk
// copies cannot.  (With a thread that passed the word on, a stage took 545 ns or more.)
// Boxes: a whole tile, a tile's codes, the scales of two tiles: each block takes
// all of the columns' scales itself, since a copy that both received would be sound only for
// a weight in this GPU's own memory, and was no faster (4096 x 17408 x 5120 113 us with either).
struct Maps {
    CUtensorMap rows, codes, scales;  // the rows' whole tiles; the weight's
};

// A range of K blocks of one tile.
struct Item {
    int expert, weight, token0, tokens;  // row block of the weight; first row, rows
    long long block;                     // first tile of the rows
    int kb0, kb1;
    int parts, first_part, left_over;    // parts > 1: sharers first_part .. + parts - 1
};

// The list of work of a block, or of a pair.  prefix[e]: token tiles of the experts in
// front of e.
template <int kTokens>
struct Schedule {
    using S = Shape<kTokens>;
    const Args& a;
    const int* prefix;
    int tiles, whole, sharers;
    int left;  // K blocks of the tiles that are left over: fewer than blocks of up to 256
    int next, range0, range1;
    int P;  // blocks, or pairs

    __device__ Schedule(const Args& args, const int* tile_prefix, int pairs, int me)
        : a(args), prefix(tile_prefix), P(pairs) {
        tiles = prefix[a.experts] * a.row_blocks;
        whole = tiles / P * P;
        left = (tiles - whole) * a.k_blocks;
        const int over = tiles - whole;
        if (S::kBlocks > 1) {
            // equal parts of each tile
            sharers = over ? over * max(1, min(P / over, a.cut / S::kLeastRange)) : 0;
        } else {
            // equal shares of them all
            sharers = a.cut ? min(P, left / S::kLeastRange) : over;
        }
        next = me;
        range0 = range1 = 0;
        if (me < sharers) {
            range0 = left * me / sharers;
            range1 = left * (me + 1) / sharers;
        }
    }

    // The sharer whose range holds K block p of the left-over tiles.
    __device__ int sharer(int p) const {
        return ((p + 1) * sharers + left - 1) / left - 1;
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

    // Where the sums of part i of a cut tile lie.  Of a sharer's ranges only the first and
    // the last can be parts of tiles, and the last begins its tile, so it is part 0 there.
    __device__ float4* part(const Item& it, int i, int rank) const {
        const int sharer = it.first_part + i;
        const bool second = i == 0 && left * sharer / sharers < it.left_over * a.k_blocks;
        const size_t block = (size_t)sharer * S::kBlocks + rank;
        return reinterpret_cast<float4*>(a.partials + (block * 2 + second) * S::kPartial);
    }

    __device__ bool take(Item& it) {
        it.parts = 1;
        if (next < whole) {
            place(next, it);
            it.kb0 = 0;
            it.kb1 = a.k_blocks;
            next += P;
            return true;
        }
        if (range0 >= range1) return false;
        const int tile = range0 / a.k_blocks, begin = tile * a.k_blocks;
        left_over(tile, it);
        it.kb0 = range0 - begin;
        it.kb1 = min(range1 - begin, a.k_blocks);
        range0 = min(range1, begin + a.k_blocks);
        return true;
    }

    // A tile that is cut, without a range of it.
    __device__ void left_over(int tile, Item& it) const {
        place(whole + tile, it);
        it.left_over = tile;
        it.first_part = sharer(tile * a.k_blocks);
        it.parts = sharer((tile + 1) * a.k_blocks - 1) - it.first_part + 1;
    }
};

// kind::mxf4nvf4: E2M1 by E2M1, E4M3 scales, fp32 sums, 128 rows per block, n columns,
// 64 deep.
template <int kBlocks>
__device__ __forceinline__ constexpr uint32_t instruction(int n) {
    return 1u << 7 | 1u << 10 | (uint32_t)(n / 8) << 17 | (uint32_t)kBlocks << 27;
}

// Shared-memory descriptors: rows of 128 bytes in the 128-byte swizzle, eight to a
// kilobyte; and 32 rows of 16 bytes, plain, eight to 128 bytes.
__device__ __forceinline__ uint64_t operand(uint32_t at) {
    return (uint64_t)((at & 0x3ffffu) >> 4) | (uint64_t)(1024 >> 4) << 32 | 1ull << 46 | 2ull << 61;
}
__device__ __forceinline__ uint64_t scale_operand(uint32_t at) {
    return (uint64_t)((at & 0x3ffffu) >> 4) | (uint64_t)(128 >> 4) << 32 | 1ull << 46;
}

// The instructions of one block's tensor cores, and of a pair's: those are issued by the
// first block's thread, for the same addresses in both.
template <int kBlocks>
__device__ __forceinline__ void tmem_alloc(uint32_t to) {
    if constexpr (kBlocks == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(to)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    } else {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(to)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
}

template <int kBlocks>
__device__ __forceinline__ void tmem_free(uint32_t at) {
    if constexpr (kBlocks == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(at) : "memory");
    else
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(at) : "memory");
}

template <int kBlocks>
__device__ __forceinline__ void copy_scales(uint32_t columns, uint64_t from) {
    if constexpr (kBlocks == 1)
        asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(columns), "l"(from)
                     : "memory");
    else
        asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(columns), "l"(from)
                     : "memory");
}

template <int kBlocks>
__device__ __forceinline__ void multiply(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                         uint32_t scales_a, uint32_t scales_b, bool add) {
    if constexpr (kBlocks == 1)
        asm volatile(
            "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
            " tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, "
            "[%4], [%5], p;\n}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(scales_a), "r"(scales_b), "r"(add ? 1 : 0)
            : "memory");
    else
        asm volatile(
            "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
            " tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, "
            "[%4], [%5], p;\n}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(scales_a), "r"(scales_b), "r"(add ? 1 : 0)
            : "memory");
}

// `bar`, in each block, completes when all products issued so far have.
template <int kBlocks>
__device__ __forceinline__ void commit(uint32_t bar) {
    if constexpr (kBlocks == 1)
        asm volatile(
            "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
            : "memory");
    else
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster"
            ".b64 [%0], %1;" ::"r"(bar),
            "h"((uint16_t)3)
            : "memory");
}

// The address of the pair's first block's copy of a shared variable.
__device__ __forceinline__ uint32_t in_first(uint32_t at) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(at));
    return r;
}

// One box (see Maps) from kilobyte y of tile (kb, block) on, into this block's memory; `bar`
// is the first block's, to which the copies into either are reported.
__device__ __forceinline__ void copy_box(uint32_t to, const CUtensorMap* map, int y, int kb,
                                         int block, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        ".cta_group::2 [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(to),
        "l"(map), "r"(0), "r"(y), "r"(kb), "r"(block), "r"(bar)
        : "memory");
}

// Asks for `bytes` (a multiple of 16) at `from` in L2.
__device__ __forceinline__ void prefetch_l2(const uint8_t* from, uint32_t bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(from), "r"(bytes) : "memory");
}

// True for one thread of the warp, which calls it together.
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile(
        "{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}"
        : "=r"(one));
    return one != 0;
}

// Arrives at the barrier at this address in the pair's first block.  (What has to be
// done before it is: reads of tensor memory that were waited for.  A release at cluster
// scope would wait for the warp's stores too, which took 540 ns.)
__device__ __forceinline__ void arrive_at_first(uint32_t bar) {
    asm volatile(
        "{\n .reg .b32 r;\n mapa.shared::cluster.u32 r, %0, 0;\n"
        " mbarrier.arrive.shared::cluster.b64 _, [r];\n}" ::"r"(bar)
        : "memory");
}

// Waits, boundedly, for a phase that a thread of the other block may complete.
__device__ __forceinline__ bool try_wait_cluster(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n"
        " mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n"
        " selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(kSuspendHintNs)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool wait_cluster(uint32_t bar, uint32_t parity,
                                             const volatile int* abort,
                                             unsigned long long limit_ns) {
    if (try_wait_cluster(bar, parity)) return true;
    const unsigned long long t0 = global_timer_ns();
    while (!try_wait_cluster(bar, parity)) {
        if (*abort) return false;
        if (global_timer_ns() - t0 > limit_ns) return false;
    }
    return true;
}

// All threads of a pair (of a block).
template <int kBlocks>
__device__ __forceinline__ void sync_blocks() {
    if constexpr (kBlocks == 1)
        __syncthreads();
    else
        asm volatile("barrier.cluster.arrive.aligned;\n barrier.cluster.wait.aligned;" ::: "memory");
}

// act(g) * u for g and u in bf16: act(g) = g * sigmoid(y), y = g or the argument of GeLU's
// tanh, doubled.  g * u is exact in fp32, and for y > 0 what sigmoid takes away from
// it is subtracted, with one rounding.  Where that is too little for fp32, g * u itself
// may be a tie of bf16 (it has 16 bits): then the result, below it, goes towards 0, unless
// sigmoid(y) is 1 in 64 bits too (a loss below 2^-54), where the tie goes to even.
__device__ __forceinline__ float gated(int act, float g, float u) {
    const float y = act == 0 ? g : 1.5957691216057308f * (g + 0.044715f * g * g * g);
    const float e = __expf(-fabsf(y)), s = __fdividef(e, 1.0f + e);  // sigmoid(-|y|)
    if (!(y > 0.0f)) {
        // far below 0 the sigmoid is e^y, which leaves fp32's normal numbers from -87 on, where a
        // product with a large u does not: in two halves
        const float half = __expf(0.5f * y);
        return y < -64.0f ? g * half * u * half : g * s * u;
    }
    const float t = g * u;
    const float p = fabsf(t) < INFINITY ? fmaf(-t, s, t) : t;
    const uint32_t bits = __float_as_uint(p);
    const bool below = p == t && s > 5.5511151e-17f && (bits & 0xffffu) == 0x8000u;
    return below ? __uint_as_float(bits - 1) : p;
}

// Sums of kColumns columns of a cut tile in one lane, parts in order, kJoin of them asked
// for at a time: a part is [column / 4][lane][4] floats.
template <int kTokens, int kColumns>
__device__ __forceinline__ void join(const Schedule<kTokens>& schedule, const Item& it, int rank,
                                     int column, int lane, float (&x)[kColumns]) {
    using S = Shape<kTokens>;
    const int here = column / 4 * kW4Rows + lane;
    const float4* const part0 = schedule.part(it, 0, rank) + here;
    const float4* const part1 = schedule.part(it, 1, rank) + here;  // the others follow it
    constexpr size_t kNext = (size_t)S::kBlocks * 2 * S::kPartial / 4;
#pragma unroll
    for (int j = 0; j < kColumns; ++j) x[j] = 0.0f;
#pragma unroll 1
    for (int i = 0; i < it.parts; i += kJoin) {
        float4 y[kJoin][kColumns / 4];
#pragma unroll
        for (int k = 0; k < kJoin; ++k)
#pragma unroll
            for (int j = 0; j < kColumns / 4; ++j) {
                y[k][j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (i + k < it.parts)
                    y[k][j] = __ldcg((i + k == 0 ? part0 : part1 + (i + k - 1) * kNext) +
                                     j * kW4Rows);
            }
#pragma unroll
        for (int k = 0; k < kJoin; ++k)
#pragma unroll
            for (int j = 0; j < kColumns / 4; ++j) {
                x[4 * j] += y[k][j].x;
                x[4 * j + 1] += y[k][j].y;
                x[4 * j + 2] += y[k][j].z;
                x[4 * j + 3] += y[k][j].w;
            }
    }
}

// The lanes of one block alone: a row of the weight each, tokens as columns.
template <bool kGated>
struct FeatureLane {
    bool odd, up;
    float scale;
    int feature, N, tokens, act;
    __nv_bfloat16* out;

    __device__ __forceinline__ FeatureLane(const Args& a, const Item& it, int quadrant) {
        const int lane = threadIdx.x & 31;
        odd = lane & 1;
        up = kGated && lane >= 16;
        scale = up ? (a.scales_b ? a.scales_b[it.expert] : a.scale_b)
                   : (a.scales_a ? a.scales_a[it.expert] : a.scale_a);
        // of a pair of lanes that trade: the even one's
        feature = kGated ? it.weight * 64 + quadrant * 16 + (lane & 14)
                         : it.weight * kW4Rows + quadrant * 32 + (lane & 30);
        N = a.N;
        tokens = it.tokens;
        act = a.act;
        out = a.out + (size_t)it.token0 * a.N + feature;
    }

    // Scales and stores eight tokens, column on (r: their rows' scales).  Neighbouring lanes
    // trade, for two features of one token each.  Of a gate/up pair 16 lanes have gate, 16 up,
    // of the same features: the first take the even tokens, the others the odd ones.
    __device__ __forceinline__ void emit(int column, const float (&x)[8],
                                         const float* r) const {
        uint32_t v[4];  // pairs of tokens, in bf16
#pragma unroll
        for (int j = 0; j < 4; ++j)
            v[j] = bf16x2(x[2 * j] * scale * r[2 * j], x[2 * j + 1] * scale * r[2 * j + 1]);
        if (kGated) {
#pragma unroll
            for (int j = 0; j < 4; j += 2) {
                float h[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint32_t o = __shfl_xor_sync(0xffffffffu, v[j + k], 16);
                    h[k] = gated(act, up ? bf16_hi(o) : bf16_lo(v[j + k]),
                                 up ? bf16_hi(v[j + k]) : bf16_lo(o));
                }
                const uint32_t own = bf16x2(h[0], h[1]);
                const uint32_t o = __shfl_xor_sync(0xffffffffu, own, 1);
                const uint32_t w = odd ? prmt(o, own, 0x7632) : prmt(own, o, 0x5410);
                const int token = column + 2 * j + (up ? 1 : 0) + (odd ? 2 : 0);
                if (token < tokens && feature < N)
                    *reinterpret_cast<uint32_t*>(out + (size_t)token * N) = w;
            }
        } else if (N & 1) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (column + j < tokens && feature + odd < N)
                    *reinterpret_cast<uint16_t*>(out + (size_t)(column + j) * N + odd) =
                        (uint16_t)(j & 1 ? v[j / 2] >> 16 : v[j / 2]);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t o = __shfl_xor_sync(0xffffffffu, v[j], 1);
                const uint32_t w = odd ? prmt(o, v[j], 0x7632) : prmt(v[j], o, 0x5410);
                const int token = column + 2 * j + odd;
                if (token < tokens && feature < N)
                    *reinterpret_cast<uint32_t*>(out + (size_t)token * N) = w;
            }
        }
    }
};

// A pair's lane: one token, whose features lie side by side.
template <bool kGated>
struct TokenRow {
    bool live;
    float r, scale_a, scale_b;
    __nv_bfloat16* out;  // from the lane's first column on
    int room;            // features of the output from there on
    int act, vector;

    __device__ __forceinline__ TokenRow(const Args& a, const Item& it, int token, int first) {
        live = token < it.tokens;
        r = live ? a.row_scales[it.token0 + token] : 0.0f;
        scale_a = a.scales_a ? a.scales_a[it.expert] : a.scale_a;
        scale_b = a.scales_b ? a.scales_b[it.expert] : a.scale_b;
        const int feature = (it.weight * 256 + first) / (kGated ? 2 : 1);
        out = a.out + (size_t)(it.token0 + token) * a.N + feature;
        room = a.N - feature;
        act = a.act;
        vector = a.vector;
    }

    __device__ __forceinline__ void store16(int feature, const uint32_t (&w)[8]) const {
        if (!live || feature >= room) return;
        __nv_bfloat16* const to = out + feature;
        if (vector == 32 && feature + 16 <= room) {
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to),
                         "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]),
                         "r"(w[6]), "r"(w[7])
                         : "memory");
        } else if (vector == 16 && feature + 16 <= room) {
            reinterpret_cast<uint4*>(to)[0] = make_uint4(w[0], w[1], w[2], w[3]);
            reinterpret_cast<uint4*>(to)[1] = make_uint4(w[4], w[5], w[6], w[7]);
        } else {
#pragma unroll
            for (int j = 0; j < 16; ++j)
                if (feature + j < room)
                    reinterpret_cast<uint16_t*>(to)[j] =
                        (uint16_t)(j & 1 ? w[j / 2] >> 16 : w[j / 2]);
        }
    }

    // 32 columns, the c-th ones: as many features, or 16 of gate and 16 of up.
    __device__ __forceinline__ void emit(int c, const float (&x)[32]) const {
        uint32_t w[8];
        if (kGated) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t g = bf16x2(x[2 * j] * scale_a * r, x[2 * j + 1] * scale_a * r);
                const uint32_t u =
                    bf16x2(x[16 + 2 * j] * scale_b * r, x[17 + 2 * j] * scale_b * r);
                w[j] = bf16x2(gated(act, bf16_lo(g), bf16_lo(u)), gated(act, bf16_hi(g), bf16_hi(u)));
            }
            store16(16 * c, w);
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    w[j] = bf16x2(x[16 * h + 2 * j] * scale_a * r,
                                  x[16 * h + 2 * j + 1] * scale_a * r);
                store16(32 * c + 16 * h, w);
            }
        }
    }
};

struct Barriers {
    uint64_t full[8], empty[8];        // stages
    uint64_t sums_full[2], sums_empty[2];
    uint64_t drained;                  // after a wait that ran out
};

template <int kTokens, bool kGated>
__global__ void __launch_bounds__(kThreads, 1)
    w4a4_gemm_kernel(const Args a, const __grid_constant__ Maps maps) {
    using S = Shape<kTokens>;
    extern __shared__ __align__(1024) uint8_t dynamic[];
    // the swizzle goes by address: stages begin on multiples of 1024
    uint8_t* const shared = dynamic + (-smem_addr(dynamic) & 1023u);
    __shared__ Barriers bars;
    __shared__ int prefix[kW4MaxExperts + 1];
    __shared__ alignas(16) float row_scale[2][kTokens];  // one block's: of two tiles in turn
    __shared__ volatile int abort;
    __shared__ uint32_t tmem_at;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t smem = smem_addr(shared);
    constexpr int kWeightWarp = 0, kIssueWarp = 1, kRowsWarp = 2 + kEpilogueWarps;
    const int rank = blockIdx.x % S::kBlocks;  // in the pair

    if (warp == kIssueWarp) tmem_alloc<S::kBlocks>(smem_addr(&tmem_at));
    if (tid == 0) {
        for (int i = 0; i < S::kStages; ++i) {
            mbar_init(smem_addr(&bars.full[i]), 1);
            mbar_init(smem_addr(&bars.empty[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_addr(&bars.sums_full[i]), 1);
            mbar_init(smem_addr(&bars.sums_empty[i]), kEpilogueWarps * S::kBlocks);
        }
        mbar_init(smem_addr(&bars.drained), 1);
        abort = 0;
        fence_mbar_init();
    }
    if (a.start) asm volatile("griddepcontrol.wait;" ::: "memory");
    // token tiles of each expert; one whose rows are not all inside has none, and none has
    // any where the list decreases (shares that overlap could be more than tiles are counted)
    if (tid == 0) prefix[0] = 0;
    bool decreases = false;
    for (int e = tid; e < a.experts; e += kThreads) {
        const int first = a.start ? a.start[e] : 0, end = a.start ? a.start[e + 1] : a.M;
        decreases |= end < first;
        prefix[e + 1] = first >= 0 && end <= a.M && end > first
                            ? (end - first + kTokens - 1) / kTokens
                            : 0;
    }
    if (__syncthreads_or(decreases)) {
        for (int e = tid; e < a.experts; e += kThreads) prefix[e + 1] = 0;
    } else if (warp == 2 && a.experts > 1) {
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
    sync_blocks<S::kBlocks>();
    if (S::kBlocks > 1) __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = tmem_at;

    // Waits for a barrier's completion number `uses` (from 0); false, with the status
    // set, when it does not come in time.
    auto wait_lane = [&](uint64_t& bar, unsigned uses) {
        if (S::kBlocks > 1 ? wait_cluster(smem_addr(&bar), uses & 1, &abort, a.wait_ns)
                           : mbar_wait_bounded(smem_addr(&bar), uses & 1, &abort, a.wait_ns))
            return true;
        abort = 1;
        *a.status = kKv8Timeout;
        return false;
    };

    auto wait = [&](uint64_t& bar, unsigned uses) {  // the same answer for a whole warp
        return __all_sync(0xffffffffu, wait_lane(bar, uses)) != 0;
    };

    Schedule<kTokens> schedule(a, prefix, gridDim.x / S::kBlocks, blockIdx.x / S::kBlocks);
    Item it{};
    auto row_block = [&] { return (it.expert * a.row_blocks + it.weight) * S::kBlocks + rank; };
    if (!a.start) {
        // Without lists to read, the work is known before the preceding kernel is done: the
        // weight's first tiles come into L2 meanwhile.  They are not read before it is done,
        // as it may be what writes them.
        if (warp == kWeightWarp) {
            Schedule<kTokens> first = schedule;
            if (first.take(it) && elect_one())
                prefetch_l2(a.packed + ((size_t)row_block() * a.k_blocks + it.kb0) * kW4Tile,
                            min(it.kb1 - it.kb0, S::kStages) * kW4Tile);
            __syncwarp();
        }
        asm volatile("griddepcontrol.wait;" ::: "memory");
    }
    // Not before: the next kernel may begin on what it takes to be finished, the kernels in
    // front of this one.
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (warp == kWeightWarp || warp == kRowsWarp) {
        // Two warps, since a copy takes its thread about 200 cycles.
        const bool issuer = elect_one(), rows = warp == kRowsWarp;
        unsigned n = 0;  // stages filled
        bool ok = true;
        while (ok && schedule.take(it)) {
            const int weight = row_block();
            const uint8_t* const from = rows ? a.rows + (size_t)it.block * a.k_blocks * kW4Tile
                                             : a.packed + (size_t)weight * a.k_blocks * kW4Tile;
            const int codes = S::columns(it.tokens) * 128;  // of the rows, to one block alone
            for (int kb = it.kb0; kb < it.kb1; ++kb, ++n) {
                const int stage = n % S::kStages;
                if (n >= S::kStages) {
                    ok = wait(bars.empty[stage], n / S::kStages - 1);
                    if (!ok) break;
                }
                if (a.stall && n >= 1) {  // testing: nothing comes any more
                    wait(bars.drained, 0);
                    ok = false;
                    break;
                }
                if (issuer) {
                    const uint32_t at = smem + stage * S::kStageBytes;
                    uint32_t bar = smem_addr(&bars.full[stage]);
                    // the weight's warp announces the bytes of all of the stage's copies
                    if constexpr (S::kBlocks == 1) {
                        const uint8_t* const t = from + (size_t)kb * kW4Tile;
                        if (rows) {
                            bulk_copy_g2s(at + S::kBAt, t, codes, bar);
                            bulk_copy_g2s(at + S::kBScalesAt, t + kW4Codes, kW4Scales, bar);
                        } else {
                            mbar_arrive_expect_tx(bar, kW4Tile + codes + kW4Scales);
                            bulk_copy_g2s(at, t, kW4Tile, bar);
                        }
                    } else if (rows) {
                        copy_box(at, &maps.rows, 0, kb, (int)it.block + rank, in_first(bar));
                    } else {
                        if (rank == 0) mbar_arrive_expect_tx(bar, 2 * S::kStageBytes);
                        bar = in_first(bar);
                        copy_box(at + S::kBAt, &maps.codes, 0, kb, weight, bar);
                        copy_box(at + S::kBScalesAt, &maps.scales, kW4Codes / 1024, kb,
                                 weight - rank, bar);
                    }
                }
                __syncwarp();
            }
        }
        // the last products' word has come before the barriers that it goes to are left
        for (unsigned i = n > S::kStages ? n - S::kStages : 0; i < n && ok; ++i)
            ok = wait(bars.empty[i % S::kStages], i / S::kStages);
        if (abort) {
            // copies under way end before the memory that they write is left; these waits
            // heed nobody's, and end for stages that lack the other warp's
            const int none = 0;
            if (rank == 0)
                for (unsigned i = n > S::kStages ? n - S::kStages : 0; i < n; ++i)
                    mbar_wait_bounded(smem_addr(&bars.full[i % S::kStages]), i / S::kStages & 1,
                                      &none, a.wait_ns);
            else  // reported to the other block: time enough for any copy
                for (const unsigned long long t0 = global_timer_ns();
                     global_timer_ns() - t0 < 100000;)
                    __nanosleep(1000);
        }
    } else if (warp == kIssueWarp && rank == 0) {
        // The whole warp runs the loop and one thread issues: in a branch of one thread from
        // the start, each of these instructions took about 60 cycles (their operands have to
        // be the same for the warp), 1030 for a stage's.
        const bool issuer = elect_one();
        unsigned n = 0, items = 0;
        bool ok = true;
        while (ok && schedule.take(it)) {
            const unsigned sums = items % S::kSums;
            if (items >= S::kSums) {
                ok = wait(bars.sums_empty[sums], items / S::kSums - 1);
                if (!ok) break;
            }
            tmem_fence_after();
            const uint32_t d = tmem + sums * kTokens;
            const int columns = S::columns(it.tokens);
            const uint32_t idesc = instruction<S::kBlocks>(columns);
            for (int kb = it.kb0; kb < it.kb1; ++kb, ++n) {
                const int stage = n % S::kStages;
                ok = wait(bars.full[stage], n / S::kStages);
                if (!ok) break;
                const uint32_t at = smem + stage * S::kStageBytes;
                // the stage's own columns: what read them last has completed, as the
                // stage was filled again
                const uint32_t scales_a = tmem + S::kScalesAt + stage * S::kScaleColumns;
                const uint32_t scales_b = scales_a + 16;
                const uint64_t from_a = scale_operand(at + kW4Codes);
                const uint64_t from_b = scale_operand(at + S::kBScalesAt);
                const uint64_t op_a = operand(at), op_b = operand(at + S::kBAt);
                if (issuer) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        copy_scales<S::kBlocks>(scales_a + 4 * j, from_a + j * (512 >> 4));
                        copy_scales<S::kBlocks>(scales_b + j * (kTokens / 32),
                                                from_b + j * (512 >> 4));
                        if (kTokens == 256)
                            copy_scales<S::kBlocks>(scales_b + j * (kTokens / 32) + 4,
                                                    from_b + (kW4Scales >> 4) + j * (512 >> 4));
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        multiply<S::kBlocks>(d, op_a + j * 2, op_b + j * 2, idesc,
                                             scales_a + 4 * j, scales_b + j * (kTokens / 32),
                                             kb > it.kb0 || j > 0);
                    commit<S::kBlocks>(smem_addr(&bars.empty[stage]));
                }
                __syncwarp();
            }
            if (!ok) break;
            if (issuer) commit<S::kBlocks>(smem_addr(&bars.sums_full[sums]));
            __syncwarp();
            ++items;
        }
        if (abort) {
            // products under way end before the memory that they read is left
            const int none = 0;
            if (issuer) commit<S::kBlocks>(smem_addr(&bars.drained));
            mbar_wait_bounded(smem_addr(&bars.drained), 0, &none);
        }
    } else if (warp > kIssueWarp) {  // the epilogue
        // a warp reads 32 lanes of a share of the columns
        constexpr int kShare = kTokens * 4 / kEpilogueWarps;
        const int quadrant = warp & 3, eid = tid - 64;
        // a pair's warp has as many columns in a run; of one block's, eight of every 32
        const int first = (warp - 2) / 4 * (S::kBlocks > 1 ? kShare : 8);
        const uint32_t lanes = tmem + ((uint32_t)(quadrant * 32) << 16);
        bool ok = true;
        auto give_back = [&](unsigned sums) {
            tmem_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (rank == 0) mbar_arrive(smem_addr(&bars.sums_empty[sums]));
                else arrive_at_first(smem_addr(&bars.sums_empty[sums]));
            }
        };
        if constexpr (S::kBlocks > 1) {
            const int token = rank * kW4Rows + quadrant * 32 + lane;
            for (unsigned items = 0; schedule.take(it); ++items) {
                const TokenRow<kGated> row(a, it, token, first);
                ok = ok && wait(bars.sums_full[0], items);
                tmem_fence_after();
                // the accumulator is given back before its columns are looked at
                float x[kShare / 32][32];
                if (ok) {
#pragma unroll
                    for (int c = 0; c < kShare / 32; ++c)
                        tmem_load32(lanes + first + 32 * c, x[c]);
#pragma unroll
                    for (int c = 0; c < kShare / 32; ++c) tmem_wait_load(x[c]);
                }
                give_back(0);
                if (!ok) continue;
                if (it.parts == 1) {
#pragma unroll
                    for (int c = 0; c < kShare / 32; ++c) row.emit(c, x[c]);
                } else {
                    float4* const to =
                        schedule.part(it, (int)blockIdx.x / S::kBlocks - it.first_part, rank) +
                        first / 4 * kW4Rows + quadrant * 32 + lane;
#pragma unroll
                    for (int j = 0; j < kShare / 4; ++j)
                        to[j * kW4Rows] =
                            make_float4(x[j / 8][j % 8 * 4], x[j / 8][j % 8 * 4 + 1],
                                        x[j / 8][j % 8 * 4 + 2], x[j / 8][j % 8 * 4 + 3]);
                }
            }
        } else {
            for (unsigned items = 0; schedule.take(it); ++items) {
                const unsigned sums = items % S::kSums;
                float* const scales = row_scale[items & 1];
                if (eid < kTokens)
                    scales[eid] = eid < it.tokens ? a.row_scales[it.token0 + eid] : 0.0f;
                const FeatureLane<kGated> feature(a, it, quadrant);
                named_barrier_sync(1, kEpilogueThreads);  // row scales are there
                ok = ok && wait(bars.sums_full[sums], items / S::kSums);
                tmem_fence_after();
                const uint32_t from = lanes + sums * kTokens;
                float4* const to =
                    it.parts == 1 ? nullptr
                                  : schedule.part(it, (int)blockIdx.x - it.first_part, 0) +
                                        quadrant * 32 + lane;
                // the other accumulator is at work meanwhile
#pragma unroll 1
                for (int column = first; column < it.tokens && ok; column += 32) {
                    float x[8];
                    tmem_load8(from + column, x);
                    if (it.parts == 1) {
                        feature.emit(column, x, scales + column);
                    } else {
                        to[column / 4 * kW4Rows] = make_float4(x[0], x[1], x[2], x[3]);
                        to[(column / 4 + 1) * kW4Rows] = make_float4(x[4], x[5], x[6], x[7]);
                    }
                }
                give_back(sums);
            }
        }
    }
    // a pair's first block reads the other's memory and both signal each other's barriers:
    // neither leaves before the other is done
    tmem_fence_before();
    __syncwarp();
    sync_blocks<S::kBlocks>();
    if (warp == kIssueWarp) tmem_free<S::kBlocks>(tmem);
}

// Joins the cut tiles of a dense product: a block has 128 lanes of a tile, and 8 columns
// of one block's or 32 of a pair's.  (Joined by the block that came last, in the
// product's kernel, four parts of a pair's tile, 512 KB through one SM, took 14 us; those
// of one block's tile of 1 token 7 us, of 128 tokens 15 us.)
template <int kTokens, bool kGated>
__global__ void __launch_bounds__(kW4Rows) w4a4_join_kernel(const Args a, int pairs) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int prefix[2] = {0, (a.M + kTokens - 1) / kTokens};
    const Schedule<kTokens> schedule(a, prefix, pairs, 0);
    Item it{};
    schedule.left_over(blockIdx.x, it);
    const int lane = threadIdx.x;
    if constexpr (kTokens == 256) {
        const int rank = blockIdx.y / 8, first = blockIdx.y % 8 * 32;
        const TokenRow<kGated> row(a, it, rank * kW4Rows + lane, first);
        float x[32];
        join<kTokens, 32>(schedule, it, rank, first, lane, x);
        row.emit(0, x);
    } else {
        const int column = blockIdx.y * 8;
        if (column >= it.tokens) return;
        const FeatureLane<kGated> feature(a, it, lane / 32);
        float x[8], r[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            r[j] = column + j < it.tokens ? a.row_scales[it.token0 + column + j] : 0.0f;
        join<kTokens, 8>(schedule, it, 0, column, lane, x);
        feature.emit(column, x, r);
    }
}

using EncodeTiled = decltype(&cuTensorMapEncodeTiled);

// The driver's function, through the runtime (the library does not link the driver).
EncodeTiled encode_tiled() {
    static std::atomic<void*> known{nullptr};
    void* f = known.load(std::memory_order_acquire);
    if (!f) {
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                             &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            return nullptr;
        known.store(f, std::memory_order_release);
    }
    return reinterpret_cast<EncodeTiled>(f);
}

// A map of `blocks` row blocks of tiles for boxes of `rows` kilobytes of `tiles` neighbours.
bool tile_map(CUtensorMap* map, const void* at, int k_blocks, long long blocks, int rows,
              int tiles) {
    const EncodeTiled encode = encode_tiled();
    if (!encode) return false;
    const cuuint64_t size[4] = {256, kW4Tile / 1024, (cuuint64_t)k_blocks, (cuuint64_t)blocks};
    const cuuint64_t stride[3] = {1024, kW4Tile, (cuuint64_t)k_blocks * kW4Tile};
    const cuuint32_t box[4] = {256, (cuuint32_t)rows, 1, (cuuint32_t)tiles}, step[4] = {1, 1, 1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_INT32, 4, const_cast<void*>(at), size, stride, box,
                  step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Tiles of a dense product behind the last whole turn.
template <int kTokens>
int left_over(const Args& a, int pairs) {
    return (int)((long long)((a.M + kTokens - 1) / kTokens) * a.row_blocks % pairs);
}

// Whether they are cut along K: where that saves more K blocks of time (0.3 us each) than
// the join costs.
template <int kTokens>
bool cuts(const Args& a, int num_sms) {
    const int pairs = num_sms / Shape<kTokens>::kBlocks, over = left_over<kTokens>(a, pairs);
    if (a.start || over == 0) return false;
    // one range of a cut tile
    const int range = kTokens == 256
                          ? a.k_blocks / std::max(1, std::min(pairs / over,
                                                              a.k_blocks / Shape<256>::kLeastRange))
                          : std::max(over * a.k_blocks / pairs, Shape<128>::kLeastRange);
    return a.k_blocks - range > kJoinCost;
}

template <int kTokens, bool kGated>
cudaError_t launch(const Args& a, const Maps& maps, int num_sms, cudaStream_t s) {
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
    cfg.gridDim = dim3(num_sms / Shape<kTokens>::kBlocks * Shape<kTokens>::kBlocks);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Shape<kTokens>::kShared;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = Shape<kTokens>::kBlocks;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = Shape<kTokens>::kBlocks > 1 ? 2 : 1;
    e = cudaLaunchKernelEx(&cfg, w4a4_gemm_kernel<kTokens, kGated>, a, maps);
    if (!a.cut || e != cudaSuccess) return e;
    const int pairs = num_sms / Shape<kTokens>::kBlocks;
    cfg.gridDim = dim3(left_over<kTokens>(a, pairs), kTokens == 256 ? 16 : (std::min(a.M, kTokens) + 7) / 8);
    cfg.blockDim = dim3(kW4Rows);
    cfg.dynamicSmemBytes = 0;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, w4a4_join_kernel<kTokens, kGated>, a, pairs);
}

// Whether a product may take pairs' tiles: by the rows of an expert on average, as far as
// the host knows them (16 experts, 4096 x 4096: 96 rows each 33.0 us with single blocks, 37.0
// with pairs, 128 rows 35.2, 37.9, 160 rows 43.2, 38.5).
bool wide(int M, int experts) { return M > 128LL * experts; }

// And whether it does: not a dense one whose 128 x 128 tiles fit in one turn, which then use
// twice as many SMs (K = 5120: 256 x 5120 9.8 us with single blocks, 11.3 with pairs, 384 x
// 5120 10.0, 12.3; more than a turn 512 x 5120 16.3, 12.3, 160 x 17408 16.3, 15.9).
bool pairs(const W4Product& p, int weight_blocks, int num_sms) {
    const long long tiles = (p.M + kW4Rows - 1LL) / kW4Rows * weight_blocks;
    return wide(p.M, p.groups.experts) && (p.groups.start || tiles > num_sms);
}

}  // namespace

size_t w4_partial_bytes(int M, int experts, int num_sms) {
    if (experts > 1) return 0;  // their tiles are not cut
    return (size_t)num_sms * 2 * kW4Rows * (wide(M, experts) ? 256 : 128) * sizeof(float);
}

cudaError_t launch_w4_gemm(const W4Product& p, int* status, void* partials, int num_sms,
                           cudaStream_t s) {
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
    const uintptr_t at = reinterpret_cast<uintptr_t>(p.out) | (uintptr_t)p.N * 2;
    a.vector = at % 32 == 0 ? 32 : at % 16 == 0 ? 16 : 2;
    a.status = status;
    a.partials = reinterpret_cast<float*>(partials);
    a.wait_ns = test_wait_ns();
    a.stall = test_stall();
    Maps maps{};
    if (pairs(p, a.row_blocks, num_sms)) {
        const long long blocks = w4_token_blocks(p.M, p.groups.experts);
        const long long weights = (long long)a.experts * a.row_blocks;
        if (!tile_map(&maps.rows, p.rows, a.k_blocks, blocks, kW4Tile / 1024, 1) ||
            !tile_map(&maps.codes, p.packed, a.k_blocks, weights, kW4Codes / 1024, 1) ||
            !tile_map(&maps.scales, p.packed, a.k_blocks, weights, kW4Scales / 1024, 2))
            return cudaErrorInvalidValue;
        a.row_blocks /= Shape<256>::kBlocks;
        a.cut = cuts<256>(a, num_sms) ? a.k_blocks : 0;
        return p.streams == 2 ? launch<256, true>(a, maps, num_sms, s)
                              : launch<256, false>(a, maps, num_sms, s);
    }
    a.cut = cuts<128>(a, num_sms) ? a.k_blocks : 0;
    return p.streams == 2 ? launch<128, true>(a, maps, num_sms, s)
                          : launch<128, false>(a, maps, num_sms, s);
}

}  // namespace nvf
