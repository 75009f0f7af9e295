// kv8_prompt.cu -- attention of many rows per kv head (a prompt's tokens, or
// a chunk of one) over the paged E4M3 cache: the same operator as
// kv8_attention.cu, on tcgen05.
//
// What bounds it: the products, 4 * head_dim flops per row and key, and beside
// them 2^t for each score.  A block takes 256 rows of one kv head as two 128-row
// tiles and goes through its keys 128 at a time:
//   S = q K^T      128 x 128, both operands in shared memory, f16 -> fp32 in TMEM
//   P = 2^(t - m)  t = log2(e) s + log2(v_scale), two threads per row, f16 in TMEM
//   O += P V       128 x head_dim, P from TMEM, V from shared memory
// While the softmax of one row tile runs, the tensor cores work on the other's
// products: one thread issues both, in turn.  16 warps do the softmax, a row's two
// threads taking 64 keys of a tile each and exchanging the largest t (with one
// thread per row, 8 warps, each warp's own latencies showed: 91 us against 87 for
// 64 tokens of 64 heads on 8 kv heads of 128, over 32805 keys).  One warp copies
// pages into shared memory (the bulk-copy engine, 16 keys at a time), 4 turn their
// E4M3 bytes into f16 tiles (exactly) in the 128-byte swizzle that the tensor cores
// read.  K and V tiles take turns in three buffers.  TMEM holds S (then P in its
// place) and O of both row tiles, all 512 columns.  K, V and q tiles are rows of
// 128 bytes (64 values), 16-byte pieces XORed with the row; V is the transposed
// operand of the second product, so both tiles are written alike.  A softmax thread
// has 80 registers, and a spilled value costs it more than its reload: shared
// memory leaves the first-level cache little room.
//
// Softmax with a scale per page, as in kv8_attention.cu: O = sum P v_code,
// l = sum P / v_scale.  m is the largest t when the row's O was last rescaled;
// O is rescaled only when a tile's largest t exceeds it by kSlack, so P stays
// below 2^(kPromptBias + kSlack) and most tiles read S twice and O never.  t,
// m, l and O are fp32, P is f16.
//
// Blocks that share a unit leave partial states, which a second kernel joins
// in the order of their ranges (its blocks read 16 bytes of many rows at once; joined
// by the last block of a unit instead, one SM would read all of its parts).  Every
// wait is bounded; when one runs out the block's others end too, then the copies and
// products under way (again with a limit), and the status word says so.
//
// Measured, 64 tokens of 64 heads over 32805 keys: 84 us, 822 Tflop/s.  A key tile
// took 4580 cycles (in calls of 86.4 us), of which the products need 2160 (512 each
// for S, 560 for PV) and 2^t 1350.  The rest is a row tile's own chain, about 1900
// cycles of softmax, 420 until the products see P, 895 for PV with its completion and
// 955 for S with its.  With heads of 128 values TMEM holds no third row tile or second
// S to fill those waits with; with 64, columns 384..511 are idle.  Up to 128 rows there
// is one row tile, with nothing beside its chain.
#include <atomic>

#include "internal.h"
#include "kv8_schedule.cuh"

namespace nvf {

namespace {

constexpr int kPromptKeys = 128;
constexpr int kPromptRows = 256;
constexpr int kHalfKeys = 64;  // keys of a tile that one of a row's two threads takes
constexpr int kSoftmaxWarps = 16;
constexpr int kBuffers = 3;    // of K and V tiles in turn
constexpr int kConvertWarps = 4;
constexpr int kPromptThreads = (kSoftmaxWarps + kConvertWarps + 2) * 32;
constexpr int kGroups = kPromptKeys / 16;  // page scales per tile
// Rows per sequence and kv head, on average, up to which one pass of
// kv8_attention.cu holds them and is the faster (8 sequences of 8192 keys, 8 kv
// heads of 128: 32 rows 70 us against 75 here, 40 rows 124 against 75, 128 rows 233
// against 70; one sequence of 1000 keys, where this kernel's longer start shows:
// 32 rows 14.6 against 16.6, 64 rows 15.1 against 16.9, 128 rows 15.8 against 17.6).
constexpr int kPromptRowsAbove = 32;
constexpr float kPromptBias = 6.0f;
constexpr float kSlack = 8.0f;

// At least 2 tiles per block; a unit, or a piece of one, costs about 4 tiles beside
// its own (2 prompts of 1500 tokens, 32 heads on 8: 96 us, 109 with 2, 97 with 7;
// 8 ragged ones of up to 1024 tokens over up to 2000 keys, 40 heads: 208, 256, 203).
using PromptTiling = TilingOf<kPromptRows, kPromptKeys, 2, 4>;

// One block's note for the join: the unit whose first part it has, if that
// unit has several.
struct JoinNote {
    int parts, q0, len, head, r;
    unsigned slot0, slot1;
    int pad;
};

template <int kDim>
struct PromptShape {
    static constexpr int kTileBytes = 128 * kDim * 2;  // of q, K or V
    static constexpr int kQAt = 0;
    static constexpr int kKAt = kQAt + 2 * kTileBytes;
    // E4M3 bytes of the next K and V tile, as they come
    static constexpr int kRawAt = kKAt + kBuffers * kTileBytes;
    static constexpr int kRawBytes = kPromptKeys * kDim;
    // for each of 4 key tiles in turn and group of 16 keys: k_scale,
    // log2(v_scale), 1 / v_scale (the copies are at most 3 tiles ahead of the
    // softmax)
    static constexpr int kScalesAt = kRawAt + 2 * kRawBytes;
    // per V tile in turn and key: which of its values are NaN (filled where rows are masked)
    static constexpr int kNansAt = kScalesAt + 4 * kGroups * 16;
    static constexpr int kRowScaleAt = kNansAt + 2 * kPromptKeys * kDim / 8;
    // per key tile in turn, half and row: the largest t there
    static constexpr int kMaxAt = kRowScaleAt + kPromptRows * 4;
    static constexpr int kSeqsAt = kMaxAt + 2 * 2 * kPromptRows * 4;
    // A partial state, in fp32 words: O as [kDim / 4][row][4] (neighbouring rows,
    // a row per thread, side by side), maxima [row], sums [row].
    static constexpr int kPartial = kPromptRows * (kDim + 2);
    // TMEM columns
    static constexpr int kO = 256;  // S of tile w at 128 w, O of tile w at kO + kDim w
};

__device__ __forceinline__ void tmem_load32(uint32_t at, float (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]),
          "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]),
          "=f"(v[14]), "=f"(v[15]), "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]),
          "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]), "=f"(v[25]),
          "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
        : "r"(at)
        : "memory");
}

__device__ __forceinline__ void tmem_store32(uint32_t at, const float (&v)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(at),
        "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]),
        "f"(v[8]), "f"(v[9]), "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]),
        "f"(v[15]), "f"(v[16]), "f"(v[17]), "f"(v[18]), "f"(v[19]), "f"(v[20]), "f"(v[21]),
        "f"(v[22]), "f"(v[23]), "f"(v[24]), "f"(v[25]), "f"(v[26]), "f"(v[27]), "f"(v[28]),
        "f"(v[29]), "f"(v[30]), "f"(v[31])
        : "memory");
}

__device__ __forceinline__ void tmem_store16(uint32_t at, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(at),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
        "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]),
        "r"(v[15])
        : "memory");
}

// The values pass through the wait, so that no use of them moves in front of it.
__device__ __forceinline__ void tmem_wait_load(float (&v)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]),
                   "+f"(v[7]), "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]),
                   "+f"(v[14]), "+f"(v[15]), "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]),
                   "+f"(v[21]), "+f"(v[22]), "+f"(v[23]), "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]),
                   "+f"(v[28]), "+f"(v[29]), "+f"(v[30]), "+f"(v[31])
                 :
                 : "memory");
}
__device__ __forceinline__ void tmem_wait_store() {
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_fence_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tmem_fence_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// Generic writes to shared memory before the tensor cores' reads.
__device__ __forceinline__ void fence_shared_to_async() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// Shared-memory operand descriptor: 128-byte swizzle, 8 rows of 128 bytes per
// 1024; `leading` is the distance of 64-value blocks (transposed operand).
__device__ __forceinline__ uint64_t operand(uint32_t at, uint32_t leading) {
    return (uint64_t)((at & 0x3ffffu) >> 4) | (uint64_t)(leading >> 4) << 16 |
           (uint64_t)(1024 >> 4) << 32 | 1ull << 46 | 2ull << 61;
}

// Instruction descriptor: f16 operands, fp32 sums, 128 rows, n columns; the
// second operand transposed or not.
__device__ __forceinline__ constexpr uint32_t instruction(int n, bool transposed) {
    return 1u << 4 | (transposed ? 1u << 16 : 0u) | (uint32_t)(n / 8) << 17 |
           (uint32_t)(128 / 16) << 24;
}

__device__ __forceinline__ void mma_shared(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                           bool add) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(add ? 1 : 0)
        : "memory");
}

__device__ __forceinline__ void mma_tmem(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                         bool add) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(add ? 1 : 0)
        : "memory");
}

// `bar` completes when all products issued so far have.
__device__ __forceinline__ void mma_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                     bar)
                 : "memory");
}

// One row of half a tile of scores, from TMEM at s_at.
struct ScoreRow {
    uint32_t s_at;
    float row_scale;
    const float4* scales;  // per 16 keys: k_scale, log2(v_scale), 1 / v_scale
    int hi, lo, sinks;     // keys that the row sees, from the half's first
};

template <bool kGuard>
__device__ __forceinline__ bool sees(const ScoreRow& r, int j) {
    return !kGuard || (j < r.hi && (j >= r.lo || j < r.sinks));
}

// The largest t of the row.
template <bool kGuard>
__device__ __forceinline__ float largest(const ScoreRow& r) {
    float most = -INFINITY;
#pragma unroll
    for (int c = 0; c < kHalfKeys / 32; ++c) {
        float x[32];
        tmem_load32(r.s_at + 32 * c, x);
        tmem_wait_load(x);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int e = 0; e < 16; ++e)
                if (sees<kGuard>(r, 32 * c + 16 * h + e)) m[e & 3] = fmaxf(m[e & 3], x[16 * h + e]);
            const float4 sc = r.scales[2 * c + h];
            most = fmaxf(most, fmaf(fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])),
                                    r.row_scale * sc.x, sc.y));
        }
    }
    return most;
}

// P = 2^(t + shift), as f16 in the first columns of the scores' place (the
// scores there have been used); returns sum P / v_scale.
template <bool kGuard>
__device__ __forceinline__ float weights(const ScoreRow& r, float shift) {
    float sum = 0.0f;
#pragma unroll
    for (int c = 0; c < kHalfKeys / 32; ++c) {
        float x[32];
        tmem_load32(r.s_at + 32 * c, x);
        tmem_wait_load(x);
        uint32_t p[16];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float4 sc = r.scales[2 * c + h];
            const float by = r.row_scale * sc.x, off = sc.y + shift;
            const uint64_t by2 = pair(by, by), off2 = pair(off, off);
            uint64_t total[2] = {pair(0.0f, 0.0f), pair(0.0f, 0.0f)};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float2 t = unpair(fma2(pair(x[16 * h + 2 * e], x[16 * h + 2 * e + 1]), by2, off2));
                if (kGuard) {
                    const int j = 32 * c + 16 * h + 2 * e;
                    if (!sees<kGuard>(r, j)) t.x = -INFINITY;
                    if (!sees<kGuard>(r, j + 1)) t.y = -INFINITY;
                }
                t.x = exp2_fast(t.x);
                t.y = exp2_fast(t.y);
                total[e & 1] = add2(total[e & 1], pair(t.x, t.y));
                p[8 * h + e] = f16x2(t.x, t.y);
            }
            const float2 two = unpair(add2(total[0], total[1]));
            sum = fmaf(two.x + two.y, sc.z, sum);
        }
        tmem_store16(r.s_at + 16 * c, p);
    }
    return sum;
}

// A barrier of 64 threads (two warps); whether all of them pass `ok`.
__device__ __forceinline__ bool pair_barrier(int id, bool ok) {
    uint32_t all;
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.u32 p, %2, 0;\n"
        " barrier.cta.red.and.pred q, %1, 64, p;\n selp.u32 %0, 1, 0, q;\n}"
        : "=r"(all)
        : "r"(id), "r"(ok ? 1u : 0u)
        : "memory");
    return all != 0;
}

struct TileNote {
    int j0;
    unsigned paged;
    bool masked;
};

// The block's barriers, each completed once per use.
struct Barriers {
    uint64_t q_full;       // q tiles of a segment written
    uint64_t full[kBuffers], empty[kBuffers];  // K and V tiles in turn
    uint64_t raw_full[2], raw_empty[2];  // E4M3 bytes of K, of V
    uint64_t scales_full[4];             // page scales of 4 key tiles in turn
    // of row tile w: scores, P in their place, O with it added
    uint64_t s_full[2], p_full[2], o_full[2];
    uint64_t drained;      // after a wait that ran out: all products issued
};

// Where the kernel leaves its notes for the join and its status, and how long a wait
// may take.  stall (testing only): the copies stop behind half of a segment's tiles.
struct PromptRun {
    JoinNote* notes;
    int* status;
    unsigned long long wait_ns;
    int stall;
};

template <int kDim, bool kFew>
__global__ void __launch_bounds__(kPromptThreads, 1)
    kv8_prompt_kernel(const AttentionArgs a, const PromptRun run) {
    using S = PromptShape<kDim>;
    extern __shared__ __align__(1024) uint8_t dynamic[];
    // the swizzle goes by address: tiles begin on multiples of 1024
    uint8_t* const shared = dynamic + (-smem_addr(dynamic) & 1023u);
    __shared__ Barriers bars;
    __shared__ Plan<PromptTiling> plan;
    __shared__ Segment segments[3];
    __shared__ int work;
    __shared__ volatile int abort;
    __shared__ int nan_tile[2];  // of 2 V tiles in turn: the last in which a NaN was found
    // of 4 key tiles in turn: first key, which groups of keys have a page, whether
    // some row does not see some key
    __shared__ TileNote tile_notes[4];
    __shared__ uint32_t tmem_at;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t smem = smem_addr(shared);
    constexpr int kIssueWarp = kSoftmaxWarps + kConvertWarps, kCopyWarp = kIssueWarp + 1;
    Seq* const seqs = reinterpret_cast<Seq*>(shared + S::kSeqsAt);

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                         smem_addr(&tmem_at))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (tid == 32) {
        mbar_init(smem_addr(&bars.q_full), kSoftmaxWarps * 32);
        for (int i = 0; i < 4; ++i) mbar_init(smem_addr(&bars.scales_full[i]), 1);
        for (int i = 0; i < kBuffers; ++i) {
            mbar_init(smem_addr(&bars.full[i]), kConvertWarps * 32);
            mbar_init(smem_addr(&bars.empty[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_addr(&bars.s_full[i]), 1);
            mbar_init(smem_addr(&bars.p_full[i]), 256);
            mbar_init(smem_addr(&bars.o_full[i]), 1);
            mbar_init(smem_addr(&bars.raw_full[i]), 1);
            mbar_init(smem_addr(&bars.raw_empty[i]), kConvertWarps);
            nan_tile[i] = -1;
        }
        mbar_init(smem_addr(&bars.drained), 1);
        abort = 0;
        fence_mbar_init();
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    Scheduler<PromptTiling, kFew> scheduler(a, &plan, seqs, segments);
    if (warp == kIssueWarp) {
        const bool some = scheduler.start();
        if (lane == 0) {
            work = some;
            run.notes[blockIdx.x].parts = 0;
        }
    }
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = tmem_at;

    // Waits for a barrier's completion number `uses` (from 0); false, with the
    // status set, when it does not come in time.
    auto wait_lane = [&](uint64_t& bar, unsigned uses) {
        if (mbar_wait_bounded(smem_addr(&bar), uses & 1, &abort, run.wait_ns)) return true;
        abort = 1;
        *run.status = kKv8Timeout;
        return false;
    };
    auto wait = [&](uint64_t& bar, unsigned uses) {  // the same answer for a whole warp
        return __all_sync(0xffffffffu, wait_lane(bar, uses)) != 0;
    };

    // of the segments before this one: key tiles, and those of the two row tiles
    // (a unit may lack the second)
    unsigned done = 0, row_done[2] = {0, 0};
    unsigned copied[2] = {0, 0};  // copying warp: tiles of K, of V whose copies were started
    for (int number = 0; work; ++number) {
        const Segment& g = segments[number % 3];
        const int n = g.x1 - g.x0;
        const bool last = g.last;
        const int rows = min(g.len * a.group - g.r * kPromptRows, kPromptRows);
        const int tiles = rows > 128 ? 2 : 1;  // 128-row tiles that hold rows
        const Keys keys = g.keys;
        auto tile_start = [&](int x) {
            return (x < keys.sink_tiles ? x : keys.lo / kPromptKeys + x - keys.sink_tiles) *
                   kPromptKeys;
        };
        auto masked = [&](int j0) {  // some row does not see some key of the tile
            return j0 + kPromptKeys > keys.hi_min ||
                   (j0 < keys.lo_max && j0 + kPromptKeys > a.sinks);
        };
        if (n <= 0) break;

        if (warp < kSoftmaxWarps) {
            // ---- q, then the softmax of row tile w: a thread has one row's keys of
            // half h of each key tile
            const int w = warp >> 3, h = warp >> 2 & 1;
            {
                constexpr int kLanes = kDim / 8;  // lanes per row
                constexpr int kSteps = kPromptRows / kSoftmaxWarps * kLanes / 32;
                const int sub = lane / kLanes, d = lane % kLanes;
                const int row0 = warp * (kPromptRows / kSoftmaxWarps) + sub;
                uint4 x[kSteps];
#pragma unroll
                for (int i = 0; i < kSteps; ++i) {
                    const int unit_row = g.r * kPromptRows + row0 + i * (32 / kLanes);
                    const int token = token_of(a, unit_row);
                    const bool live = token < g.len;
                    const __nv_bfloat16* const from =
                        a.q + (long long)(g.q0 + (live ? token : 0)) * a.q_stride +
                        (size_t)(g.head * a.group + (live ? unit_row - token * a.group : 0)) * kDim;
                    x[i] = reinterpret_cast<const uint4*>(from)[d];
                }
#pragma unroll
                for (int i = 0; i < kSteps; ++i) {
                    const int row = row0 + i * (32 / kLanes);
                    // rows beyond the last are zeros
                    if (token_of(a, g.r * kPromptRows + row) >= g.len)
                        x[i] = make_uint4(0, 0, 0, 0);
                    const uint32_t u[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
                    float big = 0.0f;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        big = fmaxf(big, fmaxf(fabsf(bf16_lo(u[e])), fabsf(bf16_hi(u[e]))));
#pragma unroll
                    for (int m = kLanes / 2; m > 0; m >>= 1)
                        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, m));
                    // 2^e brings the row's largest value into [2^14, 2^15); a negative
                    // softmax_scale goes into the sign of q, so larger scores stay larger
                    const int e = min(14 + 127 - (int)(__float_as_uint(big) >> 23), 126);
                    float up = __uint_as_float((uint32_t)(e + 127) << 23);
                    if (a.scale < 0.0f) up = -up;
                    uint32_t f[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        f[k] = f16x2(bf16_lo(u[k]) * up, bf16_hi(u[k]) * up);
                    uint8_t* const to = shared + S::kQAt + (row >> 7) * S::kTileBytes +
                                        (d >> 3) * 128 * 128 + (row & 127) * 128 +
                                        ((d ^ row) & 7) * 16;
                    *reinterpret_cast<uint4*>(to) = make_uint4(f[0], f[1], f[2], f[3]);
                    if (d == 0)
                        reinterpret_cast<float*>(shared + S::kRowScaleAt)[row] =
                            fabsf(a.scale) * __uint_as_float((uint32_t)(127 - e) << 23);
                }
                fence_shared_to_async();
                mbar_arrive(smem_addr(&bars.q_full));
            }
            if (w < tiles) {
                bool ok = wait(bars.q_full, number);  // and the row scales
                const int row = w * 128 + (tid & 127);
                const int unit_row = g.r * kPromptRows + row;
                const int token = token_of(a, unit_row);
                const int hi = token < g.len ? g.first + token + 1 : 0;
                const int lo = window_start(a, hi);
                const float row_scale =
                    reinterpret_cast<const float*>(shared + S::kRowScaleAt)[row];
                const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21);
                const uint32_t s_at = lanes + w * 128 + h * kHalfKeys;
                constexpr int kMine = kDim / 2;  // columns of O that this thread scales and writes
                const uint32_t o_at = lanes + S::kO + w * kDim + h * kMine;
                const int partners = 1 + w * 4 + (warp & 3);  // their barrier
                float* const maxima = reinterpret_cast<float*>(shared + S::kMaxAt) + row;
                float top = -INFINITY, sum = 0.0f;
                const unsigned before = w ? row_done[1] : row_done[0];
                {
                    float zero[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) zero[e] = 0.0f;
#pragma unroll
                    for (int c = 0; c < kMine / 32; ++c) tmem_store32(o_at + 32 * c, zero);
                }
#pragma unroll 1
                for (int i = 0; i < n; ++i) {
                    const unsigned at = done + i;
                    ok = ok && wait(bars.scales_full[at & 3], at >> 2) &&
                         wait(bars.s_full[w], before + i);
                    tmem_fence_after();
                    const int from = tile_notes[at & 3].j0 + h * kHalfKeys;
                    const bool guard = tile_notes[at & 3].masked;
                    const ScoreRow scores{s_at, row_scale,
                                          reinterpret_cast<const float4*>(shared + S::kScalesAt) +
                                              (at & 3) * kGroups + h * (kGroups / 2),
                                          hi - from, lo - from, a.sinks - from};
                    float most = guard ? largest<true>(scores) : largest<false>(scores);
                    float* const here = maxima + (at & 1) * 2 * kPromptRows;
                    here[h * kPromptRows] = most;
                    // A row's two threads leave the loop together.
                    ok = pair_barrier(partners, ok);
                    if (!ok) break;
                    most = fmaxf(most, here[(h ^ 1) * kPromptRows]);
                    if (__any_sync(0xffffffffu, most > top + kSlack)) {
                        const float now = fmaxf(most, top);
                        const float keep = now == -INFINITY ? 1.0f : exp2_fast(top - now);
                        top = now;
                        sum *= keep;
                        // all of O so far: these scores came after it
#pragma unroll 1
                        for (int c = 0; c < kMine / 32 && i > 0; ++c) {
                            float v[32];
                            tmem_load32(o_at + 32 * c, v);
                            tmem_wait_load(v);
#pragma unroll
                            for (int e = 0; e < 32; ++e) v[e] *= keep;
                            tmem_store32(o_at + 32 * c, v);
                        }
                    }
                    const float shift = kPromptBias - (top == -INFINITY ? 0.0f : top);
                    sum += guard ? weights<true>(scores, shift) : weights<false>(scores, shift);
                    if (guard) {
                        const unsigned item = 2 * at + 1;
                        ok = wait(bars.full[item % kBuffers], item / kBuffers);
                        if (ok && nan_tile[at & 1] == (int)at) {
                            // NaNs among the keys that the row sees, straight into O
                            const uint32_t* const bits =
                                reinterpret_cast<const uint32_t*>(shared + S::kNansAt +
                                                                  (at & 1) * kPromptKeys * kDim / 8) +
                                h * kMine / 32;
#pragma unroll 1
                            for (int c = 0; c < kMine / 32; ++c) {
                                uint32_t bad = 0;
                                for (int j = 0; j < kPromptKeys; ++j)
                                    if (sees<true>(scores, j - h * kHalfKeys))
                                        bad |= bits[j * kDim / 32 + c];
                                __syncwarp();
                                tmem_wait_store();
                                float v[32];
                                tmem_load32(o_at + 32 * c, v);
                                tmem_wait_load(v);
#pragma unroll
                                for (int e = 0; e < 32; ++e)
                                    if (bad >> e & 1) v[e] = NAN;
                                tmem_store32(o_at + 32 * c, v);
                            }
                        }
                        __syncwarp();
                    }
                    tmem_wait_store();
                    tmem_fence_before();
                    mbar_arrive(smem_addr(&bars.p_full[w]));
                }
                ok = ok && wait(bars.o_full[w], before + n - 1);
                tmem_wait_store();  // where the loop was left early
                // in the place that the partner has read two tiles ago
                float* const here = maxima + ((done + n) & 1) * 2 * kPromptRows;
                here[h * kPromptRows] = sum;
                if (pair_barrier(partners, ok)) {
                    sum += here[(h ^ 1) * kPromptRows];
                    tmem_fence_after();
                    const bool live = token < g.len;
                    const bool whole = g.parts == 1;
                    const size_t out_row = (size_t)(g.q0 + (live ? token : 0)) * a.heads +
                                           g.head * a.group +
                                           (live ? unit_row - token * a.group : 0);
                    float* const part = a.partials + (size_t)g.slot * S::kPartial;
                    const float inv = sum == 0.0f ? 0.0f : __fdiv_rn(1.0f, sum);
#pragma unroll
                    for (int c = 0; c < kMine / 32; ++c) {
                        float v[32];
                        __syncwarp();
                        tmem_load32(o_at + 32 * c, v);
                        tmem_wait_load(v);
                        if (live && whole) {
                            uint4* const to = reinterpret_cast<uint4*>(a.out + out_row * kDim +
                                                                       h * kMine + 32 * c);
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                to[e] = make_uint4(bf16x2(v[8 * e] * inv, v[8 * e + 1] * inv),
                                                   bf16x2(v[8 * e + 2] * inv, v[8 * e + 3] * inv),
                                                   bf16x2(v[8 * e + 4] * inv, v[8 * e + 5] * inv),
                                                   bf16x2(v[8 * e + 6] * inv, v[8 * e + 7] * inv));
                        } else if (live) {
                            float4* const to = reinterpret_cast<float4*>(part) +
                                               (h * kMine + 32 * c) / 4 * kPromptRows + row;
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                to[e * kPromptRows] = make_float4(v[4 * e], v[4 * e + 1],
                                                                  v[4 * e + 2], v[4 * e + 3]);
                        }
                    }
                    if (live && whole && a.lse && h == 0)
                        a.lse[out_row] = sum == 0.0f ? -INFINITY
                                                     : 0.69314718055994531f *
                                                           ((top - kPromptBias) + log2f(sum));
                    if (live && !whole && h == 0) {
                        part[kPromptRows * kDim + row] = top;
                        part[kPromptRows * (kDim + 1) + row] = sum;
                    }
                    tmem_fence_before();
                }
            }
        } else if (warp < kIssueWarp) {
            // ---- E4M3 bytes to f16 tiles: a lane has 16 values of one key at a time
            const int t = warp - kSoftmaxWarps, q = lane >> 2;
            constexpr int kItems = kDim / 16;
            // neighbouring rows read and write different halves of a line: no two of
            // 8 lanes meet on a bank, neither in the bytes nor in the swizzled tile
            const int piece = kDim == 128 ? (lane & 3) + 4 * ((q & 1) ^ (t >> 1)) : lane & 3;
            const int row0 = kDim == 128 ? 8 * (t & 1) + q : 8 * t + q;
            constexpr int kRowStep = kDim == 128 ? 16 : 32;
            const uint32_t raw = smem + S::kRawAt + row0 * kDim + piece * 16;
            auto store = [&](const uint4& x, uint32_t tile, int row) {
                const uint32_t u[4] = {x.x, x.y, x.z, x.w};
                uint32_t h[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    h[2 * e] = e4m3x2_to_f16x2(u[e]);
                    h[2 * e + 1] = e4m3x2_hi_to_f16x2(u[e]);
                }
                uint8_t* const to = shared + tile + (piece >> 2) * 128 * 128 + row * 128;
                const int c = 2 * (piece & 3);
                *reinterpret_cast<uint4*>(to + ((c ^ row) & 7) * 16) =
                    make_uint4(h[0], h[1], h[2], h[3]);
                *reinterpret_cast<uint4*>(to + (((c + 1) ^ row) & 7) * 16) =
                    make_uint4(h[4], h[5], h[6], h[7]);
            };
            bool ok = true;
            for (int i = 0; i < n && ok; ++i) {
                const unsigned at = done + i;
                // a buffer's barrier completes once per use
                auto buffer = [&](unsigned item) {
                    if (item >= kBuffers)
                        ok = wait(bars.empty[item % kBuffers], item / kBuffers - 1);
                    return S::kKAt + item % kBuffers * S::kTileBytes;
                };
                ok = wait(bars.raw_full[0], at);
                if (!ok) break;
                const int j0 = tile_notes[at & 3].j0;
                const bool guard = tile_notes[at & 3].masked;
                const unsigned pages = tile_notes[at & 3].paged;
                const bool partly = pages != (1u << kGroups) - 1 || j0 + kPromptKeys > keys.hi ||
                                    (j0 < keys.lo && j0 + kPromptKeys > a.sinks);
                // all of a tile's bytes first: their latency is paid once
                uint4 x[kItems];
                auto read = [&](int which) {
#pragma unroll
                    for (int m = 0; m < kItems; ++m)
                        x[m] = lds128(raw + which * S::kRawBytes + m * kRowStep * kDim);
                    if (!partly) return;
                    // keys that no row sees, and those without a page, become zeros
#pragma unroll
                    for (int m = 0; m < kItems; ++m) {
                        const int row = row0 + m * kRowStep, j = j0 + row;
                        if (!(pages >> (row >> 4) & 1) || j >= keys.hi ||
                            (j < keys.lo && j >= a.sinks))
                            x[m] = make_uint4(0, 0, 0, 0);
                    }
                };
                read(0);
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&bars.raw_empty[0]));
                const uint32_t k_at = buffer(2 * at);
                if (!ok) break;
#pragma unroll
                for (int m = 0; m < kItems; ++m) store(x[m], k_at, row0 + m * kRowStep);
                fence_shared_to_async();
                mbar_arrive(smem_addr(&bars.full[2 * at % kBuffers]));
                ok = wait(bars.raw_full[1], at);
                if (!ok) break;
                read(1);
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&bars.raw_empty[1]));
                const uint32_t v_at = buffer(2 * at + 1);
                if (!ok) break;
                if (guard) {
                    // NaNs out of the product, and where they were
                    uint32_t any = 0;
#pragma unroll
                    for (int m = 0; m < kItems; ++m) {
                        uint32_t u[4] = {x[m].x, x[m].y, x[m].z, x[m].w}, bits = 0;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint32_t bad = nan_bytes(u[e]) >> 7;
                            u[e] &= ~(bad * 0xffu);
                            bits |= ((bad * 0x00204081u) >> 21 & 0xfu) << (4 * e);
                        }
                        x[m] = make_uint4(u[0], u[1], u[2], u[3]);
                        any |= bits;
                        reinterpret_cast<uint16_t*>(
                            shared + S::kNansAt +
                            (at & 1) * kPromptKeys * kDim / 8)[(row0 + m * kRowStep) * kDim / 16 + piece] =
                            (uint16_t)bits;
                    }
                    if (any) nan_tile[at & 1] = (int)at;
                }
#pragma unroll
                for (int m = 0; m < kItems; ++m) store(x[m], v_at, row0 + m * kRowStep);
                fence_shared_to_async();
                mbar_arrive(smem_addr(&bars.full[(2 * at + 1) % kBuffers]));
            }
        } else if (warp == kCopyWarp) {
            // ---- pages into shared memory as they are: a group of 16 keys is one
            // piece of a page, copied by lane l < 8
            const int page_mask = (1 << a.bt.page_shift) - 1;
            // the table's entry for the lane's keys of tile x, -2 without keys
            auto find_page = [&](int x) {
                const int j = tile_start(x) + 16 * lane;
                if (lane >= kGroups || x >= g.x1 || j >= keys.hi) return -2;
                return a.bt.page_table[(size_t)g.b * a.bt.table_width + (j >> a.bt.page_shift)];
            };
            auto exists = [&](int page) { return page >= 0 && page < a.c.pages; };
            auto scale_of = [&](const float* scales, int page) {
                return exists(page) ? scales[(size_t)page * a.c.kv_heads + g.head] : 0.0f;
            };
            int page = find_page(g.x0), next = find_page(g.x0 + 1);
            float ks = scale_of(a.c.k_scales, page), vs = scale_of(a.c.v_scales, page);
            bool ok = true;
            const int tiles_to_copy = run.stall ? n / 2 : n;
            for (int i = 0; i < tiles_to_copy && ok; ++i) {
                const unsigned at = done + i;
                const int x = g.x0 + i;
                const bool have = exists(page);
                if (!have && page != -2) kv8_report(a.bt);
                const unsigned groups = __ballot_sync(0xffffffffu, have);
                const uint32_t bytes = __popc(groups) * 16 * kDim;
                const int j = tile_start(x) + 16 * lane;
                const size_t from =
                    ((((size_t)(have ? page : 0) * a.c.kv_heads + g.head) << a.bt.page_shift) +
                     (j & page_mask)) *
                    kDim;
                const int after = find_page(x + 2);
                const float ks1 = scale_of(a.c.k_scales, next), vs1 = scale_of(a.c.v_scales, next);
#pragma unroll
                for (int which = 0; which < 2; ++which) {
                    if (ok && at >= 1) ok = wait(bars.raw_empty[which], at - 1);
                    if (!ok) break;
                    if (which == 0) {
                        if (lane < kGroups) {
                            const float v = usable_scale(vs);
                            reinterpret_cast<float4*>(shared +
                                                      S::kScalesAt)[(at & 3) * kGroups + lane] =
                                have ? make_float4(ks, __log2f(v), __fdividef(1.0f, v), 0.0f)
                                     : make_float4(0.0f, -INFINITY, 0.0f, 0.0f);
                        }
                        if (lane == 0) {
                            const int j0 = tile_start(x);
                            tile_notes[at & 3] = TileNote{j0, groups, masked(j0)};
                        }
                        __syncwarp();
                        if (lane == 0) mbar_arrive(smem_addr(&bars.scales_full[at & 3]));
                    }
                    const uint32_t bar = smem_addr(&bars.raw_full[which]);
                    if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
                    copied[which] = at + 1;
                    __syncwarp();
                    if (have)
                        bulk_copy_g2s(smem + S::kRawAt + which * S::kRawBytes + lane * 16 * kDim,
                                      (which ? a.c.v_codes : a.c.k_codes) + from, 16 * kDim, bar);
                }
                page = next;
                next = after;
                ks = ks1;
                vs = vs1;
            }
        } else if (lane == 0) {
            // ---- the products.  One thread issues both row tiles' in turn: issued by
            // two, they would share the tensor cores evenly and end together, and both
            // softmaxes would then run at one time and leave the tensor cores idle.
            const uint64_t q_op = operand(smem + S::kQAt, 16);
            const uint64_t k_op = operand(smem + S::kKAt, 16);
            const uint64_t v_op = operand(smem + S::kKAt, 128 * 128);
            constexpr uint32_t kTileUnits = S::kTileBytes >> 4, kBlockUnits = 128 * 128 >> 4;
            auto filled = [&](unsigned item) {
                return wait_lane(bars.full[item % kBuffers], item / kBuffers);
            };
            auto release = [&](unsigned item) {
                mma_commit(smem_addr(&bars.empty[item % kBuffers]));
            };
            auto scores = [&](int w, unsigned item) {
                const uint64_t q = q_op + w * kTileUnits, key = k_op + item % kBuffers * kTileUnits;
#pragma unroll
                for (int k = 0; k < kDim / 16; ++k) {
                    const uint32_t off = (k / 4) * kBlockUnits + (k % 4) * 2;
                    mma_shared(tmem + w * 128, q + off, key + off, instruction(kPromptKeys, false),
                               k > 0);
                }
                mma_commit(smem_addr(&bars.s_full[w]));
                if (w + 1 == tiles) release(item);
            };
            bool ok = wait_lane(bars.q_full, number) && filled(2 * done);
            if (ok) {
                tmem_fence_after();
#pragma unroll 1
                for (int w = 0; w < tiles; ++w) scores(w, 2 * done);
            }
#pragma unroll 1
            for (int i = 0; i < n && ok; ++i) {
                const unsigned item = 2 * (done + i) + 1;  // V
                const uint64_t value = v_op + item % kBuffers * kTileUnits;
                ok = filled(item);
#pragma unroll 1
                for (int w = 0; w < tiles && ok; ++w) {
                    const unsigned use = (w ? row_done[1] : row_done[0]) + i;
                    ok = wait_lane(bars.p_full[w], use);
                    if (!ok) break;
                    tmem_fence_after();
#pragma unroll
                    for (int k = 0; k < kPromptKeys / 16; ++k)
                        mma_tmem(tmem + S::kO + w * kDim,
                                 tmem + w * 128 + (k / 4) * kHalfKeys + (k % 4) * 8,
                                 value + k * (2048 >> 4), instruction(kDim, true), true);
                    mma_commit(smem_addr(&bars.o_full[w]));
                    if (w + 1 == tiles) release(item);
                    if (i + 1 == n) continue;
                    // The next scores take the place of P: products on different sums are
                    // not ordered, so these have to be complete.
                    ok = filled(item + 1) && wait_lane(bars.o_full[w], use);
                    if (!ok) break;
                    tmem_fence_after();
                    scores(w, item + 1);
                }
            }
        }
        __syncwarp();
        if (warp == kIssueWarp) {
            if (lane == 0 && g.parts > 1 && g.counter == blockIdx.x)
                run.notes[blockIdx.x] =
                    JoinNote{g.parts, g.q0, g.len, g.head, g.r, g.slot0, g.slot1, 0};
            if (!last) scheduler.next();
        }
        done += n;
        row_done[0] += n;
        if (tiles == 2) row_done[1] += n;
        tmem_fence_before();
        __syncthreads();
        tmem_fence_after();
        if (last || abort) break;
    }
    if (abort) {
        // Copies and products under way end before the memory that they use is left:
        // by the threads that started them, whose waits heed no other's.
        const int none = 0;
        if (warp == kCopyWarp && lane == 0)
            for (int i = 0; i < 2; ++i)
                if (copied[i] > 0)
                    mbar_wait_bounded(smem_addr(&bars.raw_full[i]), (copied[i] - 1) & 1, &none);
        if (warp == kIssueWarp && lane == 0) {
            mma_commit(smem_addr(&bars.drained));
            mbar_wait_bounded(smem_addr(&bars.drained), 0, &none);
        }
    }
    __syncthreads();
    if (warp == 0)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem)
                     : "memory");
}

// Joins the parts of the unit whose first part block blockIdx.x had, for
// kJoinValues of each row's values: a row per thread.
constexpr int kJoinValues = 8;

template <int kDim>
__global__ void __launch_bounds__(kPromptRows) kv8_prompt_join_kernel(const AttentionArgs a,
                                                                      const JoinNote* const notes) {
    using S = PromptShape<kDim>;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const JoinNote g = notes[blockIdx.x];
    const int row = threadIdx.x, unit_row = g.r * kPromptRows + row;
    if (g.parts < 2 || token_of(a, unit_row) >= g.len) return;
    auto part = [&](int i) {
        return a.partials + (size_t)(i == 0 ? g.slot0 : g.slot1 + 2 * (i - 1)) * S::kPartial;
    };
    float top = -INFINITY;
#pragma unroll 8
    for (int i = 0; i < g.parts; ++i) top = fmaxf(top, part(i)[kPromptRows * kDim + row]);
    constexpr int kVectors = kJoinValues / 4;
    float sum = 0.0f;
    float4 v[kVectors];
#pragma unroll
    for (int k = 0; k < kVectors; ++k) v[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
    for (int i = 0; i < g.parts; ++i) {
        const float* p = part(i);
        const float f = weight_of(p[kPromptRows * kDim + row], top);
        sum = fmaf(p[kPromptRows * (kDim + 1) + row], f, sum);
#pragma unroll
        for (int k = 0; k < kVectors; ++k) {
            const float4 y = reinterpret_cast<const float4*>(
                p)[(blockIdx.y * kVectors + k) * kPromptRows + row];
            v[k].x = fmaf(y.x, f, v[k].x);
            v[k].y = fmaf(y.y, f, v[k].y);
            v[k].z = fmaf(y.z, f, v[k].z);
            v[k].w = fmaf(y.w, f, v[k].w);
        }
    }
#pragma unroll
    for (int k = 0; k < kVectors; ++k)
        store_row<kDim>(a, g.q0, g.len, g.head, unit_row, (blockIdx.y * kVectors + k) * 4, v[k],
                        top - kPromptBias, sum);
}

template <int kDim, bool kFew>
cudaError_t launch(const AttentionArgs& a, const PromptRun& run, int num_sms, cudaStream_t s) {
    using S = PromptShape<kDim>;
    static std::atomic<bool> allowed[64];  // per device: the kernel's shared memory limit is set
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !allowed[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(kv8_prompt_kernel<kDim, kFew>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 1024 + S::kSeqsAt + kKv8MaxBatch * (int)sizeof(Seq));
        if (e != cudaSuccess) return e;
        if (dev < 64) allowed[dev].store(true, std::memory_order_release);
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(num_sms);
    cfg.blockDim = dim3(kPromptThreads);
    cfg.dynamicSmemBytes = 1024 + S::kSeqsAt + a.bt.batch * sizeof(Seq);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kv8_prompt_kernel<kDim, kFew>, a, run);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3(num_sms, kDim / kJoinValues);
    cfg.blockDim = dim3(kPromptRows);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, kv8_prompt_join_kernel<kDim>, a,
                              (const JoinNote*)run.notes);
}

}  // namespace

bool kv8_prompt_applies(int head_dim, long long tokens, int group, int batch) {
    return head_dim <= 128 && tokens * group > (long long)kPromptRowsAbove * batch;
}

size_t kv8_prompt_data_bytes(int head_dim, int num_sms) {
    const size_t notes = ((size_t)num_sms * sizeof(JoinNote) + 255) / 256 * 256;
    return notes + (size_t)num_sms * 2 * kPromptRows * (head_dim + 2) * sizeof(float);
}

cudaError_t launch_kv8_prompt(AttentionArgs a, void* data, int* status, int num_sms,
                              cudaStream_t s) {
    const PromptRun run{reinterpret_cast<JoinNote*>(data), status, test_wait_ns(), test_stall()};
    a.partials = reinterpret_cast<float*>(reinterpret_cast<char*>(data) +
                                          ((size_t)num_sms * sizeof(JoinNote) + 255) / 256 * 256);
    // equal parts, as in kv8_attention.cu (one prompt of 512 tokens, 32 heads on 8: 24.2 us
    // against 25.1 in one line of tiles)
    const long long rows = (long long)a.bt.tokens * a.group;
    const bool few = (rows / kPromptRows + a.bt.batch) * a.c.kv_heads <= num_sms / 2;
    if (a.c.head_dim == 64)
        return few ? launch<64, true>(a, run, num_sms, s)
                   : launch<64, false>(a, run, num_sms, s);
    return few ? launch<128, true>(a, run, num_sms, s)
               : launch<128, false>(a, run, num_sms, s);
}

}  // namespace nvf
