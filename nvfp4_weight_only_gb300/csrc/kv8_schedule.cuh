// kv8_schedule.cuh -- what the attention kernels share: their arguments, the
// keys that a tile of rows sees, and how the work is cut into equal ranges, one
// per block, from lengths that are read on the device.
//
// Unit: one sequence, one kv head and a tile of rows (new tokens x the query
// heads that share the kv head, the head fastest).  A unit's visible keys form
// tiles; a unit that several blocks share is joined from their partial states
// in the order of the ranges, so results do not depend on timing.
#pragma once
#include "kv8.cuh"

namespace nvf {

struct AttentionArgs {
    Kv8CacheArgs c;
    Kv8BatchArgs bt;
    const __nv_bfloat16* q;
    __nv_bfloat16* out;
    float* lse;  // or null
    int* counters;
    float* partials;
    long long q_stride;
    int heads, group;
    unsigned group_inverse;  // floor(2^32 / group), at most 2^32 - 1
    float scale;  // softmax_scale * log2(e)
    int window, sinks;  // window 2^31 - 1: every key
};

// row / group: the product with the inverse is the quotient or one less.
__device__ __forceinline__ int token_of(const AttentionArgs& a, int row) {
    const unsigned q = __umulhi((unsigned)row, a.group_inverse);
    return (int)(q + ((unsigned)row - q * a.group >= (unsigned)a.group ? 1 : 0));
}

// kv8_prompt.cu: the same operator for many rows per sequence and kv head.
bool kv8_prompt_applies(int head_dim, long long tokens, int group, int batch);
size_t kv8_prompt_data_bytes(int head_dim, int num_sms);
cudaError_t launch_kv8_prompt(AttentionArgs a, void* data, int* status, int num_sms,
                              cudaStream_t s);

// Rows per unit, keys per tile, least tiles per block, and what a unit or a
// piece of one costs beside its tiles, in tiles.
template <int kRowsOf, int kTileOf, int kMinTilesOf, int kUnitCostOf>
struct TilingOf {
    static constexpr int kRows = kRowsOf, kTile = kTileOf;
    static constexpr int kMinTiles = kMinTilesOf, kUnitCost = kUnitCostOf;
};

// A sequence in shared memory: its new tokens, length, and the tiles of all
// sequences before it.
struct Seq {
    int q0, len, kv;
    unsigned before;
};

// The keys of one unit: [lo, hi) and the sinks in front, as tiles.
struct Keys {
    int lo, hi;          // hi <= 0: none
    int lo_max, hi_min;  // visible to every row of the tile
    int sink_tiles, tiles;
};

// The first key in the window of a query that sees keys below hi (negative for a token
// without a position: as low as -2^30).
__device__ __forceinline__ int window_start(const AttentionArgs& a, int hi) {
    return hi > a.window ? hi - a.window : 0;
}

template <typename T>
__device__ __forceinline__ Keys unit_keys(const AttentionArgs& a, int first, int len, int r) {
    constexpr int kRows = T::kRows, kTile = T::kTile;
    Keys k;
    const int i0 = token_of(a, r * kRows);
    const int i1 = min(token_of(a, r * kRows + kRows - 1), len - 1);
    k.hi_min = first + i0 + 1;
    k.hi = first + i1 + 1;
    k.lo = window_start(a, k.hi_min);
    k.lo_max = window_start(a, k.hi);
    const int lo_tile = k.lo / kTile;
    k.sink_tiles = min((min(a.sinks, k.lo) + kTile - 1) / kTile, lo_tile);
    // a tile that holds no key writes the empty result
    k.tiles = k.hi > 0 ? k.sink_tiles + (k.hi + kTile - 1) / kTile - lo_tile : 1;
    return k;
}

// A piece of one unit that a block takes, and how its state is joined.
struct Segment {
    int b, q0, len, first, head, r;
    Keys keys;
    int x0, x1;            // its tiles
    unsigned slot;         // of its partial state
    unsigned counter;      // of the unit's finished parts
    unsigned slot0, slot1;  // of part 0, of part 1 (then every second one)
    int parts;
    int last;              // the block's last segment
};

__device__ __forceinline__ int row_tiles(const AttentionArgs& a, int len, int rows) {
    return (len * a.group + rows - 1) / rows;  // at most 2^30 rows, `rows` a constant
}

__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void* src, bool full) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(full ? 16 : 0)
                 : "memory");
}

__device__ __forceinline__ void cp_async_commit() {
    asm volatile("cp.async.commit_group;" ::: "memory");
}

template <int kPending>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(at)
                 : "memory");
    return v;
}

__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// Bytes of w that are E4M3's NaN, as 0x80 each.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) {
    return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
}

__device__ __forceinline__ void prefetch_l2(const void* p) {
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}

// Value scales as the softmax takes them.  The denominator is a sum of P / v_scale, P up
// to 2^14, over fewer than 2^31 keys: finite down to 2^-83; and the fast reciprocal of
// a number above 2^126 is 0.
__device__ __forceinline__ float usable_scale(float vs) {
    return fminf(fmaxf(vs, 0x1p-80f), 0x1p126f);
}

__device__ __forceinline__ float weight_of(float top, float all) {
    return all == -INFINITY ? 0.0f : exp2_fast(top - all);
}

// out and lse of one row from its joined state: O and the sum of the weights
// are in units of 2^top.
template <int kDim>
__device__ __forceinline__ void store_row(const AttentionArgs& a, int q0, int len, int head,
                                          int row, int d, float4 v, float top, float sum) {
    const int i = token_of(a, row);
    if (i >= len) return;
    const size_t at = (size_t)(q0 + i) * a.heads + head * a.group + (row - i * a.group);
    const float inv = sum == 0.0f ? 0.0f : __fdiv_rn(1.0f, sum);
    uint2 w;
    w.x = bf16x2(v.x * inv, v.y * inv);
    w.y = bf16x2(v.z * inv, v.w * inv);
    *reinterpret_cast<uint2*>(a.out + at * kDim + d) = w;
    if (d == 0 && a.lse)
        a.lse[at] = sum == 0.0f ? -INFINITY
                                : 0.69314718055994531f * (top + log2f(sum));
}

// The blocks' shares of the work.  Kept in shared memory and advanced by one
// warp while the others join states, two segments ahead, so that it takes no
// registers from the products and every warp can begin the next segment's
// copies before the current one's states are joined.
//
// Many units: all units' tiles, T::kUnitCost more for each, in one line that is
// cut into equal ranges, one per block.  Few units (a single sequence, say):
// each is cut evenly into parts of at most `most` tiles, one per block; with U
// units, total / (blocks - U) tiles per part give at most `blocks` parts.  About as
// many units as blocks, none much longer than the others: one block each.  A part or
// range always has a block: a unit's counter and partial states are joined when all
// its parts have come, so one part too many would spoil the workspace for later calls.
template <typename T>
struct Plan {
    unsigned total, ranges;
    unsigned most;          // units cut into equal parts: tiles per part; else 0
    unsigned size, longer;  // a range has `size` tiles, the first `longer` one more
    unsigned t, x, end;     // next tile in the line and in its unit; the range's end
    int b, head, r;
    int number;             // segments so far

    __device__ __forceinline__ unsigned begin(unsigned i) const {
        return i * size + min(i, longer);
    }
    __device__ __forceinline__ unsigned owner(unsigned t) const {
        const unsigned head = longer * (size + 1);
        return t < head ? t / (size + 1) : longer + (t - head) / size;
    }
    // what a unit of n tiles takes in the line
    __device__ __forceinline__ unsigned weight(int n) const {
        return most ? (n + most - 1) / most : n + (unsigned)T::kUnitCost;
    }
};

constexpr unsigned kMostTiles = 0x7fffffff;

__device__ __forceinline__ unsigned times(unsigned a, unsigned b) {
    return (unsigned)min((unsigned long long)a * b, (unsigned long long)kMostTiles);
}

__device__ __forceinline__ unsigned add_tiles(unsigned a, unsigned b) {
    return min(a + b, kMostTiles);  // both at most kMostTiles
}

template <typename T, bool kFew>
class Scheduler {
    static constexpr int kRows = T::kRows, kUnitCost = T::kUnitCost, kMinTiles = T::kMinTiles;
    const AttentionArgs& a;
    Plan<T>* const plan;
    Seq* const seqs;
    Segment* const segments;  // three: the current, the next and the one after
    const int lane;

    __device__ __forceinline__ Keys keys_of(const Seq& s, int r) const {
        return unit_keys<T>(a, s.kv - s.len, s.len, r);
    }

    // What a sequence's units take in the line.
    __device__ __forceinline__ unsigned weight_of_units(const Plan<T>& p, const Seq& s,
                                                        int& longest) const {
        const int rt = row_tiles(a, s.len, kRows);
        unsigned n = 0;
#pragma unroll 1
        for (int r = 0; r < rt; ++r) {
            const int tiles = keys_of(s, r).tiles;
            longest = max(longest, tiles);
            n = add_tiles(n, p.weight(tiles));
        }
        return times(n, a.c.kv_heads);
    }

public:
    __device__ __forceinline__ Scheduler(const AttentionArgs& args, Plan<T>* p, Seq* s, Segment* out)
        : a(args), plan(p), seqs(s), segments(out), lane(threadIdx.x & 31) {}

    // Reads the sequences and cuts the work (one warp); the block's first segment
    // when there is one.  One warp's latency, so the fewest dependent steps.
    __device__ __forceinline__ bool start() {
        const int batch = a.bt.batch;
        Plan<T> p;
        p.most = kFew ? 1 : 0;  // first pass: tiles
        unsigned sum = 0, units = 0;
        int longest = 0;
#pragma unroll 1
        for (int b = lane; b < batch; b += 32) {
            const Kv8Seq k = kv8_seq(a.bt, b);
            if (k.bad) kv8_report(a.bt);
            const Seq s{k.q0, k.len, k.kv, 0};
            seqs[b] = s;
            sum = add_tiles(sum, weight_of_units(p, s, longest));
            units = add_tiles(units, times(row_tiles(a, s.len, kRows), a.c.kv_heads));
        }
        __syncwarp();
        // lanes' sums below 2^26 each cannot overflow the warp's
        if (__any_sync(0xffffffffu, sum >= 1u << 26 || units >= 1u << 26)) {
#pragma unroll 1
            for (int d = 16; d > 0; d >>= 1) {
                sum = add_tiles(sum, __shfl_xor_sync(0xffffffffu, sum, d));
                units = add_tiles(units, __shfl_xor_sync(0xffffffffu, units, d));
            }
        } else {
            sum = __reduce_add_sync(0xffffffffu, sum);
            units = __reduce_add_sync(0xffffffffu, units);
        }
        if (sum == kMostTiles) kv8_report(a.bt);  // more than the line can count
        if (sum == 0 || sum == kMostTiles) return false;
        // At most half of the blocks go to rounding.  The host has bounded the units by
        // the tokens; only a malformed list, whose sequences overlap, holds more of them,
        // and their parts would outnumber the blocks: no part of the batch is taken.
        // (Going over to the line instead costs every other call: one sequence of 1000
        // keys 8.4 us against 8.2.)
        if (kFew) {
            if (units > gridDim.x / 2) {
                kv8_report(a.bt);
                return false;
            }
            p.most = max((unsigned)kMinTiles, sum / (gridDim.x - units) + 1);
        }
        // a block per unit, where cutting the longest would cost more than it saves
        if (!kFew && units <= gridDim.x) {
            longest = __reduce_max_sync(0xffffffffu, longest);
            if ((unsigned)longest <= sum / gridDim.x) p.most = longest;
        }
        if (batch > 1 || p.most) {
            sum = 0;
#pragma unroll 1
            for (int b0 = 0; b0 < batch; b0 += 32) {
                const int b = b0 + lane;
                const unsigned n = b < batch ? weight_of_units(p, seqs[b], longest) : 0;
                unsigned upto = n;
                if (batch > 1)
#pragma unroll
                    for (int d = 1; d < 32; d <<= 1) {
                        const unsigned v = __shfl_up_sync(0xffffffffu, upto, d);
                        if (lane >= d) upto += v;
                    }
                if (b < batch) seqs[b].before = sum + upto - n;
                sum += __shfl_sync(0xffffffffu, upto, batch > 1 ? 31 : 0);
            }
        }
        __syncwarp();
        p.total = sum;
        p.ranges = p.most ? sum : min((sum + kMinTiles - 1) / kMinTiles, gridDim.x);
        if (blockIdx.x >= p.ranges) return false;
        p.size = p.total / p.ranges;
        p.longer = p.total - p.size * p.ranges;
        p.t = p.begin(blockIdx.x);
        p.end = p.begin(blockIdx.x + 1);
        // the sequence, row tile and head of tile t: the last sequence that
        // begins at or before it
        p.b = 0;
#pragma unroll 1
        for (int b0 = 0; b0 < batch; b0 += 32) {
            const unsigned m = __ballot_sync(0xffffffffu,
                                             b0 + lane < batch && seqs[b0 + lane].before <= p.t);
            if (m) p.b = b0 + 31 - __clz(m);
        }
        const Seq s = seqs[p.b];
        p.x = p.t - s.before;
        p.r = 0;
        unsigned one;
#pragma unroll 1
        for (;;) {  // a row tile's heads lie side by side in the line
            one = p.weight(keys_of(s, p.r).tiles);
            if (p.x < one * a.c.kv_heads) break;
            p.x -= one * a.c.kv_heads;
            ++p.r;
        }
        p.head = p.x / one;
        p.x -= p.head * one;
        p.number = 0;
        if (lane == 0) *plan = p;
        __syncwarp();
        next();
        return true;
    }

    // Writes the next segment, if there is one, and advances.
    __device__ __forceinline__ void next() {
        Plan<T> p = *plan;
        if (p.t >= p.end) return;
        Seq s = seqs[p.b];
        Segment g;
#pragma unroll 1
        do {
            g.keys = keys_of(s, p.r);
            g.b = p.b;
            g.q0 = s.q0;
            g.len = s.len;
            g.first = s.kv - s.len;
            g.head = p.head;
            g.r = p.r;
            const unsigned tiles = g.keys.tiles;
            const unsigned unit = p.t - p.x, all = p.weight(tiles);
            const unsigned take = min(all - p.x, p.end - p.t);
            unsigned c0, c1;
            if (p.most) {  // part x of `all` equal ones (take is 1)
                c0 = unit;
                c1 = c0 + all - 1;
                g.slot0 = 2 * c0;
                const unsigned each = tiles / all, more = tiles - each * all;
                g.x0 = p.x * each + min(p.x, more);
                g.x1 = g.x0 + each + (p.x < more ? 1 : 0);
            } else {
                g.x0 = max((int)p.x - kUnitCost, 0);
                g.x1 = (int)(p.x + take) - kUnitCost;
                // ranges that hold the unit's first and last tile
                const unsigned u0 = unit + kUnitCost, u1 = u0 + tiles - 1;
                c0 = u0 >= p.begin(blockIdx.x) ? blockIdx.x : p.owner(u0);
                c1 = u1 < p.end ? blockIdx.x : p.owner(u1);
                // a range's slots: of the unit it begins in, of the unit it ends in
                g.slot0 = 2 * c0 + (unit < p.begin(c0) ? 0 : 1);
            }
            g.slot = c0 == blockIdx.x ? g.slot0 : 2 * blockIdx.x;
            g.slot1 = 2 * c0 + 2;
            g.counter = c0;
            g.parts = (int)(c1 - c0) + 1;
            p.t += take;
            g.last = p.t >= p.end;
            p.x = 0;
            if (!g.last && ++p.head == a.c.kv_heads) {
                p.head = 0;
                if (++p.r >= row_tiles(a, s.len, kRows)) {
                    p.r = 0;
                    do s = seqs[++p.b];
                    while (s.len == 0);
                }
            }
            // a range may hold only the cost, not the tiles, of its last unit
        } while (g.x1 <= g.x0 && !g.last);
        const int at = p.number % 3;
        ++p.number;
        __syncwarp();
        if (lane == 0) {
            *plan = p;
            segments[at] = g;
        }
        __syncwarp();
    }
};

}  // namespace nvf
