// kv8_attention.cu -- attention of new tokens over the paged E4M3 cache.
//
// Query i of a sequence of n new tokens and length kv has position
// p = kv - n + i and sees key j <= p, and with a window W only j > p - W or
// j < sinks:
//   s_j = softmax_scale * k_scale * (q . k_code_j),  out = sum_j softmax(s)_j v_scale v_code_j
// lse = log(sum exp s).  A query that sees nothing gives 0 and -inf.
//
// What bounds it: the cache's bytes for one or a few new tokens (2 * head_dim
// bytes per key and kv head, 4 * rows flops per byte), so every byte of the
// cache is copied once per unit and the products run on the tensor cores.
//
// Unit: one sequence, one kv head and a tile of kRows rows (new tokens x the
// query heads that share the kv head).  A unit's visible keys form tiles of
// kTile keys.  All units' tiles, in order, are cut into one equal range per
// block (lengths are read on the device, so ragged batches balance and a
// captured graph follows them); the 8 warps of a block take a range's tiles in
// turn, each with its own ring of asynchronous copies and its own running
// softmax, and their states are joined in shared memory.  A unit that several
// blocks share is joined by the last of them to finish, in the order of the
// ranges, so results do not depend on timing.
//
// Products: keys (values' columns) are the 16-row operand and the new rows the
// 8-column one, m16n8k16 with f16 operands and f32 sums; E4M3 codes are exact
// in f16, q is scaled per row by a power of two into f16's range (as exact as
// bf16 down to 2^-28 of the row's largest value).  S^T = K q^T leaves a key's
// scores of two rows in a thread; P^T reaches the operand layout of
// O^T = V^T P^T by an 8x8 transpose (movmatrix).  The order of keys within 16
// and of the head's values is free, so each thread reads 16-byte pieces.
//
// Softmax with a scale per page: with t = log2(e) s + log2(v_scale), the
// weights are P = 2^(t - max t + 14), so O = sum P v_code needs no scale per
// key and l = sum P / v_scale restores the denominator.  P is rounded to f16
// (11 bits, kept normal down to 2^-28 of the largest); t, maxima, l and O are
// fp32.
//
// Measured (8 kv heads of 128 unless said): one sequence of 131071 keys, 8 rows per
// kv head, 49 us for 269 MB (5.4 TB/s; 7.0 while the tiles run, then about 4 us
// before the first, for lengths, cut and pages, and 5 after the last, for the
// slowest warp and the join); 32 sequences of 1000 to 16000 keys 66 us for 363 MB
// (5.5 TB/s); one of 1000 keys 8.2 us, which is those two ends.  From 9 rows on the
// work per tile of 16 keys, which grows with every 8 rows, shows (8 sequences of 8192
// keys, 134 MB: 29 us with 8 rows, 45 with 16, 70 with 24 and 32).
#include <atomic>

#include "kv8_schedule.cuh"

namespace nvf {

namespace {

constexpr float kBias = 14.0f;  // the largest weight is 2^14 in f16
constexpr int kTile = 16;  // keys per tile: within one page
constexpr int kMostBlocks = 320;

// Units of kRows rows in tiles of kTile keys; at least 16 tiles per block (one
// sequence of 1000 keys: 8.5 us; 9.6 with 4, 10.8 with 64), and a unit, or a piece
// of one, costs about 24 tiles beside its own (16 sequences of 4 new tokens, window
// 1024: 19.3 us, 23.3 with 8, 19.3 with 72; 32 sequences of 1000 to 16000 keys and
// one new token: 65.8, 66.8 and 68.1).
template <int kRows>
using Tiling = TilingOf<kRows, kTile, 16, 24>;

template <int kDim, int kNT, bool kFew>
struct Shape {
    static constexpr int kRows = 8 * kNT;
    // 16 warps per SM where the state leaves room for 128 registers: two blocks,
    // so that one's unit ends and begins under the other's products (the 32 sequences
    // above 65 us, in one block of 16 warps 70), or, when few units are cut into many
    // parts, one block, which halves the parts.  Where q's fragments and the state do
    // not fit together, q is read from shared memory (64 sequences of 2000 keys, 16
    // rows: 82 us against 88 in 8 warps with q in registers).
    static constexpr bool kNarrow = kNT * kDim <= 256 && kDim <= 128;
    static constexpr bool kQInRegs = kNarrow ? kNT == 1 : kNT * kDim <= 256;  // else shared
    static constexpr int kBlocks = kNarrow && !kFew ? 2 : 1;
    static constexpr int kWarps = kNarrow && kFew ? 16 : 8;
    static constexpr int kThreads = kWarps * 32;
    static constexpr int kStages = kDim == 64 || (kDim == 128 && !kNarrow) ? 6 : 3;
    static constexpr int kStageBytes = 2 * kTile * kDim;
    static constexpr int kSteps = kDim / 16;  // k16 steps of q . k, m16 tiles of the head
    // shared memory: ring, page scales of each stage, q fragments, row scales,
    // warps' maxima and sums
    static constexpr int kScalesAt = kWarps * kStages * kStageBytes;
    static constexpr int kQAt = kScalesAt + kWarps * kStages * 8;
    static constexpr int kRowScaleAt = kQAt + kNT * kSteps * 32 * 8;
    static constexpr int kMaxAt = kRowScaleAt + kRows * 4;
    static constexpr int kSumAt = kMaxAt + kWarps * kRows * 4;
    static constexpr int kSeqsAt = kSumAt + kWarps * kRows * 4;
    // then a Seq per sequence
    // fp32 words of one partial state: O, maxima, sums
    static constexpr int kPartial = kRows * kDim + 2 * kRows;
    // a warp's state takes the first kNT stages of its ring
    static_assert(kRows * kDim * 4 == kNT * kStageBytes && kNT < kStages, "state and ring");
    // float index of value d of a state's row: the XOR spreads the rows that one
    // store touches over the banks and keeps 8 values together
    static __device__ __forceinline__ int state_at(int row, int d) {
        return row * kDim + (d ^ ((row & 6) << 2));
    }
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, bool full) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src),
                 "r"(full ? 4 : 0)
                 : "memory");
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

__device__ __forceinline__ uint2 lds64(uint32_t at) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at) : "memory");
    return v;
}

__device__ __forceinline__ float lds32(uint32_t at) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
    return v;
}

// Byte offset of 16-byte piece `piece` of row `row` in a tile: rows of 128 or
// 256 bytes XOR the low piece bits with the row; two 64-byte rows share a line
// of 128.  With the orders of keys and values below, the 8 (or 16) lanes of
// one access phase then touch all 32 banks once.
template <int kDim>
__device__ __forceinline__ uint32_t piece_at(int row, int piece) {
    if constexpr (kDim == 64) {
        const int line = row >> 1;
        const int p = (((row & 1) << 2) | piece) ^ (((line & 1) << 1) | ((line & 2) << 1));
        return line * 128 + p * 16;
    } else {
        return row * kDim + ((piece & ~7) | ((piece ^ row) & 7)) * 16;
    }
}

template <int kDim, int kNT, bool kFew>
class Worker {
    using S = Shape<kDim, kNT, kFew>;
    static constexpr int kWarps = S::kWarps;
    static constexpr bool kQInRegs = S::kQInRegs;
    static constexpr int kWords = kDim / 32;  // 32-bit words of a value row that a lane holds

public:
    const AttentionArgs& a;
    const int lane, warp, g, c, tg;
    const uint32_t smem;
    const Segment* seg;  // in shared memory: read there, not held in registers
    // the state: column pairs (2c, 2c + 1) of each n8 tile
    float o[kNT][S::kSteps][4];
    float top[kNT][2], sum[kNT][2];
    uint2 qf[kQInRegs ? kNT : 1][kQInRegs ? S::kSteps : 1];
    float row_scale[kNT][2];
    int pages;   // lane l: the page (not yet checked) of the segment's tile number pages_at + l
    int pages_at;

    __device__ __forceinline__ Worker(const AttentionArgs& args, uint32_t base)
        : a(args), lane(threadIdx.x & 31), warp(threadIdx.x >> 5), g(lane >> 2), c(lane & 3),
          tg(((lane >> 2) & 1) << 2 | (lane >> 3)), smem(base) {}

    __device__ __forceinline__ static int tile_start(const Keys& k, int x) {
        return (x < k.sink_tiles ? x : k.lo / kTile + x - k.sink_tiles) * kTile;
    }

    // The table's entry for tile x; -2 where there is no key.
    __device__ __forceinline__ int page_of(const Segment& s, int x) const {
        const int j = tile_start(s.keys, x);
        if (x >= s.x1 || j >= s.keys.hi) return -2;
        return a.bt.page_table[(size_t)s.b * a.bt.table_width + (j >> a.bt.page_shift)];
    }

    // Where the lane's 16 bytes of a tile's it-th 512 bytes go: 8 rows of 128
    // bytes on the swizzle is the same again.
    __device__ __forceinline__ uint32_t copy_at(int it) const {
        constexpr int kPieces = kDim / 16, kPeriod = 8 * kDim / 512;
        const int piece = (it % kPeriod) * 32 + lane;
        return piece_at<kDim>(piece / kPieces, piece % kPieces) + it / kPeriod * kPeriod * 512;
    }

    // Starts the copy of tile x, the warp's number-th of the segment.
    __device__ __forceinline__ void issue(int x, int number, int stage) {
        if (x < seg->x1) {
            if (number - pages_at == 32) {
                pages = page_of(*seg, x + lane * kWarps);
                pages_at = number;
            }
            const int entry = __shfl_sync(0xffffffffu, pages, number - pages_at);
            const bool ok = entry >= 0 && entry < a.c.pages;
            if (!ok && entry != -2) kv8_report(a.bt);
            const uint32_t dst = smem + (warp * S::kStages + stage) * S::kStageBytes;
            const Keys& keys = seg->keys;
            const int j0 = tile_start(keys, x);
            const size_t at = (size_t)(ok ? entry : 0) * a.c.kv_heads + seg->head;
            const size_t from =
                ((at << a.bt.page_shift) + (j0 & ((1 << a.bt.page_shift) - 1))) * kDim + lane * 16;
            const uint8_t* const k = a.c.k_codes + from;
            const uint8_t* const v = a.c.v_codes + from;
            constexpr int kPieces = kDim / 16;
            if (ok && j0 + kTile <= keys.hi && (j0 >= keys.lo || j0 + kTile <= a.sinks)) {
#pragma unroll
                for (int it = 0; it < kPieces / 2; ++it) {
                    const uint32_t to = dst + copy_at(it);
                    cp_async16(to, k + it * 512);
                    cp_async16(to + kTile * kDim, v + it * 512);
                }
            } else {
                // keys that no row sees are filled with zeros
#pragma unroll
                for (int it = 0; it < kPieces / 2; ++it) {
                    const int j = j0 + (it * 32 + lane) / kPieces;
                    const bool live =
                        ok && j < keys.hi && (j >= keys.lo || j < a.sinks);
                    const uint32_t to = dst + copy_at(it);
                    cp_async16_or_zero(to, live ? k + it * 512 : a.c.k_codes, live);
                    cp_async16_or_zero(to + kTile * kDim, live ? v + it * 512 : a.c.v_codes, live);
                }
            }
            if (lane < 2) {
                const uint32_t to =
                    smem + S::kScalesAt + (warp * S::kStages + stage) * 8 + lane * 4;
                cp_async4(to, (lane ? a.c.v_scales : a.c.k_scales) + at, ok);
            }
        }
        cp_async_commit();
    }

    // Lane (g, c)'s share of row g of n-tile nt of q: values 16 (c + 4h) .. + 15.
    struct QRow {
        uint4 w[kDim / 64][2];
    };

    __device__ __forceinline__ QRow load_q(int nt) const {
        const int row = seg->r * S::kRows + nt * 8 + g;
        const int i = token_of(a, row);
        const bool live = i < seg->len;
        const __nv_bfloat16* src =
            a.q + (long long)(seg->q0 + (live ? i : 0)) * a.q_stride +
            (size_t)(seg->head * a.group + (live ? row - i * a.group : 0)) * kDim;
        QRow q;
#pragma unroll
        for (int h = 0; h < kDim / 64; ++h)
#pragma unroll
            for (int e = 0; e < 2; ++e)
                q.w[h][e] = live ? reinterpret_cast<const uint4*>(src + 16 * (c + 4 * h))[e]
                                 : make_uint4(0, 0, 0, 0);
        return q;
    }

    // Scales the row by a power of two into f16 operand fragments (lane's values
    // 16 (c + 4h) + 4j + 0..3 for step 4h + j); returns the scale of its scores.
    __device__ __forceinline__ float make_fragments(const QRow& q, uint2 (&f)[S::kSteps]) const {
        float big = 0.0f;
#pragma unroll
        for (int h = 0; h < kDim / 64; ++h)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint32_t w[4] = {q.w[h][e].x, q.w[h][e].y, q.w[h][e].z, q.w[h][e].w};
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    big = fmaxf(big, fmaxf(fabsf(bf16_lo(w[i])), fabsf(bf16_hi(w[i]))));
            }
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
        // 2^e brings the row's largest value into [2^14, 2^15)
        const int e = min(14 + 127 - (int)(__float_as_uint(big) >> 23), 126);
        const float up = __uint_as_float((uint32_t)(e + 127) << 23);
#pragma unroll
        for (int h = 0; h < kDim / 64; ++h)
#pragma unroll
            for (int e2 = 0; e2 < 2; ++e2) {
                const uint32_t w[4] = {q.w[h][e2].x, q.w[h][e2].y, q.w[h][e2].z, q.w[h][e2].w};
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    f[4 * h + 2 * e2 + i] =
                        make_uint2(f16x2(bf16_lo(w[2 * i]) * up, bf16_hi(w[2 * i]) * up),
                                   f16x2(bf16_lo(w[2 * i + 1]) * up, bf16_hi(w[2 * i + 1]) * up));
            }
        return a.scale * __uint_as_float((uint32_t)(127 - e) << 23);
    }

    // Fragments of n-tile nt into shared memory (where registers do not hold
    // all rows'), by one warp.
    __device__ __forceinline__ void stage_q(int nt) {
        uint2 f[S::kSteps];
        const float scale = make_fragments(load_q(nt), f);
#pragma unroll
        for (int k = 0; k < S::kSteps; ++k)
            asm volatile("st.shared.v2.u32 [%0], {%1,%2};" ::"r"(
                             smem + S::kQAt + (nt * S::kSteps + k) * 256 + lane * 8),
                         "r"(f[k].x), "r"(f[k].y)
                         : "memory");
        if (c == 0)
            asm volatile("st.shared.f32 [%0], %1;" ::"r"(smem + S::kRowScaleAt + (nt * 8 + g) * 4),
                         "f"(scale)
                         : "memory");
    }

    __device__ __forceinline__ void begin() {
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                top[nt][e] = -INFINITY;
                sum[nt][e] = 0.0f;
#pragma unroll
                for (int m = 0; m < S::kSteps; ++m) o[nt][m][e] = o[nt][m][e + 2] = 0.0f;
            }
    }

    // Rows' scales from the lanes (or shared memory) that hold them to the
    // column pairs of the scores.
    __device__ __forceinline__ void take_q(const QRow (&q)[kQInRegs ? kNT : 1]) {
        if constexpr (kQInRegs) {
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt) {
                const float v = make_fragments(q[nt], qf[nt]);
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    row_scale[nt][e] = __shfl_sync(0xffffffffu, v, 8 * c + 4 * e);
            }
        } else {
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    row_scale[nt][e] = lds32(smem + S::kRowScaleAt + (nt * 8 + 2 * c + e) * 4);
        }
    }

    __device__ __forceinline__ uint2 q_fragment(int nt, int k) const {
        if constexpr (kQInRegs)
            return qf[nt][k];
        else
            return lds64(smem + S::kQAt + (nt * S::kSteps + k) * 256 + lane * 8);
    }

    // Whether row column e of n-tile nt sees key j.
    __device__ __forceinline__ bool sees(int nt, int e, int j, bool page_ok) const {
        const int i = token_of(a, seg->r * S::kRows + nt * 8 + 2 * c + e);
        const int hi = seg->first + i + 1;
        const int lo = window_start(a, hi);
        return page_ok && i < seg->len && j < hi && (j >= lo || j < a.sinks);
    }

    // V^T fragments (values g and g + 8 of m16 tiles 2i and 2i + 1) of four keys'
    // words x0..x3, times P^T.
    template <bool kSecond>
    __device__ __forceinline__ static void v_fragment(uint32_t x0, uint32_t x1, uint32_t x2,
                                                      uint32_t x3, uint32_t (&f)[4]) {
        const uint32_t lo = prmt(x0, x1, kSecond ? 0x7362 : 0x5140);
        const uint32_t hi = prmt(x2, x3, kSecond ? 0x7362 : 0x5140);
        f[0] = e4m3x2_to_f16x2(lo);
        f[1] = e4m3x2_hi_to_f16x2(lo);
        f[2] = e4m3x2_to_f16x2(hi);
        f[3] = e4m3x2_hi_to_f16x2(hi);
    }

    // O^T += V^T P^T.  guard: some row does not see some
    // key of the tile; a NaN value then must not reach it through 0 * NaN, so
    // NaNs are taken out of the product and put into the rows that see them.
    __device__ __forceinline__ void accumulate(uint32_t v_at, const uint32_t (&p)[kNT][2],
                                               bool guard, int j0, bool page_ok) {
        uint32_t w[4][kWords];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int row = 4 * k + c;
            if constexpr (kDim == 64) {
                const uint2 x = lds64(v_at + piece_at<64>(row, g >> 1) + (g & 1) * 8);
                w[k][0] = x.x, w[k][1] = x.y;
            } else {
#pragma unroll
                for (int u = 0; u < kDim / 128; ++u) {
                    const uint4 x = lds128(v_at + piece_at<kDim>(row, tg + 8 * u));
                    w[k][4 * u] = x.x, w[k][4 * u + 1] = x.y;
                    w[k][4 * u + 2] = x.z, w[k][4 * u + 3] = x.w;
                }
            }
        }
        if (guard) {
            uint32_t any = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int i = 0; i < kWords; ++i) any |= nan_bytes(w[k][i]);
            if (__any_sync(0xffffffffu, any != 0)) {
                // 1 where a row sees a key
                uint32_t see[kNT][2];
#pragma unroll
                for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int j = j0 + tg + 8 * e;
                        see[nt][e] = transpose8x8(f16x2(sees(nt, 0, j, page_ok) ? 1.0f : 0.0f,
                                                        sees(nt, 1, j, page_ok) ? 1.0f : 0.0f));
                    }
#pragma unroll
                for (int i = 0; i < kWords; ++i) {
                    uint32_t x[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t bad = nan_bytes(w[k][i]) >> 7;
                        w[k][i] &= ~(bad * 0xffu);
                        x[k] = bad * 0x38u;  // E4M3's 1
                    }
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        uint32_t f[4];
                        if (half)
                            v_fragment<true>(x[0], x[1], x[2], x[3], f);
                        else
                            v_fragment<false>(x[0], x[1], x[2], x[3], f);
#pragma unroll
                        for (int nt = 0; nt < kNT; ++nt) {
                            float seen[4];
                            mma_f16_16816_zero(seen, f[0], f[1], f[2], f[3], see[nt][0],
                                               see[nt][1]);
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (seen[e] > 0.0f) o[nt][2 * i + half][e] = NAN;
                        }
                    }
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            uint32_t f[4];
            v_fragment<false>(w[0][i], w[1][i], w[2][i], w[3][i], f);
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt)
                mma_f16_16816(o[nt][2 * i], f[0], f[1], f[2], f[3], p[nt][0], p[nt][1]);
            v_fragment<true>(w[0][i], w[1][i], w[2][i], w[3][i], f);
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt)
                mma_f16_16816(o[nt][2 * i + 1], f[0], f[1], f[2], f[3], p[nt][0], p[nt][1]);
        }
    }

    __device__ __forceinline__ void consume(int x, int stage) {
        const uint32_t k_at = smem + (warp * S::kStages + stage) * S::kStageBytes;
        const uint32_t v_at = k_at + kTile * kDim;
        const uint32_t scales = smem + S::kScalesAt + (warp * S::kStages + stage) * 8;
        const Keys& keys = seg->keys;
        const int j0 = tile_start(keys, x);
        const float ks = lds32(scales);
        float vs = lds32(scales + 4);
        const bool page_ok = vs > 0.0f;  // copied as 0 without a page
        const bool guard = !page_ok || j0 + kTile > keys.hi_min ||
                           (j0 < keys.lo_max && j0 + kTile > a.sinks);
        vs = usable_scale(vs);
        float s[kNT][4];
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[nt][e] = 0.0f;
#pragma unroll
        for (int h = 0; h < kDim / 64; ++h) {
            const uint4 x = lds128(k_at + piece_at<kDim>(tg, c + 4 * h));
            const uint4 y = lds128(k_at + piece_at<kDim>(tg + 8, c + 4 * h));
            const uint32_t wx[4] = {x.x, x.y, x.z, x.w}, wy[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t a0 = e4m3x2_to_f16x2(wx[j]), a2 = e4m3x2_hi_to_f16x2(wx[j]);
                const uint32_t a1 = e4m3x2_to_f16x2(wy[j]), a3 = e4m3x2_hi_to_f16x2(wy[j]);
#pragma unroll
                for (int nt = 0; nt < kNT; ++nt) {
                    const uint2 q = q_fragment(nt, 4 * h + j);
                    mma_f16_16816(s[nt], a0, a1, a2, a3, q.x, q.y);
                }
            }
        }
        // t = log2(e) s + log2(v_scale), maxima over the keys
        const float lv = __log2f(vs);
        bool grown = false;
        float most[kNT][2];
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float t = fmaf(s[nt][e], row_scale[nt][e & 1] * ks, lv);
                if (guard && !sees(nt, e & 1, j0 + tg + 8 * (e >> 1), page_ok)) t = -INFINITY;
                s[nt][e] = t;
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float v = fmaxf(s[nt][e], s[nt][e + 2]);
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
                grown |= v > top[nt][e];
                most[nt][e] = fmaxf(v, top[nt][e]);
            }
        }
        if (__any_sync(0xffffffffu, grown)) {
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float keep =
                        most[nt][e] == -INFINITY ? 1.0f : exp2_fast(top[nt][e] - most[nt][e]);
                    top[nt][e] = most[nt][e];
                    sum[nt][e] *= keep;
#pragma unroll
                    for (int m = 0; m < S::kSteps; ++m) {
                        o[nt][m][e] *= keep;
                        o[nt][m][e + 2] *= keep;
                    }
                }
        }
        const float inv = __fdividef(1.0f, vs);
        uint32_t p[kNT][2];
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) {
            float w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float base = top[nt][e & 1] == -INFINITY ? 0.0f : top[nt][e & 1];
                w[e] = exp2_fast(s[nt][e] - (base - kBias));
            }
            sum[nt][0] = fmaf(w[0] + w[2], inv, sum[nt][0]);
            sum[nt][1] = fmaf(w[1] + w[3], inv, sum[nt][1]);
            p[nt][0] = transpose8x8(f16x2(w[0], w[1]));
            p[nt][1] = transpose8x8(f16x2(w[2], w[3]));
        }
        accumulate(v_at, p, guard, j0, page_ok);
    }

    // The warp's state into its part of shared memory.
    __device__ __forceinline__ void put_state() {
        const uint32_t mine = smem + warp * S::kStages * S::kStageBytes;
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float v = sum[nt][e];
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
                const int row = nt * 8 + 2 * c + e;
                if (g == 0) {
                    const uint32_t at = smem + (warp * S::kRows + row) * 4;
                    asm volatile("st.shared.f32 [%0], %1;" ::"r"(at + S::kMaxAt), "f"(top[nt][e])
                                 : "memory");
                    asm volatile("st.shared.f32 [%0], %1;" ::"r"(at + S::kSumAt), "f"(v)
                                 : "memory");
                }
#pragma unroll
                for (int m = 0; m < S::kSteps; ++m) {
                    // value of the head: pairs within the lane's 16-byte (8-byte) pieces
                    const int d = kDim == 64 ? 8 * g + 2 * m
                                             : 16 * (tg + 8 * (m / 8)) + 2 * (m % 8);
                    asm volatile("st.shared.v2.f32 [%0], {%1,%2};" ::"r"(
                                     mine + S::state_at(row, d) * 4),
                                 "f"(o[nt][m][e]), "f"(o[nt][m][e + 2])
                                 : "memory");
                }
            }
    }
};

// Joins the partial states of the segment's unit, by a whole block.  Many
// parts' weights (one per part and row) and the thread groups' sums go to the
// rings' first stages, which hold nothing any more.
template <int kDim, int kNT, bool kFew>
__device__ __forceinline__ void join_parts(const AttentionArgs& a, const Segment& g,
                                           uint8_t* shared) {
    using S = Shape<kDim, kNT, kFew>;
    constexpr int kItems = S::kRows * kDim / 4;
    const int parts = g.parts, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const unsigned slot0 = g.slot0, slot1 = g.slot1;
    auto part = [&](int i) {
        return a.partials + (size_t)(i == 0 ? slot0 : slot1 + 2 * (i - 1)) * S::kPartial;
    };
    constexpr int kFewParts = 8;
    if (parts <= kFewParts) {
        // everything in one round of loads
        for (int item = threadIdx.x; item < kItems; item += S::kThreads) {
            const int row = item / (kDim / 4), d = item % (kDim / 4) * 4;
            float4 y[kFewParts];
            float tops[kFewParts], sums[kFewParts];
#pragma unroll
            for (int i = 0; i < kFewParts; ++i) {
                tops[i] = -INFINITY;
                sums[i] = 0.0f;
                y[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (i < parts) {
                    const float* p = part(i);
                    y[i] = __ldcg(reinterpret_cast<const float4*>(p + row * kDim + d));
                    tops[i] = __ldcg(p + S::kRows * kDim + row);
                    sums[i] = __ldcg(p + S::kRows * kDim + S::kRows + row);
                }
            }
            float top = -INFINITY, sum = 0.0f;
#pragma unroll
            for (int i = 0; i < kFewParts; ++i) top = fmaxf(top, tops[i]);
            float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int i = 0; i < kFewParts; ++i) {
                const float f = weight_of(tops[i], top);
                sum = fmaf(sums[i], f, sum);
                v.x = fmaf(y[i].x, f, v.x);
                v.y = fmaf(y[i].y, f, v.y);
                v.z = fmaf(y[i].z, f, v.z);
                v.w = fmaf(y[i].w, f, v.w);
            }
            store_row<kDim>(a, g.q0, g.len, g.head, g.r * S::kRows + row, d, v, top - kBias, sum);
        }
        return;
    }
    // each row's largest maximum and the parts' weights, a warp per row:
    // [part][row], in pieces of one warp's free stages
    constexpr int kPiece = kNT * S::kStageBytes / 4 / S::kRows;
    static_assert(kPiece * S::kWarps >= kMostBlocks, "a weight for every part");
    auto weight = [&](int i, int row) -> float& {
        return reinterpret_cast<float*>(shared + (i / kPiece) * S::kStages * S::kStageBytes)
            [(i % kPiece) * S::kRows + row];
    };
    float* const all = reinterpret_cast<float*>(shared + S::kSumAt);
    for (int row = warp; row < S::kRows; row += S::kWarps) {
        float top = -INFINITY;
        for (int i = lane; i < parts; i += 32) {
            const float v = __ldcg(part(i) + S::kRows * kDim + row);
            weight(i, row) = v;
            top = fmaxf(top, v);
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        float sum = 0.0f;
        for (int i = lane; i < parts; i += 32) {
            const float f = weight_of(weight(i, row), top);
            weight(i, row) = f;
            sum = fmaf(__ldcg(part(i) + S::kRows * kDim + S::kRows + row), f, sum);
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        if (lane == 0) {
            all[row] = sum;
            all[S::kRows + row] = top;
        }
    }
    __syncthreads();
    // groups of threads take every kGroups-th part
    constexpr int kGroups = S::kThreads > kItems ? S::kThreads / kItems : 1;
    const int group = kGroups > 1 ? threadIdx.x / kItems : 0;
    for (int item = kGroups > 1 ? threadIdx.x % kItems : threadIdx.x; item < kItems;
         item += S::kThreads) {
        const int row = item / (kDim / 4), d = item % (kDim / 4) * 4;
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
        for (int i = group; i < parts; i += kGroups) {
            const float4 y = __ldcg(reinterpret_cast<const float4*>(part(i) + row * kDim + d));
            const float f = weight(i, row);
            v.x = fmaf(y.x, f, v.x);
            v.y = fmaf(y.y, f, v.y);
            v.z = fmaf(y.z, f, v.z);
            v.w = fmaf(y.w, f, v.w);
        }
        if constexpr (kGroups > 1) {
            // the groups' sums, in order, through the last warps' free stages
            float4* const mine = reinterpret_cast<float4*>(
                shared + (S::kWarps - kGroups + group) * S::kStages * S::kStageBytes);
            static_assert(kItems * 16 <= kNT * S::kStageBytes &&
                              kPiece * (S::kWarps - kGroups) >= kMostBlocks, "room for both");
            mine[item] = v;
            __syncthreads();
            if (group > 0) break;
            v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int i = 0; i < kGroups; ++i) {
                const float4 y = reinterpret_cast<const float4*>(
                    shared + (S::kWarps - kGroups + i) * S::kStages * S::kStageBytes)[item];
                v.x += y.x;
                v.y += y.y;
                v.z += y.z;
                v.w += y.w;
            }
        }
        store_row<kDim>(a, g.q0, g.len, g.head, g.r * S::kRows + row, d, v,
                        all[S::kRows + row] - kBias, all[row]);
    }
}

template <int kDim, int kNT, bool kFew>
__global__ void __launch_bounds__(Shape<kDim, kNT, kFew>::kThreads,
                                  Shape<kDim, kNT, kFew>::kBlocks)
    kv8_attention_kernel(const AttentionArgs a) {
    using S = Shape<kDim, kNT, kFew>;
    constexpr int kWarps = S::kWarps, kThreads = S::kThreads;
    extern __shared__ __align__(128) uint8_t shared[];
    __shared__ Plan<Tiling<S::kRows>> plan;
    __shared__ Segment segments[3];
    __shared__ int work, joins;
    const int tid = threadIdx.x;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // the lists' first lines into L2 while the preceding kernel ends
    if (blockIdx.x == 0) {
        const int* const lists[2] = {a.bt.kv_len, a.bt.q_start};
        if (tid < 2) prefetch_l2(lists[tid]);
        const size_t entries = (size_t)a.bt.batch * a.bt.table_width;
        if ((size_t)tid * 32 < entries) prefetch_l2(a.bt.page_table + tid * 32);
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    Worker<kDim, kNT, kFew> w(a, smem_addr(shared));
    Seq* const seqs = reinterpret_cast<Seq*>(shared + S::kSeqsAt);
    Scheduler<Tiling<S::kRows>, kFew> scheduler(a, &plan, seqs, segments);
    if (w.warp == kWarps - 1) {
        const bool some = scheduler.start();
        if (w.lane == 0) work = some;
    }
    __syncthreads();
    if (!work) return;

    // the first copies of a segment go to the stages behind the state of the one
    // before it, which may still be waiting to be joined
    constexpr int kEarly = S::kStages - kNT < S::kStages - 1 ? S::kStages - kNT : S::kStages - 1;
    typename Worker<kDim, kNT, kFew>::QRow q[S::kQInRegs ? kNT : 1];
    int ahead_pages = -2;  // of the next segment's first tiles
    auto look_ahead = [&](const Segment& g) {
        ahead_pages = w.page_of(g, g.x0 + w.warp + w.lane * kWarps);
    };
    auto enter = [&](const Segment& g) {
        w.seg = &g;
        const int mine = g.x0 + w.warp;
        w.pages = ahead_pages;
        w.pages_at = 0;
        if constexpr (S::kQInRegs) {
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt) q[nt] = w.load_q(nt);
        }
#pragma unroll
        for (int i = 0; i < kEarly; ++i) w.issue(mine + i * kWarps, i, kNT + i);
    };
    look_ahead(segments[0]);
    enter(segments[0]);
    // the second segment, while the first one's copies are under way
    if (!segments[0].last) {
        if (w.warp == kWarps - 1) scheduler.next();
        __syncthreads();
    }
    for (int at = 0;; at = at == 2 ? 0 : at + 1) {
        const Segment& g = segments[at];
        const int x1 = g.x1, mine = g.x0 + w.warp;
        if (x1 <= g.x0) break;
        if (!g.last) look_ahead(segments[at == 2 ? 0 : at + 1]);
#pragma unroll
        for (int i = kEarly; i < S::kStages - 1; ++i)
            w.issue(mine + i * kWarps, i, (kNT + i) % S::kStages);
        if constexpr (!S::kQInRegs) {
            if (w.warp < kNT) w.stage_q(w.warp);
            __syncthreads();
        }
        w.begin();
        w.take_q(q);
        int stage = kNT, number = S::kStages - 1;
#pragma unroll 1
        for (int i = mine; i < x1; i += kWarps) {
            const int ahead = stage == 0 ? S::kStages - 1 : stage - 1;
            w.issue(i + (S::kStages - 1) * kWarps, number, ahead);
            ++number;
            cp_async_wait<S::kStages - 1>();
            __syncwarp();
            w.consume(i, stage);
            __syncwarp();
            stage = stage + 1 == S::kStages ? 0 : stage + 1;
        }
        cp_async_wait<0>();
        w.put_state();
        const bool last = g.last;
        if (!last) enter(segments[at == 2 ? 0 : at + 1]);
        __syncthreads();
        if (!last && w.warp == kWarps - 1) scheduler.next();

        // the warps' states joined, 4 values of one row per thread
        const int parts = g.parts;
        const float* tops = reinterpret_cast<const float*>(shared + S::kMaxAt);
        const float* sums = reinterpret_cast<const float*>(shared + S::kSumAt);
        float* const mine_out = a.partials + (size_t)g.slot * S::kPartial;
        for (int item = tid; item < S::kRows * kDim / 4; item += kThreads) {
            const int row = item / (kDim / 4), d = item % (kDim / 4) * 4;
            float top = -INFINITY;
#pragma unroll
            for (int i = 0; i < kWarps; ++i) top = fmaxf(top, tops[i * S::kRows + row]);
            float sum = 0.0f;
            float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int i = 0; i < kWarps; ++i) {
                const float f = weight_of(tops[i * S::kRows + row], top);
                const float4 y = *reinterpret_cast<const float4*>(
                    shared + i * S::kStages * S::kStageBytes + S::state_at(row, d) * 4);
                sum = fmaf(sums[i * S::kRows + row], f, sum);
                v.x = fmaf(y.x, f, v.x);
                v.y = fmaf(y.y, f, v.y);
                v.z = fmaf(y.z, f, v.z);
                v.w = fmaf(y.w, f, v.w);
            }
            if (parts == 1) {
                store_row<kDim>(a, g.q0, g.len, g.head, g.r * S::kRows + row, d, v, top - kBias, sum);
            } else {
                *reinterpret_cast<float4*>(mine_out + row * kDim + d) = v;
                if (d == 0) {
                    mine_out[S::kRows * kDim + row] = top;
                    mine_out[S::kRows * kDim + S::kRows + row] = sum;
                }
            }
        }
        if (parts > 1) {
            __syncthreads();
            if (tid == 0) {
                const int seen = atom_add_acq_rel_gpu(a.counters + g.counter, 1);
                joins = seen == parts - 1;
                if (joins) a.counters[g.counter] = 0;
            }
            __syncthreads();
            if (joins) join_parts<kDim, kNT, kFew>(a, g, shared);
        }
        if (last) break;
        __syncthreads();  // the states' memory becomes the ring again
    }
    cp_async_wait<0>();
}

template <int kDim, int kNT, bool kFew>
cudaError_t launch_as(const AttentionArgs& a, int num_sms, cudaStream_t s) {
    using S = Shape<kDim, kNT, kFew>;
    static std::atomic<bool> allowed[64];  // per device: the kernel's shared memory limit is set
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !allowed[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(kv8_attention_kernel<kDim, kNT, kFew>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 S::kSeqsAt + kKv8MaxBatch * (int)sizeof(Seq));
        if (e != cudaSuccess) return e;
        if (dev < 64) allowed[dev].store(true, std::memory_order_release);
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(min(num_sms * S::kBlocks, kMostBlocks));
    cfg.blockDim = dim3(S::kThreads);
    cfg.dynamicSmemBytes = S::kSeqsAt + a.bt.batch * sizeof(Seq);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kv8_attention_kernel<kDim, kNT, kFew>, a);
}

// Few units (row tiles times kv heads of all sequences) are cut into equal parts,
// which takes at least two blocks per unit (heads of 128, 8 of them: one sequence of
// 131071 keys 49.8 us against 54.1 in one line of tiles, 8 of 8192 keys 28.9 against
// 31.8, 4 of 20000 keys and two new tokens 53.1 against 52.2).
template <int kDim, int kNT>
cudaError_t launch(const AttentionArgs& a, int num_sms, cudaStream_t s) {
    constexpr int kRows = 8 * kNT;
    const long long rows = (long long)a.bt.tokens * a.group;
    // a sequence's rows are a multiple of the group: so much its last tile can lack
    const int lack = kRows - min(kRows, a.group & -a.group);
    const long long most = (rows + (long long)a.bt.batch * lack) / kRows * a.c.kv_heads;
    return most <= num_sms / 2 ? launch_as<kDim, kNT, true>(a, num_sms, s)
                               : launch_as<kDim, kNT, false>(a, num_sms, s);
}

}  // namespace

size_t kv8_attention_data_bytes(int head_dim, long long tokens, int group, int batch,
                                int num_sms) {
    if (kv8_prompt_applies(head_dim, tokens, group, batch))
        return kv8_prompt_data_bytes(head_dim, num_sms);
    // two partial states per block; the most rows that an SM's blocks hold: two
    // blocks of 32 rows of 64 values, two of 16 or one of 32 rows of 128, one of 16
    // of 256
    const size_t rows = head_dim == 64 ? 64 : head_dim == 128 ? 32 : 16;
    return (size_t)num_sms * 2 * rows * (head_dim + 2) * sizeof(float);
}

cudaError_t launch_kv8_attention(const void* q, long long q_stride, int heads,
                                 const Kv8CacheArgs& c, const Kv8BatchArgs& bt,
                                 float softmax_scale, int window, int sinks, void* out, float* lse,
                                 int* status, int* counters, void* partials, int num_sms,
                                 cudaStream_t s) {
    AttentionArgs a;
    a.c = c;
    a.bt = bt;
    a.q = reinterpret_cast<const __nv_bfloat16*>(q);
    a.out = reinterpret_cast<__nv_bfloat16*>(out);
    a.lse = lse;
    a.counters = counters;
    a.partials = reinterpret_cast<float*>(partials);
    a.q_stride = q_stride;
    a.heads = heads;
    a.group = heads / c.kv_heads;
    a.group_inverse = a.group == 1 ? 0xffffffffu : (unsigned)((1ull << 32) / a.group);
    a.scale = softmax_scale * 1.4426950408889634f;
    a.window = window > 0 ? window : 0x7fffffff;
    a.sinks = sinks;
    if (kv8_prompt_applies(c.head_dim, bt.tokens, a.group, bt.batch))
        return launch_kv8_prompt(a, partials, status, num_sms, s);
    // rows that share a kv head, per sequence on average: the narrowest tile
    // that holds them reads the cache once
    const long long rows = ((long long)bt.tokens * a.group + bt.batch - 1) / bt.batch;
    if (c.head_dim == 64)
        return rows <= 8    ? launch<64, 1>(a, num_sms, s)
               : rows <= 16 ? launch<64, 2>(a, num_sms, s)
                            : launch<64, 4>(a, num_sms, s);
    if (c.head_dim == 128)
        return rows <= 8    ? launch<128, 1>(a, num_sms, s)
               : rows <= 16 ? launch<128, 2>(a, num_sms, s)
                            : launch<128, 4>(a, num_sms, s);
    return rows <= 8 ? launch<256, 1>(a, num_sms, s) : launch<256, 2>(a, num_sms, s);
}

}  // namespace nvf
