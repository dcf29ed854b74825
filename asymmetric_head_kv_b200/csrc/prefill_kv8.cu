// prefill_kv8.cu -- causal attention of a ragged batch of query rows over an 8-bit paged cache.
//
//   out[r, h] = sum_{j <= p_r} softmax_j(scale q[r, h] . k_j) v_j,   k_j = kc_j 2^ke_j,  v_j = vc_j 2^ve_j
//
// with p_r the row's position, kc, vc the e4m3 codes and ke, ve the exponents of their blocks.  A dense contraction,
// 2 (d_k + d_v) operations for every row, head and position, on tcgen05 kind::f16:
//
//  * One CTA takes 256 query rows of one request and head as two 128-row tiles that share every 64-position K/V tile
//    (128-position tiles, whose S cannot be double-buffered in TMEM: 766 us where these take 500).  Four warps turn a
//    tile's codes into f16 once for both: code * 2^(e - e_ref), with e_ref the tile's largest exponent, exactly.  (Feeding
//    codes to fp8 MMAs instead would split every softmax weight into e4m3 terms, five more instructions for each pair of
//    scores in the warps that bound this kernel; conversion costs the tile 12 instructions for 16 codes in warps that have
//    nothing else to do.)  K's e_ref goes into the scores' multiplier, V's into the weights' exponent.
//  * O is held relative to 2^R, R a row's running maximum of (a tile's largest score + its V e_ref), the row sum relative to
//    2^M, the largest score.  A tile whose exponents lie further apart (K: 2^15, beyond which f16 would round; V: 2^8,
//    since R may be that much above every real weight) is `mixed`: codes are converted as they are, and the softmax
//    applies each position's exponents, in fp32, with an exponential more a score.
//  * Queries are scaled by a power of two per row into f16's range (8 significant bits fit its 11).
//  * Softmax: two threads a row, 32 columns each, so that four warps a scheduler hide one another's latencies; S is
//    double-buffered in TMEM, P (f16) goes back over S and is the A operand of P.V; O is rescaled in TMEM only when a
//    row's R grows by 2^8.  Weights are held at 2^7 of the reference, so that f16 resolves 2^-31 of it, and of the largest
//    weight 2^-23 at least; their sum is fp32, of the unrounded weights.
//  * A weight of zero times a NaN is NaN, so a NaN code of V would reach rows before it in the tiles on the diagonal.  There the
//    warp that fetches the scales looks the codes over before it hands the tile on, puts zeros in the place of NaN and notes
//    each column's first one; the rows from that position on get their NaN with the output.  (Two prompts of 8192: 491 us
//    without, 493 so; 542 with the look at the codes inline, 523 with it in the conversion warps, 510 in a warp of its own.)
//  * MMA, commit and TMA are issued by an elected lane (kv8.cuh).
//  * Rows of Q come in, and rows of the output go out, with a row's 16-byte pieces in neighbouring lanes.
//  * Units are taken longest first.  Where they are fewer than half of the SMs, each is cut into pieces of equal length, one
//    CTA each; records in the workspace, merged by the last CTA of the unit: 256 rows over 131072 positions, 16 heads, in
//    266 us with 9 pieces a unit, 527 with 4.
//    Equal shares of all the work on persistent CTAs were slower, 739 us against 500 for two prompts of 8192: each
//    further unit of a CTA costs about 10 us of pipeline, and the softmax loop inside a loop over units lacks registers.
// What bounds it: the softmax warps, 64 exponentials a row and tile (16 a clock and SM: half of the tile's 1900 clocks) and
// their latencies.  Two prompts of 8192, 16 heads of 64/128: 488 us, 845 TFLOP/s, 0.50 of the measured GEMM peak (tensor
// pipe 40% busy, XU 56%, 62% of issue slots); four requests of 17 rows over 1003 positions: 20.5 us, of which about 14 are
// one CTA's start and end.
#include <cuda_fp16.h>
#include <math.h>

#include <algorithm>
#include <numeric>

#include "internal.h"
#include "kv8.cuh"

namespace diffqkv {

namespace {

constexpr int BM = 128, QT = 2, BN = 64, DV_MAX = 128;
constexpr int kRows = QT * BM;
constexpr int kSoftmaxWarps = 8 * QT;  // two warps per 32 rows, 32 columns of S each
constexpr int kLoadWarp = 16, kMmaWarp = 17, kScaleWarp = 18, kConvWarp0 = 19, kConvWarps = 4;
constexpr int kThreads = 32 * (kConvWarp0 + kConvWarps);
constexpr int kRaw = 4;         // stages of codes
constexpr int kScaleSlots = 8;  // tiles of scales, fetched four at a time
constexpr int kExpSlots = 16;   // tiles of exponents that the softmax may still read
constexpr int kSlots = 160;     // partial records of the workspace: one for each piece of a call whose units are cut
constexpr int kCutBatch = 32;   // requests, at most, of a call whose units are cut
constexpr float kRescale = 8.f;  // growth (log2) of R before O is rescaled: weights stay below 2^(kShift + kRescale), inside f16
constexpr float kShift = 7.f;    // weights are held at 2^kShift of the reference
constexpr float kGrow = 40.f;    // growth of the largest score before the row sum is rescaled, where R does not ask for it
constexpr float kFloor = 80.f;   // weights of a tile whose V is this far below the row's: 2^(kShift + kGrow - kFloor) at most,
                                 // zero in f16, and still normal in fp32, for the row sum, down to 2^-53 of the largest
constexpr int kSpreadK = 15, kSpreadV = 8;  // of a tile's exponents, above which it is mixed
constexpr float kMixed = 0x1p120f;          // stands for V's e_ref of such a tile: above every R, so that the vote is for it

struct PreArgs {
    const __nv_bfloat16 *q;
    const uint8_t *k_scales, *v_scales;
    const int32_t *query_start, *block_table, *seq_lens;
    __nv_bfloat16 *out;
    float *partials;
    uint32_t *counters;
    int32_t *status;
    int32_t batch, n_q, n_k, n_v, tokens, t_max, max_blocks;
    int32_t page_size, page_shift, num_pages, sb, sub_rows, sub_shift;
    int32_t max_pieces;  // of a call whose units are cut, 0: they are not
    long long scale_blocks;
    float scale_log2;
    uint64_t wait_limit_ns;
};

__device__ __forceinline__ int div_page(const PreArgs &a, int x) {
    return a.page_shift >= 0 ? x >> a.page_shift : x / a.page_size;
}
__device__ __forceinline__ int clamp_to(int v, int hi) { return min(max(v, 0), hi); }

// Rows of request b: first row of q and their number, both inside [0, tokens].
__device__ __forceinline__ int2 request_rows(const PreArgs &a, int b) {
    const int s = clamp_to(__ldg(a.query_start + b), a.tokens), e = clamp_to(__ldg(a.query_start + b + 1), a.tokens);
    return make_int2(s, max(0, e - s));
}

// mbar_wait_bounded with what follows a failed first try out of line: a dozen copies of that loop among the roles' code cost
// two prompts of 8192 3% (504 against 491 us).  The TMA producer keeps it inline: five rows over 131072 positions, which its
// requests bound, take 171 us so and 191 without.
__device__ __noinline__ bool wait_on(uint32_t a, uint32_t parity, uint64_t limit_ns, volatile int *abort_flag, int32_t *status) {
    if (abort_flag && *abort_flag) return false;
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t n = 1;; ++n) {
        if (mbar_try_wait(a, parity)) return true;
        if ((n & 63u) == 0) {
            if (abort_flag && *abort_flag) return false;
            if (globaltimer_ns() - t0 > limit_ns) {
                if (abort_flag) *abort_flag = 1;
                record_error(status, DIFFQKV_ERR_DEVICE_TIMEOUT);
                return false;
            }
        }
    }
}
__device__ __forceinline__ bool wait_for(uint64_t *bar, uint32_t parity, uint64_t limit_ns, volatile int *abort_flag,
                                         int32_t *status) {
    const uint32_t a = smem_addr(bar);
    return mbar_try_wait(a, parity) || wait_on(a, parity, limit_ns, abort_flag, status);
}

template <int DK, int DV>
struct Cfg {
    static constexpr int Q_BYTES = BM * DK * 2;       // one query tile
    static constexpr int RAW_K = BN * DK, RAW_V = BN * DV, RAW = RAW_K + RAW_V;
    static constexpr int K_BYTES = 2 * RAW_K, V_BYTES = 2 * RAW_V, CONV = K_BYTES + V_BYTES;
    static constexpr int STAGES = DK == 64 ? 3 : 2;   // converted tiles
    static constexpr int REC = kRows * (DV + 2);      // floats of a partial record
    static constexpr int OFF_CONV = QT * Q_BYTES;
    static constexpr int OFF_RAW = OFF_CONV + STAGES * CONV;
    static constexpr int OFF_MISC = OFF_RAW + kRaw * RAW;
};

struct Misc {
    uint64_t raw_full[kRaw], raw_empty[kRaw], cv_full[3], cv_empty[3], sc_full[kScaleSlots], sc_empty[kScaleSlots];
    uint64_t q_full, s_full[QT][2], p_full[QT][2], pv_done[QT][2], mma_done;
    uint32_t k_mul[kScaleSlots][BN], v_mul[kScaleSlots][BN];  // 2^(e - e_ref) as f16 pairs, 0 behind the sequence
    float2 scale_ref[kScaleSlots];  // 2^(e_ref) of K and e_ref of V, or kMixed
    float2 ref[4];                  // the same for the softmax, tile k in slot k & 3
    // K's and V's exponents of mixed tiles, tile k in slot k % kExpSlots.  (Tile k's are written when k - kScaleSlots
    // has been converted, and so at least k - kScaleSlots - 3 been multiplied.)
    alignas(16) char2 exps[kExpSlots][BN];
    float row_s[QT][2][BM], row_y[QT][2][BM];                 // exchange between the two halves of a row
    int nan_pos[DV_MAX], nan_seen;  // first position with a NaN of each column of V, on the diagonal; whether there is one
    int found[8];  // unit: request, block, q row, rows, length; its pieces, which of them, its first record
    uint32_t tmem_slot;
    int abort_flag, last_flag;
};

constexpr uint32_t idesc_f16(int M, int N, bool b_mn_major) {
    return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t x, uint32_t m) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(m));
    return r;
}

// Sixteen codes -> sixteen f16 values times m, as two 16-byte chunks.
__device__ __forceinline__ void widen16(const uint4 &c, uint32_t m, uint4 &lo, uint4 &hi) {
    lo.x = mul_f16x2(e4m3x2_to_f16x2(c.x & 0xffffu), m);
    lo.y = mul_f16x2(e4m3x2_to_f16x2(c.x >> 16), m);
    lo.z = mul_f16x2(e4m3x2_to_f16x2(c.y & 0xffffu), m);
    lo.w = mul_f16x2(e4m3x2_to_f16x2(c.y >> 16), m);
    hi.x = mul_f16x2(e4m3x2_to_f16x2(c.z & 0xffffu), m);
    hi.y = mul_f16x2(e4m3x2_to_f16x2(c.z >> 16), m);
    hi.z = mul_f16x2(e4m3x2_to_f16x2(c.w & 0xffffu), m);
    hi.w = mul_f16x2(e4m3x2_to_f16x2(c.w >> 16), m);
}

// Codes [64][D] -> f16 in 64-wide blocks [64 rows][128 bytes] with the 128-byte swizzle, by kConvWarps warps: a thread has
// the same 16 columns of every kStep-th row, so that its addresses are one base and constant steps.
template <int D>
struct Widen {
    static constexpr int LPR = D / 16;                       // 16-code pieces of a row
    static constexpr int kStep = 32 * kConvWarps / LPR;      // rows between a thread's pieces: a multiple of 8
    static constexpr int kRounds = BN / kStep;
    static_assert(kStep % 8 == 0 && BN % kStep == 0, "swizzle phase of a thread");
    uint32_t src, dst0, dst1, row;
    bool swap;
    __device__ explicit Widen(int tid) {
        const int piece = tid % LPR, chunk = piece * 2 & 7;
        row = tid / LPR;
        src = tid * 16;
        // the two blocks of a 128-wide row lie in the same banks: the second half's threads store their two chunks the
        // other way round
        swap = piece >= 4;
        const uint32_t at = (piece >> 2) * (BN * 128) + row * 128;
        dst0 = at + ((chunk + (swap ? 1 : 0)) ^ (row & 7)) * 16;
        dst1 = at + ((chunk + (swap ? 0 : 1)) ^ (row & 7)) * 16;
    }
    __device__ __forceinline__ void run(const uint8_t *raw, uint8_t *out, const uint32_t *mul, bool tail) const {
        uint4 c[kRounds];
        uint32_t m[kRounds];
#pragma unroll
        for (int i = 0; i < kRounds; ++i) {
            c[i] = lds128(raw + src + i * (kStep * D));
            m[i] = mul[row + i * kStep];
        }
        if (tail) {  // behind the sequence: whatever is there may be NaN
#pragma unroll
            for (int i = 0; i < kRounds; ++i)
                if (m[i] == 0u) c[i] = make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < kRounds; ++i) {
            uint4 lo, hi;
            widen16(c[i], m[i], lo, hi);
            *reinterpret_cast<uint4 *>(out + dst0 + i * (kStep * 128)) = swap ? hi : lo;
            *reinterpret_cast<uint4 *>(out + dst1 + i * (kStep * 128)) = swap ? lo : hi;
        }
    }
};

// NaN in a V tile of codes, rows of DV bytes, the first at position `pos` (one warp): zeros in their place, and their columns'
// least positions in `first`.
template <int DV>
__device__ __noinline__ void take_nans(uint8_t *tile, int pos, int lane, int *first, int *seen) {
    auto nan4 = [](uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; };  // (codes 0x7f and 0xff)
#pragma unroll 1
    for (int i = lane * 16; i < BN * DV; i += 4 * 32 * 16) {
        uint4 c[4];
        uint32_t any = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) c[k] = lds128(tile + i + k * (32 * 16));
#pragma unroll
        for (int k = 0; k < 4; ++k) any |= nan4(c[k].x) | nan4(c[k].y) | nan4(c[k].z) | nan4(c[k].w);
        if (!any) continue;
        *seen = 1;
#pragma unroll 1
        for (int e = 0; e < 64; ++e) {
            const int at = i + (e >> 4) * (32 * 16) + (e & 15);
            if ((tile[at] & 0x7f) != 0x7f) continue;
            tile[at] = 0;
            atomicMin(first + at % DV, pos + at / DV);
        }
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// Barrier of the two warps of `id`; true where the predicate holds in any of their threads.
__device__ __forceinline__ bool pair_any(int id, bool x) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %2, 0;\n\t"
        "barrier.cta.red.or.pred q, %1, 64, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(id), "r"((uint32_t)x)
        : "memory");
    return r != 0;
}

// Factor of a row's products with keys of scale k: scale * log2(e) * 2^(the query's exponent) * k.  (A zero would turn masked
// scores into NaN; NaN stays.)
__device__ __forceinline__ float score_factor(float sc_row, float k) {
    const float x = sc_row * k;
    return x < 0x1p-126f ? 0x1p-126f : x;
}

// Half of a row of a mixed tile: its 32 columns of S and their positions' exponents, the columns that the row sees (0 .. last),
// the row's factor.  Read eight columns at a time, twice, and out of line: in the softmax loop it took two prompts of 8192,
// none of whose tiles is mixed, from 496 to 569 us, out of line to 505.  (All tiles mixed: 2290 us.)
struct MixedHalf {
    uint32_t t_s;
    const char2 *exps;
    int last;
    float sc_row;
};
__device__ __forceinline__ void mixed_scores(const MixedHalf &x, int c, float (&s)[8], float (&ve)[8]) {
    uint32_t z[8];
    tmem_ld_cols<8>(x.t_s + (uint32_t)c, z);
    tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const char2 ex = x.exps[c + e];
        s[e] = c + e > x.last ? -INFINITY : __uint_as_float(z[e]) * score_factor(x.sc_row, exp2_int(ex.x));
        ve[e] = (float)ex.y;
    }
}
// Largest score, and score plus V exponent.
__device__ __noinline__ float2 mixed_max(const MixedHalf x) {
    float m = -INFINITY, y = -INFINITY;
#pragma unroll 1
    for (int c = 0; c < 32; c += 8) {
        float s[8], ve[8];
        mixed_scores(x, c, s, ve);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            m = fmaxf(m, s[e]);
            y = fmaxf(y, s[e] + ve[e]);
        }
    }
    return make_float2(m, y);
}
// Weights 2^(s + ve - R + 7) to the columns of P at t_p; returns l and their sum relative to 2^M.  The second half's weights
// go over columns of the first half's scores.
__device__ __noinline__ float mixed_weights(const MixedHalf x, float M, float R, float l, int half, int bar, uint32_t t_p) {
    if (half == 1) named_barrier(bar, 64);
#pragma unroll 1
    for (int c = 0; c < 32; c += 8) {
        float s[8], ve[8];
        uint32_t pk[4];
        mixed_scores(x, c, s, ve);
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            l += fast_exp2(s[e] - M) + fast_exp2(s[e + 1] - M);
            pk[e >> 1] = pack_f16x2(fast_exp2(s[e] + (ve[e] + kShift - R)), fast_exp2(s[e + 1] + (ve[e + 1] + kShift - R)));
        }
        tmem_st_cols<4>(t_p + (uint32_t)(c / 2), pk);
    }
    if (half == 0) named_barrier(bar, 64);
    return l;
}

// The rows of a unit from the records of its pieces, in the order of its tiles.  A thread takes kItems (row, four columns)
// at once and the records kAhead at a time: one after the other, the loads' latency made it 40 us for 256 rows.
template <int DV, int kItems, int kAhead>
__device__ __forceinline__ void merge_pieces(const PreArgs &a, int record, int n, int q0, int rows, int h, int tid) {
    constexpr size_t kRec = (size_t)kRows * (DV + 2);
    if (!in_bounds(record, kSlots, a.status) || !in_bounds(record + n - 1, kSlots, a.status) ||
        !in_bounds(q0 + rows - 1, a.tokens, a.status))
        return;
    // a warp: 8 rows by 4 fours of columns, whole sectors in the records (columns by fours ahead of rows) and in the output
    const int r8 = (rows + 7) >> 3, items = r8 * DV * 2;
    auto row_of = [&](int e) { return (e >> 5) % r8 * 8 + (e & 7); };
    auto col_of = [&](int e) { return (e >> 5) / r8 * 4 + (e >> 3 & 3); };
    for (int e0 = tid; e0 < items; e0 += kItems * kThreads) {
        float M[kItems], L[kItems];
        float4 x[kItems];
        int at_o[kItems], at_ml[kItems];
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
            const int e = min(e0 + k * kThreads, items - 1), col = col_of(e), r = min(row_of(e), rows - 1);
            M[k] = -INFINITY;
            L[k] = 0.f;
            x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            at_o[k] = (col * kRows + r) * 4;
            at_ml[k] = DV * kRows + 2 * r;
        }
#pragma unroll kAhead
        for (int s = 0; s < n; ++s) {
            const float *rec = a.partials + (size_t)(record + s) * kRec;
            float2 ml[kItems];
            float4 o[kItems];
#pragma unroll
            for (int k = 0; k < kItems; ++k) {
                ml[k] = __ldcg(reinterpret_cast<const float2 *>(rec + at_ml[k]));
                o[k] = __ldcg(reinterpret_cast<const float4 *>(rec + at_o[k]));
            }
#pragma unroll
            for (int k = 0; k < kItems; ++k) {
                if (ml[k].x == -INFINITY) continue;  // nothing of this piece is seen by the row
                const float m = fmaxf(M[k], ml[k].x), f = fast_exp2(M[k] - m), g = fast_exp2(ml[k].x - m);
                M[k] = m;
                L[k] = fmaf(f, L[k], g * ml[k].y);
                x[k].x = fmaf(f, x[k].x, g * o[k].x);
                x[k].y = fmaf(f, x[k].y, g * o[k].y);
                x[k].z = fmaf(f, x[k].z, g * o[k].z);
                x[k].w = fmaf(f, x[k].w, g * o[k].w);
            }
        }
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
            const int e = e0 + k * kThreads, col = col_of(e), r = row_of(e);
            if (e >= items || r >= rows) continue;
            const float inv = M[k] == -INFINITY ? 0.f : 1.f / L[k];
            *reinterpret_cast<uint2 *>(a.out + ((size_t)(q0 + r) * a.n_q + h) * DV + col * 4) =
                make_uint2(pack_bf16x2(x[k].x * inv, x[k].y * inv), pack_bf16x2(x[k].z * inv, x[k].w * inv));
        }
    }
}

// Number of pieces that the blocks of this lane's request (n blocks of 256 of its last `rows` positions of T) are cut into.
// All lanes hold a request each; lane l looks at pieces of at most 1 / (l + 1) of the longest unit, and the lane whose
// longest piece is shortest wins, if every piece has an SM.  A piece takes kPieceCost tiles besides its own, more where its
// rows are merged.
__device__ __forceinline__ int cut_units(const PreArgs &a, int n, int rows, int T, int lane) {
    constexpr int kPieceCost = 6, kCutCost = 2, kRowCost = 32;  // (rows of a merge that cost a tile)
    const int tiles = n > 0 ? (T - 1) / BN + 1 : 0;  // of its last block
    const int longest = max(1, __reduce_max_sync(0xffffffffu, tiles));
    // (s = ceil(tiles / most) in floats: any s would be right, and all CTAs work out the same)
    auto cut = [&](int t, float per) { return max(1, (int)ceilf((float)t * per - 1e-3f)); };
    const float per = (float)(lane + 1) / (float)longest;
    int count = 0, time = 0;
    for (int j = 0; j < a.batch; ++j) {
        const int nj = __shfl_sync(0xffffffffu, n, j), tj = __shfl_sync(0xffffffffu, tiles, j);
        const int rj = __shfl_sync(0xffffffffu, rows, j);
        if (nj == 0) continue;
        const int s = cut(tj, per);
        count += nj * s;
        time = max(time, (int)__fdividef((float)tj, (float)s) + kPieceCost + (s > 1 ? kCutCost + min(rj, kRows) / kRowCost : 0));
    }
    if ((long long)count * a.n_q > a.max_pieces) time = lane == 0 ? 0x3ffffff : 0x7ffffff;  // lane 0 cuts nothing
    const int best = (int)__reduce_min_sync(0xffffffffu, (uint32_t)min(time, 0x7ffffff) * 32u + (uint32_t)lane) & 31;
    return cut(tiles, (float)(best + 1) / (float)longest);
}

template <int DK, int DV>
__global__ void __launch_bounds__(kThreads, 1)
    prefill_kv8_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                       const PreArgs a) {
    using C = Cfg<DK, DV>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = align_smem_1024(smem_raw);
    Misc &ms = *reinterpret_cast<Misc *>(smem + C::OFF_MISC);
    volatile int *abort_flag = &ms.abort_flag;
    const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
    if (tid == 32) {
        for (int s = 0; s < kRaw; ++s) {
            mbar_init(&ms.raw_full[s], 1);
            mbar_init(&ms.raw_empty[s], kConvWarps);
        }
        for (int s = 0; s < 3; ++s) {
            mbar_init(&ms.cv_full[s], kConvWarps);
            mbar_init(&ms.cv_empty[s], 1);
        }
        for (int s = 0; s < kScaleSlots; ++s) {
            mbar_init(&ms.sc_full[s], 1);
            mbar_init(&ms.sc_empty[s], kConvWarps);
        }
        mbar_init(&ms.q_full, kSoftmaxWarps);
        for (int t = 0; t < QT; ++t) {
            mbar_init(&ms.s_full[t][0], 1);
            mbar_init(&ms.s_full[t][1], 1);
            mbar_init(&ms.p_full[t][0], 8);
            mbar_init(&ms.p_full[t][1], 8);
            mbar_init(&ms.pv_done[t][0], 1);
            mbar_init(&ms.pv_done[t][1], 1);
        }
        mbar_init(&ms.mma_done, 1);
        ms.nan_seen = 0;
        ms.abort_flag = 0;
        ms.last_flag = 0;
        fence_barrier_init();
    }
    if (tid < DV) ms.nan_pos[tid] = 0x7fffffff;
    // ---- the piece: of a unit (256-row block, head), heaviest first: up to 32 requests by their length, more in the reverse
    // of their order; a request's last block (the longest context) first, the pieces of a block side by side
    if (warp == 0) {
        const bool flags = blockIdx.x == 0;
        auto look = [&](int b, int2 &r, int &T) {  // blocks of request b
            r = make_int2(0, 0);
            T = 0;
            if (b >= a.batch) return 0;
            r = request_rows(a, b);
            const int raw_T = __ldg(a.seq_lens + b);
            T = clamp_to(raw_T, a.t_max);
            if (flags) {
                const int raw_s = __ldg(a.query_start + b), raw_e = __ldg(a.query_start + b + 1);
                if (raw_s < 0 || raw_e < raw_s || raw_e > a.tokens || raw_T != T || r.y > raw_T)
                    record_error(a.status, DIFFQKV_ERR_DEVICE_SEQLEN);
            }
            return (r.y + kRows - 1) / kRows;
        };
        auto found = [&](int b, int block, const int2 &r, int T, int pieces, int piece, int record) {
            ms.found[0] = b;
            ms.found[1] = block;
            ms.found[2] = r.x;
            ms.found[3] = r.y;
            ms.found[4] = T;
            ms.found[5] = pieces;
            ms.found[6] = piece;
            ms.found[7] = record;
        };
        const int want = (int)(blockIdx.x / a.n_q);
        if (lane == 0) ms.found[0] = -1;
        __syncwarp();
        int2 r;
        int T;
        if (a.batch <= kCutBatch) {
            const int n = look(lane, r, T);
            const int s = a.max_pieces > 0 ? cut_units(a, n, r.y, T, lane) : 1;  // pieces of each of this request's blocks
            const int mine = n * s;
            int before = 0, records = 0;
            for (int j = 0; j < a.batch; ++j) {
                const int Tj = __shfl_sync(0xffffffffu, T, j), nj = __shfl_sync(0xffffffffu, mine, j);
                const int cj = __shfl_sync(0xffffffffu, s > 1 ? mine : 0, j);
                if (Tj > T || (Tj == T && j > lane)) {
                    before += nj;
                    records += cj;
                }
            }
            if (want >= before && want < before + mine) {
                const int x = want - before, block = x / s;
                found(lane, n - 1 - block, r, T, s, x - block * s, (records + block * s) * a.n_q);
            }
        } else {
            int after = 0;  // blocks of the requests behind this group of 32
            for (int base = (a.batch - 1) / 32 * 32; base >= 0; base -= 32) {
                const int n = look(base + lane, r, T);
                int incl = n;
#pragma unroll
                for (int off = 1; off < 32; off <<= 1) {
                    const int y = __shfl_down_sync(0xffffffffu, incl, off);
                    if (lane + off < 32) incl += y;
                }
                const int before = after + incl - n;
                if (want >= before && want < before + n) found(base + lane, n - 1 - (want - before), r, T, 1, 0, 0);
                after += __shfl_sync(0xffffffffu, incl, 0);
            }
        }
    }
    __syncthreads();
    const int b = ms.found[0];
    if (b < 0) return;
    const int h = blockIdx.x % a.n_q;
    const int row0 = ms.found[1] * kRows, n_rows = ms.found[3], T = ms.found[4];
    const int first = T - n_rows;  // position of the request's first row
    const int q0 = ms.found[2] + row0;
    const int kh = h / (a.n_q / a.n_k), vh = h / (a.n_q / a.n_v);

    int n_kv[QT];  // K/V tiles that a query tile's rows see
#pragma unroll
    for (int t = 0; t < QT; ++t) {
        const int rows = min(n_rows - row0 - t * BM, BM);
        const int last = first + row0 + t * BM + rows - 1;
        n_kv[t] = uniform(rows > 0 && last >= 0 ? last / BN + 1 : 0);
    }
    const int n_all = max(n_kv[0], n_kv[1]);
    const int chunk = uniform((n_all + ms.found[5] - 1) / ms.found[5]), piece = uniform(ms.found[6]);
    const int n0 = piece * chunk, n1 = min(n_all, n0 + chunk);
    // this unit's records and counter, piece by piece; 0 where it is whole
    const int pieces = chunk > 0 ? (n_all + chunk - 1) / chunk : 1, record = ms.found[7] + h * ms.found[5];
    if (n_all == 0 || n0 >= n1) {
        if (n_all == 0 && piece == 0)  // rows without a position
            for (int e = tid; e < min(n_rows - row0, kRows) * (DV / 8); e += kThreads)
                if (in_bounds(q0 + e / (DV / 8), a.tokens, a.status))
                    *reinterpret_cast<uint4 *>(a.out + ((size_t)(q0 + e / (DV / 8)) * a.n_q + h) * DV + e % (DV / 8) * 8) =
                        make_uint4(0, 0, 0, 0);
        return;
    }
    const int end[QT] = {min(n_kv[0], n1), min(n_kv[1], n1)};

    if (warp == kMmaWarp) {
        tmem_alloc(&ms.tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = (uint32_t)uniform((int)ms.tmem_slot);
    constexpr uint32_t T_O = QT * 2 * BN;  // S_0 | S_0' | S_1 | S_1' | O_0 | O_1

    if (warp == kLoadWarp) {
        // ======================= TMA producer: codes, in sub-boxes inside one page (lane f holds sub-box f's page)
        if (lane == 0) {
            prefetch_tensormap(&tm_k);
            prefetch_tensormap(&tm_v);
        }
        auto subs = [&](int n) {
            const int v = min(BN, T - n * BN) + a.sub_rows - 1;
            return a.sub_shift >= 0 ? v >> a.sub_shift : v / a.sub_rows;
        };
        auto entry = [&](int n) {
            return lane < subs(n)
                       ? __ldg(a.block_table + (size_t)b * a.max_blocks + div_page(a, n * BN + lane * a.sub_rows))
                       : 0;
        };
        int next = entry(n0), issued = 0, st = 0;
        uint32_t par = 0;
        for (int n = n0; n < n1; ++n) {
            int page = next;
            if (page < 0 || page >= a.num_pages) {
                record_error(a.status, DIFFQKV_ERR_DEVICE_PAGE);
                page = 0;
            }
            const int cnt = uniform(subs(n)), p = n * BN + lane * a.sub_rows;
            const int row = p - div_page(a, p) * a.page_size;
            if (n + 1 < n1) next = entry(n + 1);
            if (issued >= kRaw) mbar_wait_bounded(&ms.raw_empty[st], par ^ 1u, a.wait_limit_ns, abort_flag, a.status);
            if (__any_sync(0xffffffffu, *abort_flag != 0)) break;
            if (elect_one()) mbar_arrive_expect_tx(&ms.raw_full[st], (uint32_t)(cnt * a.sub_rows * (DK + DV)));
            __syncwarp();
            uint8_t *kd = smem + C::OFF_RAW + st * C::RAW, *vd = kd + C::RAW_K;
#pragma unroll 2
            for (int f = 0; f < cnt; ++f) {
                const int row_f = __shfl_sync(0xffffffffu, row, f), page_f = __shfl_sync(0xffffffffu, page, f);
                if (elect_one()) {
                    tma_load_4d(kd + f * a.sub_rows * DK, &tm_k, &ms.raw_full[st], 0, kh, row_f, page_f);
                    tma_load_4d(vd + f * a.sub_rows * DV, &tm_v, &ms.raw_full[st], 0, vh, row_f, page_f);
                }
            }
            __syncwarp();
            ++issued;
            if (++st == kRaw) {
                st = 0;
                par ^= 1u;
            }
        }
        for (int k = max(0, issued - kRaw); k < issued; ++k)  // drain
            mbar_wait_bounded(&ms.raw_full[k % kRaw], (uint32_t)(k / kRaw & 1), a.wait_limit_ns, nullptr, a.status);
    } else if (warp == kScaleWarp) {
        // ======================= scales, four tiles at a time: lane l looks after positions 2 l and 2 l + 1 of a tile
        const int per_page = a.page_size / a.sb;
        for (int n = n0; n < n1; n += 4) {
            int ek[4][2], ev[4][2];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int p = min((n + i) * BN + 2 * lane + e, T - 1);
                    const int lp = div_page(a, p);
                    int page = __ldg(a.block_table + (size_t)b * a.max_blocks + lp);
                    if (page < 0 || page >= a.num_pages) page = 0;
                    long long blk = (long long)page * per_page + (p - lp * a.page_size) / a.sb;
                    if (!in_bounds(blk, a.scale_blocks, a.status)) blk = 0;
                    ek[i][e] = __ldg(a.k_scales + blk * a.n_k + kh);
                    ev[i][e] = __ldg(a.v_scales + blk * a.n_v + vh);
                }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (n + i >= n1) break;
                const int k = n + i - n0, slot = k % kScaleSlots;
                if (k >= kScaleSlots)
                    wait_for(&ms.sc_empty[slot], (uint32_t)((k / kScaleSlots - 1) & 1), a.wait_limit_ns, abort_flag, a.status);
                const int k0 = kv8_exp(ek[i][0]), k1 = kv8_exp(ek[i][1]), v0 = kv8_exp(ev[i][0]), v1 = kv8_exp(ev[i][1]);
                int kr = __reduce_max_sync(0xffffffffu, max(k0, k1)), vr = __reduce_max_sync(0xffffffffu, max(v0, v1));
                const bool mixed = kr - __reduce_min_sync(0xffffffffu, min(k0, k1)) > kSpreadK ||
                                   vr - __reduce_min_sync(0xffffffffu, min(v0, v1)) > kSpreadV;
                // 2^(e - ref) in f16 for both halves of a word, 1 in a mixed tile; 0 for positions behind the end
                auto mul = [&](int e, int ref, int pos) -> uint32_t {
                    const int d = mixed ? 0 : e - ref;  // (2^-15 is the one that is subnormal)
                    return pos >= T ? 0u : (d >= -14 ? (uint32_t)(d + 15) << 10 : 0x200u) * 0x10001u;
                };
                const int p = (n + i) * BN + 2 * lane;
                ms.k_mul[slot][2 * lane] = mul(k0, kr, p);
                ms.k_mul[slot][2 * lane + 1] = mul(k1, kr, p + 1);
                ms.v_mul[slot][2 * lane] = mul(v0, vr, p);
                ms.v_mul[slot][2 * lane + 1] = mul(v1, vr, p + 1);
                if (mixed) {
                    ms.exps[k % kExpSlots][2 * lane] = make_char2((signed char)k0, (signed char)v0);
                    ms.exps[k % kExpSlots][2 * lane + 1] = make_char2((signed char)k1, (signed char)v1);
                }
                if (lane == 0) ms.scale_ref[slot] = make_float2(exp2_int(kr), mixed ? kMixed : (float)vr);
                if ((n + i + 1) * BN - 1 > first + row0) {  // positions that not every row sees
                    wait_for(&ms.raw_full[k % kRaw], (uint32_t)(k / kRaw & 1), a.wait_limit_ns, abort_flag, a.status);
                    take_nans<DV>(smem + C::OFF_RAW + k % kRaw * C::RAW + C::RAW_K, (n + i) * BN, lane, ms.nan_pos, &ms.nan_seen);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&ms.sc_full[slot]);
            }
        }
    } else if (warp >= kConvWarp0) {
        // ======================= codes -> f16
        const int ct = tid - kConvWarp0 * 32;
        const Widen<DK> widen_k(ct);
        const Widen<DV> widen_v(ct);
        int rs = 0, cs = 0;
        uint32_t rp = 0, cp = 0;
        for (int k = 0; k < n1 - n0; ++k) {
            const int slot = k % kScaleSlots;
            wait_for(&ms.sc_full[slot], (uint32_t)(k / kScaleSlots & 1), a.wait_limit_ns, abort_flag, a.status);
            wait_for(&ms.raw_full[rs], rp, a.wait_limit_ns, abort_flag, a.status);
            if (k >= C::STAGES) wait_for(&ms.cv_empty[cs], cp ^ 1u, a.wait_limit_ns, abort_flag, a.status);
            const uint8_t *raw = smem + C::OFF_RAW + rs * C::RAW;
            uint8_t *dst = smem + C::OFF_CONV + cs * C::CONV;
            const bool tail = (n0 + k + 1) * BN > T;
            widen_k.run(raw, dst, ms.k_mul[slot], tail);
            widen_v.run(raw + C::RAW_K, dst + C::K_BYTES, ms.v_mul[slot], tail);
            if (ct == 0) ms.ref[k & 3] = ms.scale_ref[slot];
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&ms.cv_full[cs]);
                mbar_arrive(&ms.raw_empty[rs]);
                mbar_arrive(&ms.sc_empty[slot]);
            }
            if (++rs == kRaw) {
                rs = 0;
                rp ^= 1u;
            }
            if (++cs == C::STAGES) {
                cs = 0;
                cp ^= 1u;
            }
        }
    } else if (warp == kMmaWarp) {
        // ======================= MMA issue
        constexpr uint32_t idesc_qk = idesc_f16(BM, BN, false), idesc_pv = idesc_f16(BM, DV, true);
        const uint64_t q_desc = smem_desc_sw128(smem_addr(smem), 16, 1024);
        const uint64_t k_desc = smem_desc_sw128(smem_addr(smem + C::OFF_CONV), 16, 1024);
        const uint64_t v_desc = smem_desc_sw128(smem_addr(smem + C::OFF_CONV + C::K_BYTES), BN * 128, 1024);
        wait_for(&ms.q_full, 0, a.wait_limit_ns, abort_flag, a.status);
        tc_fence_after();
        int cs = 0, pst = 0;  // stage of tile n, of tile n - 1
        uint32_t cp = 0;
        for (int n = n0; n <= n1; ++n) {
            const int k = n - n0;
            if (n < n1) {
                wait_for(&ms.cv_full[cs], cp, a.wait_limit_ns, abort_flag, a.status);
                tc_fence_after();
                const uint64_t kd = k_desc + (uint32_t)(cs * (C::CONV >> 4));
#pragma unroll
                for (int t = 0; t < QT; ++t) {
                    if (n >= end[t]) continue;
                    // S buffer k & 1 held S and P of tile n - 2: its P.V was issued ahead of this
                    const uint64_t qd = q_desc + (uint32_t)(t * (C::Q_BYTES >> 4));
                    const uint32_t t_s = tmem + (uint32_t)(t * 2 * BN + (k & 1) * BN);
                    if (elect_one()) {
#pragma unroll
                        for (int ks = 0; ks < DK / 16; ++ks)
                            umma_bf16(t_s, qd + (ks >> 2) * (BM * 128 >> 4) + (ks & 3) * 2,
                                      kd + (ks >> 2) * (BN * 128 >> 4) + (ks & 3) * 2, idesc_qk, ks > 0 ? 1u : 0u);
                        umma_commit(&ms.s_full[t][k & 1]);
                    }
                    __syncwarp();
                }
            }
            if (k >= 1) {
                const uint64_t vd = v_desc + (uint32_t)(pst * (C::CONV >> 4));
                const uint32_t onto = (uint32_t)(k > 1);
#pragma unroll
                for (int t = 0; t < QT; ++t) {
                    if (n - 1 >= end[t]) continue;
                    wait_for(&ms.p_full[t][(k - 1) & 1], (uint32_t)((k - 1) >> 1 & 1), a.wait_limit_ns, abort_flag, a.status);
                    tc_fence_after();
                    const uint32_t t_p = tmem + (uint32_t)(t * 2 * BN + ((k - 1) & 1) * BN);
                    if (elect_one()) {
#pragma unroll
                        for (int ks = 0; ks < BN / 16; ++ks)
                            umma_bf16_tmem_a(tmem + T_O + (uint32_t)(t * DV), t_p + ks * 8, vd + ks * (16 * 128 >> 4),
                                             idesc_pv, ks > 0 ? 1u : onto);
                        umma_commit(&ms.pv_done[t][(k - 1) & 1]);
                    }
                    __syncwarp();
                }
                if (elect_one()) umma_commit(&ms.cv_empty[pst]);
                __syncwarp();
                if (++pst == C::STAGES) pst = 0;
            }
            if (++cs == C::STAGES) {
                cs = 0;
                cp ^= 1u;
            }
        }
        if (elect_one()) umma_commit(&ms.mma_done);
        __syncwarp();
        wait_for(&ms.mma_done, 0, a.wait_limit_ns, nullptr, a.status);
    } else {
        // ======================= softmax: warps 8 t .. 8 t + 7 hold query tile t; a row (TMEM lane r) belongs to two threads,
        // one for each half of a tile's columns.  Four warps a scheduler hide one another's latencies.
        const int t = warp >> 3, half = warp >> 2 & 1, r = (warp & 3) * 32 + lane;
        const int bar = 1 + t * 4 + (warp & 3);  // named barrier of the two warps that share rows
        const int rr = row0 + t * BM + r;        // row of the request
        const int i = first + rr;                // its position
        const bool live = rr < n_rows;
        const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
        constexpr int HV = DV / 2;               // this thread's columns of O
        const uint32_t t_o = tmem + T_O + (uint32_t)(t * DV + half * HV) + lane_base;
        float sc_row;  // scale * log2(e) * 2^(the query's exponent)
        {
            // The rows in f16, a row's largest element brought into [2^14, 2^15) by a power of two.  Of the 32 rows of two
            // warps each takes 16, a row's 16-byte pieces side by side: a thread to a row would touch 32 lines a load.
            constexpr int LPR = DK / 8, RPI = 32 / LPR, NI = 16 / RPI;
            const int c = lane % LPR, rb = (warp & 3) * 32 + half * 16 + lane / LPR;
            uint4 x[NI];
#pragma unroll
            for (int k = 0; k < NI; ++k) {
                const size_t g = (size_t)(q0 + t * BM + rb + k * RPI) * a.n_q + h;
                x[k] = row0 + t * BM + rb + k * RPI < n_rows && in_bounds((long long)g, (long long)a.tokens * a.n_q, a.status)
                           ? __ldg(reinterpret_cast<const uint4 *>(a.q + g * DK) + c)
                           : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int k = 0; k < NI; ++k) {
                const int rq = rb + k * RPI;
                uint32_t m = __vmaxu2(__vmaxu2(x[k].x & 0x7fff7fffu, x[k].y & 0x7fff7fffu),
                                      __vmaxu2(x[k].z & 0x7fff7fffu, x[k].w & 0x7fff7fffu));
                m = max(m & 0xffffu, m >> 16);
#pragma unroll
                for (int off = 1; off < LPR; off <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, off));
                const float f = exp2_int(min(141 - (int)(m >> 7), 126));
                uint4 y;
                y.x = pack_f16x2(bf16lo(x[k].x) * f, bf16hi(x[k].x) * f);
                y.y = pack_f16x2(bf16lo(x[k].y) * f, bf16hi(x[k].y) * f);
                y.z = pack_f16x2(bf16lo(x[k].z) * f, bf16hi(x[k].z) * f);
                y.w = pack_f16x2(bf16lo(x[k].w) * f, bf16hi(x[k].w) * f);
                *reinterpret_cast<uint4 *>(smem + t * C::Q_BYTES + (c >> 3) * (BM * 128) + rq * 128 + ((c & 7) ^ (rq & 7)) * 16) = y;
                if (c == 0) ms.row_s[t][0][rq] = __uint_as_float(m);
            }
            named_barrier(bar, 64);
            const uint32_t m = __float_as_uint(ms.row_s[t][0][r]);
            const int se = min(141 - (int)(m >> 7), 126);
            named_barrier(bar, 64);
            // a row with infinities or NaN has no scale: its scores become NaN
            sc_row = m >= 0x7f80u ? __int_as_float(0x7fffffff) : a.scale_log2 * exp2_int(-se);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(&ms.q_full);
        }
        float R = 0.f;       // O holds the sum of 2^(s - R + 7) v (R and M: the same in both halves)
        float M = 0.f;       // l is relative to 2^M
        float l = 0.f;       // this half's sum of the weights
        for (int n = n0; n < end[t]; ++n) {
            const int k = n - n0;
            const uint32_t t_s = tmem + (uint32_t)(t * 2 * BN + (k & 1) * BN) + lane_base;
            wait_for(&ms.s_full[t][k & 1], (uint32_t)(k >> 1 & 1), a.wait_limit_ns, abort_flag, a.status);
            tc_fence_after();
            uint32_t x[32];
            tmem_ld32(t_s + (uint32_t)(half * 32), x);
            // (written before the tile's conversion was handed over, and so before its S; the slot is written again after
            // the P.V of tile k + 1)
            const float2 ref = ms.ref[k & 3];
            const float sc = score_factor(sc_row, ref.x);
            tmem_wait_ld();
            const int j0 = n * BN + half * 32;
            if (j0 + 31 > first + row0 + t * BM) {  // causal mask, on columns that reach past the tile's first row
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    if (j0 + e > i) x[e] = 0xff800000u;
            }
            auto sv = [&](int e) { return __uint_as_float(x[e]); };
            float m4[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) m4[e] = fmaxf(sv(e), sv(4 + e));
#pragma unroll
            for (int e = 8; e < 32; e += 8)
#pragma unroll
                for (int c = 0; c < 4; ++c) m4[c] = fmax3f(m4[c], sv(e + c), sv(e + 4 + c));
            float m_half = fmaxf(fmax3f(m4[0], m4[1], m4[2]), m4[3]) * sc, y_half = m_half + ref.y;
            // Both halves have read S behind this barrier (P goes over columns of the other half), and agree on whether a
            // reference has to move: the first tile, a row whose R grew by 2^8, a row sum that would leave its range, a mixed tile.
            // (Two warps none of whose rows see any of a mixed tile may go on without: all of their weights are zero.)
            do {
                if (pair_any(bar, k == 0 || y_half > R + kRescale || m_half > M + kGrow)) {
                    const MixedHalf mix{t_s + (uint32_t)(half * 32), ms.exps[k % kExpSlots] + half * 32, i - j0, sc_row};
                    if (ref.y == kMixed) {
                        const float2 my = mixed_max(mix);
                        m_half = my.x;
                        y_half = my.y;
                    }
                    ms.row_s[t][half][r] = m_half;
                    ms.row_y[t][half][r] = y_half;
                    named_barrier(bar, 64);
                    const float m_new = fmaxf(m_half, ms.row_s[t][1 - half][r]), y_new = fmaxf(y_half, ms.row_y[t][1 - half][r]);
                    named_barrier(bar, 64);
                    if (k == 0) {
                        M = m_new == -INFINITY ? 0.f : m_new;
                        R = y_new == -INFINITY ? 0.f : y_new;
                    } else {
                        // (S of tile k has been waited for, so P.V of tiles up to k - 2 is done: k - 1 is this barrier's next phase)
                        wait_for(&ms.pv_done[t][(k - 1) & 1], (uint32_t)((k - 1) >> 1 & 1), a.wait_limit_ns, abort_flag,
                                          a.status);
                        tc_fence_after();
                        const bool grow = y_new > R + kRescale;
                        const float alpha = grow ? fast_exp2(R - y_new) : 1.f;
                        if (grow) R = y_new;
                        if (m_new > M) {  // (with R, so that R - M stays an exponent of V)
                            l *= fast_exp2(M - m_new);
                            M = m_new;
                        }
#pragma unroll 1
                        for (int c = 0; c < HV; c += 16) {
                            uint32_t y[16];
                            tmem_ld_cols<16>(t_o + c, y);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 16; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * alpha);
                            tmem_st_cols<16>(t_o + c, y);
                        }
                        tmem_wait_st();
                    }
                    if (ref.y == kMixed) {
                        l = mixed_weights(mix, M, R, l, half, bar, t_s + (uint32_t)(half * 16));
                        break;
                    }
                }
                uint32_t pk[16];
                // weights 2^(s + e_ref - R + 7).  Where V's exponent is so far below the row's that they are zero in f16, larger
                // ones that still are, lest they vanish from the sum
                const float c = fmaxf(ref.y - R, -kFloor - M) + kShift;
                const f32x2_t sc2 = f2_pack(sc, sc), c2 = f2_pack(c, c);
                f32x2_t l2[2] = {0ull, 0ull};
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    float t0, t1;
                    f2_unpack(f2_fma(f2_pack(sv(e), sv(e + 1)), sc2, c2), t0, t1);
                    const float p0 = fast_exp2(t0), p1 = fast_exp2(t1);
                    l2[(e >> 1) & 1] = f2_add(l2[(e >> 1) & 1], f2_pack(p0, p1));
                    pk[e >> 1] = pack_f16x2(p0, p1);
                }
                float la, lb;
                f2_unpack(f2_add(l2[0], l2[1]), la, lb);
                l = fmaf(la + lb, fast_exp2(-c - M), l);
                tmem_st_cols<16>(t_s + (uint32_t)(half * 16), pk);
            } while (false);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ms.p_full[t][k & 1]);
        }
        const int done = end[t] - n0;
        if (done > 0) {
            wait_for(&ms.pv_done[t][(done - 1) & 1], (uint32_t)((done - 1) >> 1 & 1), a.wait_limit_ns, abort_flag,
                              a.status);
            tc_fence_after();
        }
        ms.row_s[t][half][r] = l;
        named_barrier(bar, 64);
        l += ms.row_s[t][1 - half][r];
        const float o_scale = exp2f(R - kShift - M);
        // A whole unit: the rows, divided by their sums.  Otherwise this piece's record: O relative to m, four columns of all
        // rows after another, then (m, l) of the rows.
        const bool whole = pieces == 1;
        const bool some = done > 0 && i >= 0 && n0 * BN <= i;  // the row sees a position of this piece
        const float inv_l = !whole ? 1.f : l > 0.f || l != l ? 1.f / l : 0.f;
        // Whole rows leave through the pair's 32 rows of Q, free now, 32 columns at a time, so that a warp's store covers whole
        // sectors of few rows (a thread to a row touches 32 lines a store).
        uint4 *rec = reinterpret_cast<uint4 *>(a.partials + (size_t)(record + piece) * C::REC) + half * (HV / 4) * kRows + t * BM + r;
        uint8_t *stage = smem + t * C::Q_BYTES + (warp & 3) * 4096 + half * 2048;
#pragma unroll 1
        for (int c = 0; c < HV; c += 16) {
            uint32_t y[16];
            if (done > 0) {
                tmem_ld_cols<16>(t_o + c, y);
                tmem_wait_ld();
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) y[e] = __float_as_uint(some ? __uint_as_float(y[e]) * inv_l * o_scale : 0.f);
            if (ms.nan_seen) {
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if (i >= ms.nan_pos[half * HV + c + e]) y[e] = 0x7fffffffu;
            }
            if (whole) {
#pragma unroll
                for (int e = 0; e < 16; e += 2)
                    y[e >> 1] = pack_bf16x2(__uint_as_float(y[e]), __uint_as_float(y[e + 1]));
                const int ch = c >> 3 & 2, sw = lane >> 1 & 3;  // 16-byte pieces of a 64-byte row, permuted
                *reinterpret_cast<uint4 *>(stage + lane * 64 + (ch ^ sw) * 16) = make_uint4(y[0], y[1], y[2], y[3]);
                *reinterpret_cast<uint4 *>(stage + lane * 64 + ((ch + 1) ^ sw) * 16) = make_uint4(y[4], y[5], y[6], y[7]);
                if (ch == 2) {
                    __syncwarp();
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int ro = k * 8 + (lane >> 2), rg = t * BM + (warp & 3) * 32 + ro;
                        const size_t g = (size_t)(q0 + rg) * a.n_q + h;
                        if (row0 + rg < n_rows && in_bounds((long long)g, (long long)a.tokens * a.n_q, a.status))
                            *reinterpret_cast<uint4 *>(a.out + g * DV + half * HV + (c - 16) + (lane & 3) * 8) =
                                lds128(stage + ro * 64 + ((lane & 3) ^ (ro >> 1 & 3)) * 16);
                    }
                    __syncwarp();
                }
            } else if (live && in_bounds(record + piece, kSlots, a.status)) {
#pragma unroll
                for (int e = 0; e < 16; e += 4, rec += kRows) __stcg(rec, make_uint4(y[e], y[e + 1], y[e + 2], y[e + 3]));
            }
        }
        if (!whole) {
            if (live && half == 0 && in_bounds(record + piece, kSlots, a.status))
                __stcg(reinterpret_cast<float2 *>(a.partials + (size_t)(record + piece) * C::REC + (size_t)DV * kRows) + t * BM + r,
                       some ? make_float2(M, l) : make_float2(-INFINITY, 0.f));
            __threadfence();
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
    if (pieces == 1) return;

    // ---- a cut unit: the last of its CTAs merges the records
    if (tid == 0) {
        __threadfence();
        ms.last_flag = in_bounds(record, kSlots, a.status) && atomicAdd(a.counters + record, 1u) == (unsigned)(pieces - 1);
    }
    __syncthreads();
    if (!*(volatile int *)&ms.last_flag) return;
    __threadfence();
    const int rows = min(n_rows - row0, kRows);
    if (rows * (DV / 4) <= kThreads) merge_pieces<DV, 1, 8>(a, record, pieces, q0, rows, h, tid);
    else merge_pieces<DV, 4, 2>(a, record, pieces, q0, rows, h, tid);
    if (tid == 0) a.counters[record] = 0u;
}

// ------------------------------------------------------------------ host side

using PreFn = void (*)(CUtensorMap, CUtensorMap, PreArgs);

template <int DK, int DV>
PreFn plan(int *smem) {
    *smem = Cfg<DK, DV>::OFF_MISC + (int)sizeof(Misc) + 1024;
    static_assert(Cfg<DK, DV>::OFF_MISC + sizeof(Misc) + 1024 <= 227 * 1024, "shared memory");
    return prefill_kv8_kernel<DK, DV>;
}

size_t prefill_kv8_workspace_size(const diffqkv_dims_t *d) {
    if (validate_dims(d) != DIFFQKV_OK) return 0;
    static_assert(kSlots <= kWsCounters, "a counter for each record");
    return kWsRecords + (size_t)kSlots * kRows * (d->d_v + 2) * sizeof(float);
}

diffqkv_status_t prefill_kv8_launch(const diffqkv_dims_t *d, const diffqkv_kv8_cache_t *cache, const void *q,
                                    const int32_t *query_start, int32_t tokens, const int32_t *block_table,
                                    int32_t max_blocks, const int32_t *seq_lens, void *out, void *workspace,
                                    size_t workspace_bytes, cudaStream_t stream) {
    diffqkv_status_t st = validate_kv8(d, cache);
    if (st != DIFFQKV_OK) return st;
    if (!q || !query_start || !block_table || !seq_lens || !out || max_blocks < 1 || tokens < 1)
        return DIFFQKV_ERR_INVALID_ARG;
    const int P = cache->page_size;
    if ((long long)max_blocks * P > 0x7fffffffLL) return DIFFQKV_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(out) || (reinterpret_cast<uintptr_t>(seq_lens) & 3u) ||
        (reinterpret_cast<uintptr_t>(block_table) & 3u) || (reinterpret_cast<uintptr_t>(query_start) & 3u))
        return DIFFQKV_ERR_MISALIGNED;
    if (!workspace || workspace_bytes < prefill_kv8_workspace_size(d)) return DIFFQKV_ERR_WORKSPACE;
    if (!aligned16(workspace)) return DIFFQKV_ERR_MISALIGNED;
    // blocks of kRows rows over all requests: at most this many
    const long long units = ((long long)tokens / kRows + d->batch) * d->n_q;
    if (units > 0x7fffffffLL) return DIFFQKV_ERR_UNSUPPORTED;
    DeviceInfo dev;
    st = current_device_info(&dev);
    if (st != DIFFQKV_OK) return st;

    PreArgs a;
    a.sub_rows = std::gcd(BN, P);
    auto log2_or_minus1 = [](int v) {
        if (v & (v - 1)) return -1;
        int l = 0;
        while ((1 << l) < v) ++l;
        return l;
    };
    a.sub_shift = log2_or_minus1(a.sub_rows);
    a.page_size = P;
    a.page_shift = log2_or_minus1(P);
    CUtensorMap tm_k, tm_v;
    auto map = [&](CUtensorMap *m, const void *base, int dim, int heads) {
        const uint64_t dims[4] = {(uint64_t)dim, (uint64_t)heads, (uint64_t)P, (uint64_t)cache->num_pages};
        const uint64_t strides[3] = {(uint64_t)dim, (uint64_t)dim * heads, (uint64_t)dim * heads * P};
        const uint32_t box[4] = {(uint32_t)dim, 1, (uint32_t)a.sub_rows, 1};
        return make_tensor_map_u8(m, base, 4, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_NONE,
                                  CU_TENSOR_MAP_L2_PROMOTION_L2_128B);
    };
    st = map(&tm_k, cache->k_pages, d->d_k, d->n_k);
    if (st == DIFFQKV_OK) st = map(&tm_v, cache->v_pages, d->d_v, d->n_v);
    if (st != DIFFQKV_OK) return st;

    uint8_t *ws = static_cast<uint8_t *>(workspace);
    a.q = static_cast<const __nv_bfloat16 *>(q);
    a.k_scales = cache->k_scales;
    a.v_scales = cache->v_scales;
    a.query_start = query_start;
    a.block_table = block_table;
    a.seq_lens = seq_lens;
    a.out = static_cast<__nv_bfloat16 *>(out);
    a.status = reinterpret_cast<int32_t *>(ws);
    a.counters = reinterpret_cast<uint32_t *>(ws + kWsHeader);
    a.partials = reinterpret_cast<float *>(ws + kWsRecords);
    a.batch = d->batch;
    a.n_q = d->n_q;
    a.n_k = d->n_k;
    a.n_v = d->n_v;
    a.tokens = tokens;
    a.t_max = max_blocks * P;
    a.max_blocks = max_blocks;
    a.num_pages = cache->num_pages;
    a.sb = cache->scale_block;
    a.scale_blocks = (long long)cache->num_pages * (P / cache->scale_block);
    a.scale_log2 = (float)((double)d->scale * 1.4426950408889634);
    a.wait_limit_ns = kWaitLimitNs;
    // Units for at most half of the SMs are cut so that every SM has a piece (on the device, which alone knows the lengths:
    // `fewest` and `units` are what their number can be).  Pieces for more than one wave measured no better than whole
    // units, longest first: 409 against 406 us for 384 units of 78 to 250 tiles.
    const long long fewest = ((long long)tokens + kRows - 1) / kRows * d->n_q;
    const int ctas = std::min(dev.num_sms, kSlots);
    a.max_pieces = d->batch <= kCutBatch && fewest * 2 <= ctas ? ctas : 0;
    const unsigned grid = (unsigned)std::max(units, (long long)a.max_pieces);
    int smem = 0;
    PreFn fn = d->d_k == 64 ? (d->d_v == 64 ? plan<64, 64>(&smem) : plan<64, 128>(&smem))
                            : (d->d_v == 64 ? plan<128, 64>(&smem) : plan<128, 128>(&smem));
    if (ensure_dynamic_smem((const void *)fn, smem) != DIFFQKV_OK) return DIFFQKV_ERR_CUDA;
    fn<<<grid, kThreads, smem, stream>>>(tm_k, tm_v, a);
    return cudaGetLastError() == cudaSuccess ? DIFFQKV_OK : DIFFQKV_ERR_CUDA;
}

}  // namespace

}  // namespace diffqkv

extern "C" size_t diffqkv_prefill_paged_kv8_workspace_size(const diffqkv_dims_t *dims) {
    return diffqkv::prefill_kv8_workspace_size(dims);
}

extern "C" diffqkv_status_t diffqkv_prefill_paged_kv8(const diffqkv_dims_t *dims, const diffqkv_kv8_cache_t *cache,
                                                      const void *q, const int32_t *query_start, int32_t tokens,
                                                      const int32_t *block_table, int32_t max_blocks,
                                                      const int32_t *seq_lens, void *out, void *workspace,
                                                      size_t workspace_bytes, diffqkv_stream_t stream) {
    diffqkv::ApiRange nvtx_range("diffqkv_prefill_paged_kv8");
    return diffqkv::prefill_kv8_launch(dims, cache, q, query_start, tokens, block_table, max_blocks, seq_lens, out,
                                       workspace, workspace_bytes, (cudaStream_t)stream);
}
