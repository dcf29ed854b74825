// decode_kv8.cu -- split/combine decode over an 8-bit paged cache (e4m3 codes, a power-of-two scale for each
// block of positions and head), on the tcgen05 tensor cores.
//
//   s_j = scale * log2(e) * 2^ke_j * (q . kc_j),   out = sum_j 2^(s_j - m) 2^ve_j vc_j / sum_j 2^(s_j - m)
//
// with kc_j, vc_j the codes and ke_j, ve_j their blocks' exponents.  The step reads every cached byte once,
// so it is bound by HBM as long as nothing is done per cached element outside the tensor cores: turning
// codes into fp32 on the CUDA cores would take about as many issue slots as the bytes take time.  So
// the codes go from TMA to kind::f8f6f4 MMAs as they are, and it is the small side that is split: a 16-bit query, and
// an fp32 softmax weight w, become three e4m3 terms each,
//   x = t0 + t1 / 32 + t2 / 1024,  t0 = e4m3(x), t1 = e4m3(32 (x - t0)), t2 = e4m3(32 (32 (x - t0) - t1)),
// 12 significant bits (a term has 4 and each remainder is exact in fp32).  With |x| <= 256 the remainders times 32
// stay within 256 again, and what three terms cannot hold of a small x is at most 2^-20, 2^-28 of the largest.  The
// terms are columns of the MMA's N side, whose smallest width, 16, they would not fill otherwise, so they cost
// nothing; their products are added in fp32.
//
//  * S^T = K q^T: M = 128 positions (TMEM lanes), N = the group's query heads x 3 terms.  A softmax thread
//    owns a position: it adds the three columns of a head, applies the block's exponent, and has both the weight of the
//    row sum (2^(s - m)) and that of the output (2^(s + ve - R)) without seeing another position.  The tile's
//    maxima cross the 128 threads by one redux a head and one shared-memory exchange.
//  * O^T = V^T P^T: M = d_v, N = 16 columns of P (the terms of up to five heads), K = 128 positions: V tiles are
//    used as they lie in the cache, positions in rows (an MN-major A operand).
//  * R is the reference of the output's exponent, score and V scale together: the running maximum of a position's score + its
//    block's V exponent, so that weights are at most 2^8 and the largest is that.  (The largest score plus the largest
//    exponent of a tile would bound the weights too, but a block of large scale and little weight would then lift R
//    above every weight and take its bits.)  O is rescaled in TMEM when it grows, a few times a unit.  (A slack that saves
//    rescales would take as many bits from the small weights.)  The row sum needs a reference too, of the score alone; it
//    may lie some way below the largest one, fp32 has the range: R's candidate less the tile's largest V exponent, where
//    the tile's exponents are close together, so that one maximum a head serves both.
//  * work split, ragged batches, ring of TMA stages, partials and the combine by the last CTA of a unit are those of
//    decode.cu.  K tiles and V head tiles have rings of their own (a V slot is one head of one tile: any number of V
//    heads per K head fits), the K tile of the next step is requested before the V tiles of this one.
//  * three warps fetch the tiles' scale bytes (through the block table), each a tile of three, up to three ahead.
//  * rows of a sequence's last tile behind its end are zeroed in shared memory before the MMA reads them: their weights
//    are zero, but the codes there may be NaN.
//  * MMA, commit and TMA are issued by an elected lane (kv8.cuh): behind a test of the lane index the MMA warp alone
//    took longer than a tile's bytes.
// 16 sequences of 32768, 4 K heads of 64 and 16 V heads of 128: 205 us from pages of 16, 5.9 TB/s, 0.91 of the measured
// copy bandwidth; 198 us from pages of 64.  32 query heads over 4 + 16 heads of 64: 3.0 TB/s, 16 + 16 heads of 128: 5.2 TB/s;
// the fewer bytes a tile has for its heads, the more the softmax warps' time shows (about 3400 clocks a tile and CTA, two
// CTAs an SM): exponentials, the e4m3 terms (a conversion of two values takes 4 clocks) and three shared-memory barriers.
// One sequence of 512: 9.4 us, a chain of launch, table, TMA, two MMAs, partials and merge.
#include <math.h>

#include <algorithm>
#include <numeric>

#include "decode_walk.cuh"
#include "internal.h"
#include "kv8.cuh"

namespace diffqkv {

namespace {

constexpr int kTT = 128;              // positions per tile
constexpr int kSoftmaxThreads = 128;  // warps 0-3
constexpr int kMmaWarp = 4, kKWarp = 5, kVWarp = 6, kScaleWarp0 = 7, kScaleWarps = 3;
constexpr int kThreads = 32 * (kScaleWarp0 + kScaleWarps);
constexpr int kMaxVSlots = 12;
constexpr int k_stages(int dk) { return dk == 64 ? 3 : 2; }
constexpr int kGridMax = kWsCounters;  // as in decode.cu: sizes the workspace
constexpr int kPad = 4;                // a partial record: o[d_v], m, l, pad, pad
constexpr float kTop = 8.f;            // weights at the reference are 2^kTop, the largest that split3 takes
constexpr float kMaxSlack = 48.f;      // growth of the row sum's own reference
constexpr int kSpread = 32;            // of a tile's V exponents, for which that reference is taken from R's; together with the
                                       // slack a term of the row sum is at most 2^80, the sum of 2^31 of them below 2^112

struct Kv8Args {
    const __nv_bfloat16 *q;
    const uint8_t *k_scales, *v_scales;
    const int32_t *block_table, *seq_lens;
    __nv_bfloat16 *out;
    float *partials;
    uint32_t *counters;
    int32_t *status;
    int32_t batch, n_q, n_k, n_v, t_max, max_blocks;
    int32_t page_size, page_shift, num_pages, sb, sub_rows, sub_shift;
    int32_t grid, vpg, q_per_v;
    int32_t nb;        // blocks of four heads that one V head's query heads lie in, at most
    int32_t v_slots;
    uint32_t tmem_cols;
    uint32_t off_v, off_p, off_q, off_sc, off_misc;  // shared-memory layout
    uint32_t sc_bytes;                               // of one scale slot
    long long partial_slots, scale_blocks;
    float scale_log2;
    uint64_t wait_limit_ns;
};

__device__ __forceinline__ int div_page(const Kv8Args &a, int x) {
    return a.page_shift >= 0 ? x >> a.page_shift : x / a.page_size;
}

// D[tmem] (+)= A[smem] * B[smem], e4m3 inputs, fp32 accumulate; one thread issues.
__device__ __forceinline__ void umma_e4m3(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Instruction descriptor of kind::f8f6f4 with e4m3 A and B (format 0) and fp32 D.
constexpr uint32_t idesc_e4m3(int M, int N, bool a_mn_major, bool b_mn_major) {
    return (1u << 4) | ((a_mn_major ? 1u : 0u) << 15) | ((b_mn_major ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// Shared-memory descriptor of rows of ROW bytes (64 or 128) in the swizzle of that width; `sbo`: bytes
// between groups of eight rows, `lbo`: bytes between row-wide blocks along M (MN-major operands).
template <int ROW>
__device__ __forceinline__ uint64_t row_desc(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
    static_assert(ROW == 64 || ROW == 128, "swizzle width");
    return (uint64_t)((saddr >> 4) & 0x3fffu) | ((uint64_t)((lbo >> 4) & 0x3fffu) << 16) |
           ((uint64_t)((sbo >> 4) & 0x3fffu) << 32) | (1ull << 46) | ((ROW == 128 ? 2ull : 4ull) << 61);
}

// Shared-memory descriptor of an MN-major operand without swizzle: 16 bytes (along M or N) a row of K, rows one behind
// another; `k_step`: bytes between groups of eight rows, `mn_step`: between 16-byte columns.
__device__ __forceinline__ uint64_t flat_desc(uint32_t saddr, uint32_t k_step, uint32_t mn_step) {
    return (uint64_t)((saddr >> 4) & 0x3fffu) | ((uint64_t)((k_step >> 4) & 0x3fffu) << 16) |
           ((uint64_t)((mn_step >> 4) & 0x3fffu) << 32) | (1ull << 46);
}

// Byte offset of byte c of row r of a swizzled layout.
template <int ROW>
__device__ __forceinline__ uint32_t swizzled(int r, int c) {
    const int x = ROW == 128 ? r & 7 : (r >> 1) & 3;
    return (uint32_t)(r * ROW + (((c >> 4) ^ x) << 4) + (c & 15));
}

// Maximum over the warp (NaN only where every lane has NaN).
__device__ __forceinline__ float warp_max(float x) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
}

// Three e4m3 terms of x and of y (|x|, |y| <= 256): x ~ t0 + t1 / 32 + t2 / 1024, to 12 significant bits or 2^-20.
// x's terms are the low bytes.
__device__ __forceinline__ void split3x2(float x, float y, uint32_t (&t)[3]) {
    float a, b;
    t[0] = e4m3x2(x, y);
    f16x2_to_floats(e4m3x2_to_f16x2(t[0]), a, b);
    x = (x - a) * 32.f;
    y = (y - b) * 32.f;
    t[1] = e4m3x2(x, y);
    f16x2_to_floats(e4m3x2_to_f16x2(t[1]), a, b);
    t[2] = e4m3x2((x - a) * 32.f, (y - b) * 32.f);
}

// Shared-memory bookkeeping behind the tiles.  The MMA warp can be a tile (or unit) ahead of the softmax and the
// softmax two tiles ahead of the MMA warp's waits, so barriers between them alternate: each is completed again
// only after its waiter has passed.
struct Misc {
    uint64_t k_full[3], k_empty[3], v_full[kMaxVSlots], v_empty[kMaxVSlots];
    uint64_t s_full[2], p_full[2], pv_done[2], q_ready[2], sc_full[kScaleWarps], sc_empty[kScaleWarps], mma_done;
    long long scan[4];
    alignas(16) float red[2][4][16];  // [tile parity][warp][head]: maxima
    float l_red[4][16];
    alignas(16) float q_scale[2][16];  // [unit parity][head]: scale * log2(e) * 2^(the query's exponent)
    uint32_t tmem_slot;
    int abort_flag, last_flag;
};

// Query heads of a group lie in blocks of four: head h's terms are columns (h / 4) * 16 + (h % 4) * 3 + term of S, of
// the query operand and of P.  V head v of the group (v0 + v of the cache) multiplies `nb` blocks from this one on:
__device__ __forceinline__ int first_block(const Kv8Args &a, int g, int qpk, int v) {
    const int h0 = max(0, (g * qpk / a.q_per_v + v) * a.q_per_v - g * qpk);  // its first query head in the group
    return min(h0 / 4, (qpk + 3) / 4 - a.nb);
}

template <int DK, int DV, int QPK>
__global__ void __launch_bounds__(kThreads, 2)
    decode_kv8_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                      const Kv8Args a) {
    constexpr int NBLK = (QPK + 3) / 4;  // blocks of four heads
    constexpr int NS = 16 * NBLK;        // S columns
    constexpr int K_TILE = kTT * DK, V_TILE = kTT * DV;
    constexpr int KST = k_stages(DK);
    constexpr uint32_t P_BLOCK = kTT * 16, P_BYTES = NBLK * P_BLOCK;  // a block of P: 16 bytes a position
    constexpr uint32_t Q_BYTES = (NS * DK + 1023) / 1024 * 1024;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = align_smem_1024(smem_raw);
    uint8_t *k_s = smem, *v_s = smem + a.off_v, *p_s = smem + a.off_p, *q_s = smem + a.off_q, *sc_s = smem + a.off_sc;
    Misc &ms = *reinterpret_cast<Misc *>(smem + a.off_misc);
    volatile int *abort_flag = &ms.abort_flag;

    const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
    const long long G = a.grid, c = blockIdx.x;

    if (tid == 0) {
        for (int s = 0; s < KST; ++s) {
            mbar_init(&ms.k_full[s], 1);
            mbar_init(&ms.k_empty[s], 1);
        }
        for (int s = 0; s < a.v_slots; ++s) {
            mbar_init(&ms.v_full[s], 1);
            mbar_init(&ms.v_empty[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&ms.s_full[s], 1);
            mbar_init(&ms.p_full[s], 4);
            mbar_init(&ms.pv_done[s], 1);
            mbar_init(&ms.q_ready[s], 1);
        }
        for (int s = 0; s < kScaleWarps; ++s) {
            mbar_init(&ms.sc_full[s], 1);
            mbar_init(&ms.sc_empty[s], 4);
        }
        mbar_init(&ms.mma_done, 1);
        ms.abort_flag = 0;
        ms.last_flag = 0;
        fence_barrier_init();
    }
    if (warp == kKWarp && lane == 0) prefetch_tensormap(&tm_k);
    if (warp == kVWarp && lane == 0) prefetch_tensormap(&tm_v);
    if (warp == 0) walker_scan<kTT>(a, c, G, lane, ms.scan);
    if (warp == kMmaWarp) {
        tmem_alloc(&ms.tmem_slot, a.tmem_cols);
        tmem_relinquish();
    }
    // unused columns of P and of the queries are operands too: start them from zero
    for (uint32_t i = tid * 16; i < 2 * (P_BYTES + Q_BYTES); i += kThreads * 16)
        *reinterpret_cast<uint4 *>(p_s + i) = make_uint4(0, 0, 0, 0);  // (the q buffers follow the P buffers)
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = (uint32_t)uniform((int)ms.tmem_slot);

    const long long N = ms.scan[0];
    // sequences without positions: zero rows, dealt out over the CTAs
    for (int b = (int)c; b < a.batch; b += (int)G)
        if (clamp_len(__ldg(a.seq_lens + b), a.t_max) == 0) {
            uint4 *o = reinterpret_cast<uint4 *>(a.out + (size_t)b * a.n_q * DV);
            for (int e = tid; e < a.n_q * DV / 8; e += kThreads) o[e] = make_uint4(0, 0, 0, 0);
        }
    const long long Ge = N < G ? N : G;  // CTAs that own tiles
    const long long t_begin = c < Ge ? c * N / Ge : 0;
    const int n_tiles = uniform(c < Ge ? (int)((c + 1) * N / Ge - t_begin) : 0);

    Walker w;
    w.b = (int)(ms.scan[2] >> 32);
    w.g = (int)(ms.scan[2] & 0xffffffff);
    w.i = (int)ms.scan[3];
    w.P = ms.scan[1];
    w.T = n_tiles ? clamp_len(__ldg(a.seq_lens + w.b), a.t_max) : 0;
    w.nt = (w.T + kTT - 1) / kTT;

    if (warp == kKWarp || warp == kVWarp) {
        // ======================= TMA producers of the two rings: sub-boxes of sub_rows positions inside one page; lane f
        // holds the pool page of sub-box f, fetched a tile ahead
        const bool is_k = warp == kKWarp;
        uint64_t *full = is_k ? ms.k_full : ms.v_full, *empty = is_k ? ms.k_empty : ms.v_empty;
        uint8_t *ring = is_k ? k_s : v_s;
        const CUtensorMap *map = is_k ? &tm_k : &tm_v;
        const int slots = is_k ? KST : a.v_slots, heads = is_k ? 1 : a.vpg;
        const int tile_bytes = is_k ? K_TILE : V_TILE, box_bytes = a.sub_rows * (is_k ? DK : DV);
        auto subs = [&](const Walker &x) {
            const int v = min(kTT, x.T - x.i * kTT) + a.sub_rows - 1;
            return a.sub_shift >= 0 ? v >> a.sub_shift : v / a.sub_rows;
        };
        auto entry = [&](const Walker &x) {
            return lane < subs(x)
                       ? __ldg(a.block_table + (size_t)x.b * a.max_blocks + div_page(a, x.i * kTT + lane * a.sub_rows))
                       : 0;
        };
        int next = n_tiles ? entry(w) : 0;
        int slot = 0, issued = 0;
        uint32_t par = 0;
        for (int k = 0; k < n_tiles; ++k) {
            int page = next;
            if (page < 0 || page >= a.num_pages) {  // a bad entry loads pool page 0: the loads stay in bounds
                if (is_k) record_error(a.status, DIFFQKV_ERR_DEVICE_PAGE);
                page = 0;
            }
            const int n = uniform(subs(w));
            const int h0 = uniform(is_k ? w.g : w.g * QPK / a.q_per_v), last = is_k ? a.n_k - 1 : a.n_v - 1;
            const int p = w.i * kTT + lane * a.sub_rows;
            const int row = p - div_page(a, p) * a.page_size;
            walker_advance<kTT>(w, a);
            if (k + 1 < n_tiles) next = entry(w);
            for (int v = 0; v < heads; ++v) {
                if (issued >= slots) mbar_wait_bounded(&empty[slot], par ^ 1u, a.wait_limit_ns, abort_flag, a.status);
                if (__any_sync(0xffffffffu, *abort_flag != 0)) {
                    k = n_tiles;
                    break;
                }
                if (elect_one()) mbar_arrive_expect_tx(&full[slot], (uint32_t)(n * box_bytes));
                __syncwarp();
                // a group at the end may span fewer V heads than the widest one: the last is loaded again
                const int head = min(h0 + v, last);
                uint8_t *dst = ring + slot * tile_bytes;
#pragma unroll 4
                for (int f = 0; f < n; ++f) {
                    const int row_f = __shfl_sync(0xffffffffu, row, f), page_f = __shfl_sync(0xffffffffu, page, f);
                    if (elect_one()) tma_load_4d(dst + f * box_bytes, map, &full[slot], 0, head, row_f, page_f);
                }
                __syncwarp();
                ++issued;
                if (++slot == slots) {
                    slot = 0;
                    par ^= 1u;
                }
            }
        }
        // drain: no copy may still be landing when the CTA exits
        for (int k = max(0, issued - slots); k < issued; ++k)
            mbar_wait_bounded(&full[k % slots], (uint32_t)(k / slots & 1), a.wait_limit_ns, nullptr, a.status);
    } else if (warp == kMmaWarp) {
        // ======================= queries into terms, MMA issue
        // descriptors of the first slots; a slot, buffer or K step further is an addition in their address field
        const uint64_t k_desc = row_desc<DK>(smem_addr(k_s), 16, 8 * DK), q_desc = row_desc<DK>(smem_addr(q_s), 16, 8 * DK);
        // d_v = 64: both halves of the 128 lanes read the one 64-wide block (lbo 0)
        const uint64_t v_desc = row_desc<DV>(smem_addr(v_s), 0, 8 * DV), p_desc = flat_desc(smem_addr(p_s), 128, P_BLOCK);
        constexpr uint32_t idesc_s = idesc_e4m3(kTT, NS, false, false);
        const uint32_t idesc_o = idesc_e4m3(128, 16 * a.nb, true, true);
        const uint32_t t_o = tmem + 2 * NS;
        Walker wk = w;      // tile whose S is issued next
        int unit = -1;      // its unit, counted from 0
        int ks = 0, vs = 0;
        uint32_t kp = 0, vp = 0;
        auto issue_s = [&](int k) {
            if (k == 0 || wk.i == 0) {
                ++unit;
                uint8_t *qb = q_s + (unit & 1) * Q_BYTES;
                constexpr int V = DK / 32;
                // amax of every head, its power-of-two scale (largest element into [128, 256)), and the three terms
#pragma unroll (QPK < 4 ? QPK : 4)
                for (int h = 0; h < QPK; ++h) {
                    const long long row = (long long)wk.b * a.n_q + wk.g * QPK + h;
                    uint32_t x[V / 2];
#pragma unroll
                    for (int e = 0; e < V / 2; ++e)
                        x[e] = in_bounds(row, (long long)a.batch * a.n_q, a.status)
                                   ? __ldg(reinterpret_cast<const uint32_t *>(a.q + row * DK) + lane * (V / 2) + e)
                                   : 0u;
                    uint32_t m = 0;
#pragma unroll
                    for (int e = 0; e < V / 2; ++e) m = max(m, max(x[e] & 0x7fffu, (x[e] >> 16) & 0x7fffu));
                    m = __reduce_max_sync(0xffffffffu, m);
                    const int se = min(134 - (int)(m >> 7), 126);
                    const float f = exp2_int(max(se, -126));
                    uint32_t t[3] = {0, 0, 0};
#pragma unroll
                    for (int e = 0; e < V / 2; ++e) {
                        uint32_t b[3];
                        split3x2(bf16lo(x[e]) * f, bf16hi(x[e]) * f, b);
#pragma unroll
                        for (int i = 0; i < 3; ++i) t[i] |= b[i] << (16 * e);
                    }
#pragma unroll
                    for (int i = 0; i < 3; ++i) {
                        uint8_t *dst = qb + swizzled<DK>(h / 4 * 16 + h % 4 * 3 + i, lane * V);
                        if constexpr (V == 2)
                            *reinterpret_cast<uint16_t *>(dst) = (uint16_t)t[i];
                        else
                            *reinterpret_cast<uint32_t *>(dst) = t[i];
                    }
                    // a query with infinities or NaN has no scale: every score of the head becomes NaN
                    if (lane == 0)
                        ms.q_scale[unit & 1][h] = m >= 0x7f80u ? __int_as_float(0x7fffffff)
                                                               : a.scale_log2 * exp2_int(min(max(-se, -126), 127));
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive(&ms.q_ready[unit & 1]);
            }
            mbar_wait_bounded(&ms.k_full[ks], kp, a.wait_limit_ns, abort_flag, a.status);
            tc_fence_after();
            const uint64_t kd = k_desc + (uint32_t)(ks * (K_TILE >> 4));
            const uint64_t qd = q_desc + (uint32_t)uniform(unit & 1) * (Q_BYTES >> 4);
            const uint32_t t_s = tmem + (uint32_t)((k & 1) * NS);
            if (elect_one()) {
#pragma unroll
                for (int s = 0; s < DK / 32; ++s) umma_e4m3(t_s, kd + s * 2, qd + s * 2, idesc_s, s > 0 ? 1u : 0u);
                umma_commit(&ms.s_full[k & 1]);
                umma_commit(&ms.k_empty[ks]);
            }
            __syncwarp();
            if (++ks == KST) {
                ks = 0;
                kp ^= 1u;
            }
            walker_advance<kTT>(wk, a);
        };
        if (n_tiles > 0) issue_s(0);
        for (int k = 0; k < n_tiles; ++k) {
            // S(k + 1) goes to the buffer that the softmax was done with before p_full(k - 1)
            if (k + 1 < n_tiles) issue_s(k + 1);
            mbar_wait_bounded(&ms.p_full[k & 1], (uint32_t)(k >> 1 & 1), a.wait_limit_ns, abort_flag, a.status);
            tc_fence_after();
            const int valid = min(kTT, w.T - w.i * kTT);
            const uint32_t onto = (uint32_t)uniform(k != 0 && w.i != 0);  // 0: the unit's first tile starts O
            const uint64_t p_buf = p_desc + (uint32_t)((k & 1) * (P_BYTES >> 4));
            uint32_t t_v = t_o;
            for (int v = 0; v < a.vpg; ++v) {
                mbar_wait_bounded(&ms.v_full[vs], vp, a.wait_limit_ns, abort_flag, a.status);
                if (valid < kTT) {
                    // rows behind the sequence (a row's swizzle stays inside the row)
                    uint4 *z = reinterpret_cast<uint4 *>(v_s + vs * V_TILE + valid * DV);
                    for (int e = lane; e < (kTT - valid) * DV / 16; e += 32) z[e] = make_uint4(0, 0, 0, 0);
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                }
                tc_fence_after();
                const uint64_t vd = v_desc + (uint32_t)(vs * (V_TILE >> 4));
                uint64_t pd = p_buf;
                if constexpr (NBLK > 1) pd += (uint32_t)(uniform(first_block(a, w.g, QPK, v)) * (int)(P_BLOCK >> 4));
                if (elect_one()) {
#pragma unroll
                    for (int s = 0; s < kTT / 32; ++s)
                        umma_e4m3(t_v, vd + s * (32 * DV >> 4), pd + s * (32 * 16 >> 4), idesc_o, s > 0 ? 1u : onto);
                    umma_commit(&ms.v_empty[vs]);
                }
                __syncwarp();
                t_v += (uint32_t)(16 * a.nb);
                if (++vs == a.v_slots) {
                    vs = 0;
                    vp ^= 1u;
                }
            }
            if (elect_one()) umma_commit(&ms.pv_done[k & 1]);
            __syncwarp();
            walker_advance<kTT>(w, a);
        }
        if (n_tiles > 0) {
            if (elect_one()) umma_commit(&ms.mma_done);
            __syncwarp();
            mbar_wait_bounded(&ms.mma_done, 0, a.wait_limit_ns, nullptr, a.status);
        }
    } else if (warp >= kScaleWarp0) {
        // ======================= scale bytes: warp j fetches those of tiles j, j + kScaleWarps, ... into slot j
        const int j = warp - kScaleWarp0;
        int8_t *ke = reinterpret_cast<int8_t *>(sc_s + j * a.sc_bytes);  // [128] K exponents, then [vpg][128] of V
        int8_t *ve = ke + kTT;
        int2 *v_range = reinterpret_cast<int2 *>(sc_s + j * a.sc_bytes + kTT * (1 + a.vpg));  // largest and least of each
        for (int s = 0; s < j && s < n_tiles; ++s) walker_advance<kTT>(w, a);
        uint32_t par = 0;
        const int per_page = a.page_size / a.sb;
        for (int k = j; k < n_tiles; k += kScaleWarps) {
            if (k >= kScaleWarps) mbar_wait_bounded(&ms.sc_empty[j], par ^ 1u, a.wait_limit_ns, abort_flag, a.status);
            const int valid = min(kTT, w.T - w.i * kTT), v0 = w.g * QPK / a.q_per_v;
            long long blk[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int t = lane + 32 * e, p = w.i * kTT + min(t, valid - 1);
                const int lp = div_page(a, p);
                const int page = __ldg(a.block_table + (size_t)w.b * a.max_blocks + lp);
                blk[e] = (long long)(page >= 0 && page < a.num_pages ? page : 0) * per_page + (p - lp * a.page_size) / a.sb;
                if (!in_bounds(blk[e], a.scale_blocks, a.status)) blk[e] = 0;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) ke[lane + 32 * e] = (int8_t)kv8_exp(__ldg(a.k_scales + blk[e] * a.n_k + w.g));
            for (int v = 0; v < a.vpg; ++v) {
                int m = kKv8MinExp, lo = kKv8MaxExp;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int x = kv8_exp(__ldg(a.v_scales + blk[e] * a.n_v + min(v0 + v, a.n_v - 1)));
                    ve[v * kTT + lane + 32 * e] = (int8_t)x;
                    m = max(m, x);
                    lo = min(lo, x);
                }
                m = __reduce_max_sync(0xffffffffu, m);
                lo = __reduce_min_sync(0xffffffffu, lo);
                if (lane == 0) v_range[v] = make_int2(m, lo);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&ms.sc_full[j]);
            par ^= 1u;
#pragma unroll 1
            for (int s = 0; s < kScaleWarps && k + s + 1 < n_tiles; ++s) walker_advance<kTT>(w, a);
        }
    } else {
        // ======================= softmax: thread tid owns position tid of a tile (TMEM lane tid)
        const uint32_t lane_base = (uint32_t)(warp * 32) << 16;
        const uint32_t t_s = tmem + lane_base, t_o = tmem + 2 * NS + lane_base;
        auto o_column = [&](int h, int v, int g) {  // head h's first column of O, its V head being v
            return (v * a.nb + h / 4 - first_block(a, g, QPK, v)) * 16 + h % 4 * 3;
        };
        float l[QPK];                    // this position's share of the row sums
        float m_ref = 0.f, R = 0.f;      // lane h: head h's references, R less kTop (the same in the four warps)
        uint32_t vls[(QPK + 7) / 8] = {};  // V head of each query head inside the group, four bits each
        auto vl = [&](int h) { return (int)(vls[h >> 3] >> (4 * (h & 7)) & 15u); };
        int unit = -1, my_vl = 0;        // (lane h's own)
        for (int k = 0; k < n_tiles; ++k) {
            const bool start = k == 0 || w.i == 0;
            const int slot = k % kScaleWarps;
            if (start) {
                ++unit;
                mbar_wait_bounded(&ms.q_ready[unit & 1], (uint32_t)(unit >> 1 & 1), a.wait_limit_ns, abort_flag, a.status);
                // (a division a lane instead of one a head)
                const int mine = lane < QPK ? (w.g * QPK + lane) / a.q_per_v - w.g * QPK / a.q_per_v : 0;
                my_vl = mine;
#pragma unroll
                for (int i = 0; i < (QPK + 7) / 8; ++i) {
                    vls[i] = 0;
#pragma unroll
                    for (int h = 8 * i; h < QPK && h < 8 * i + 8; ++h)
                        vls[i] |= (uint32_t)__shfl_sync(0xffffffffu, mine, h) << (4 * (h & 7));
                }
#pragma unroll
                for (int h = 0; h < QPK; ++h) l[h] = 0.f;
            }
            const int valid = min(kTT, w.T - w.i * kTT);
            mbar_wait_bounded(&ms.sc_full[slot], (uint32_t)(k / kScaleWarps & 1), a.wait_limit_ns, abort_flag, a.status);
            const int8_t *ke = reinterpret_cast<const int8_t *>(sc_s + slot * a.sc_bytes);
            const int8_t *ve = ke + kTT;
            const float kf = exp2_int(ke[tid]);
            float vx[QPK];
#pragma unroll
            for (int h = 0; h < QPK; ++h) vx[h] = (float)ve[vl(h) * kTT + tid];
            const int2 v_range = reinterpret_cast<const int2 *>(sc_s + slot * a.sc_bytes + kTT * (1 + a.vpg))[my_vl];
            mbar_wait_bounded(&ms.s_full[k & 1], (uint32_t)(k >> 1 & 1), a.wait_limit_ns, abort_flag, a.status);
            tc_fence_after();
            float s[QPK];
            {
                uint32_t r[NBLK][16];
#pragma unroll
                for (int i = 0; i < NBLK; ++i) tmem_ld_cols<16>(t_s + (uint32_t)((k & 1) * NS + i * 16), r[i]);
                tmem_wait_ld();
#pragma unroll
                for (int h = 0; h < QPK; ++h) {
                    auto col = [&](int i) { return __uint_as_float(r[h / 4][h % 4 * 3 + i]); };
                    const float x = fmaf(fmaf(col(2), 0.03125f, col(1)), 0.03125f, col(0));
                    s[h] = tid < valid ? x * (ms.q_scale[unit & 1][h] * kf) : -INFINITY;
                }
            }
            // vx: the logarithm of the whole weight, V scale included
#pragma unroll
            for (int h = 0; h < QPK; ++h) vx[h] += s[h];
            // a tile's maxima: across the warp by redux, across the warps through shared memory
            auto tile_max = [&](const float(&x)[QPK]) {
                float m[QPK];
#pragma unroll
                for (int h = 0; h < QPK; ++h) m[h] = warp_max(x[h]);
                if (lane == 0) {
#pragma unroll
                    for (int h = 0; h < QPK; h += 4) {
                        if constexpr (QPK >= 4)
                            *reinterpret_cast<float4 *>(&ms.red[k & 1][warp][h]) =
                                make_float4(m[h], m[h + 1], m[h + 2], m[h + 3]);
                        else
#pragma unroll
                            for (int e = 0; e < QPK; ++e) ms.red[k & 1][warp][e] = m[e];
                    }
                }
                named_barrier(1, kSoftmaxThreads);
                const int h = lane < QPK ? lane : 0;
                return fmaxf(fmax3f(ms.red[k & 1][0][h], ms.red[k & 1][1][h], ms.red[k & 1][2][h]), ms.red[k & 1][3][h]);
            };
            // lane h moves head h's references where the tile exceeds them
            float alpha = 1.f, l_scale = 1.f;
            {
                const float top = tile_max(vx);
                const float r_new = (top == -INFINITY ? (float)v_range.x : top) - kTop;
                float m_new = r_new + (kTop - (float)v_range.x);
                // (the same in all four warps) exponents too far apart for that: the scores' own maximum
                if (__any_sync(0xffffffffu, lane < QPK && v_range.x - v_range.y > kSpread)) {
                    named_barrier(1, kSoftmaxThreads);  // every warp has read the maxima
                    const float m = tile_max(s);
                    m_new = m == -INFINITY ? 0.f : m;
                }
                if (start) {
                    m_ref = m_new;
                    R = r_new;
                } else if (r_new > R || m_new > m_ref + kMaxSlack) {
                    const float r2 = fmaxf(r_new, R), m2 = fmaxf(m_new, m_ref);
                    alpha = fast_exp2(R - r2);
                    l_scale = fast_exp2(m_ref - m2);
                    R = r2;
                    m_ref = m2;
                }
            }
            if (__any_sync(0xffffffffu, alpha != 1.f || l_scale != 1.f)) {
                // (the same in all four warps) O is final for tile k - 1, then the heads' columns are rescaled
                mbar_wait_bounded(&ms.pv_done[(k - 1) & 1], (uint32_t)((k - 1) >> 1 & 1), a.wait_limit_ns, abort_flag,
                                  a.status);
                tc_fence_after();
#pragma unroll
                for (int h = 0; h < QPK; ++h) l[h] *= __shfl_sync(0xffffffffu, l_scale, h);
#pragma unroll 1
                for (int h = 0; h < QPK; ++h) {
                    const float f = __shfl_sync(0xffffffffu, alpha, h);
                    const int v = __shfl_sync(0xffffffffu, my_vl, h);
                    if (f == 1.f) continue;
                    const uint32_t at = t_o + (uint32_t)o_column(h, v, w.g);
                    uint32_t r[2], r2[1];
                    tmem_ld_cols<2>(at, r);
                    tmem_ld_cols<1>(at + 2, r2);
                    tmem_wait_ld();
                    r[0] = __float_as_uint(__uint_as_float(r[0]) * f);
                    r[1] = __float_as_uint(__uint_as_float(r[1]) * f);
                    r2[0] = __float_as_uint(__uint_as_float(r2[0]) * f);
                    tmem_st_cols<2>(at, r);
                    tmem_st_cols<1>(at + 2, r2);
                }
                tmem_wait_st();
            }
            uint4 pk[NBLK];  // this position's row of each block: terms of heads 4 i, 4 i + 1, ... in bytes 0 .. 11
#pragma unroll
            for (int i = 0; i < NBLK; ++i) {
                uint32_t t[2][3] = {{0, 0, 0}, {0, 0, 0}};
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int h0 = 4 * i + 2 * j, h1 = h0 + 1 < QPK ? h0 + 1 : h0;
                    if (h0 >= QPK) continue;
                    const float m0 = __shfl_sync(0xffffffffu, m_ref, h0), r0 = __shfl_sync(0xffffffffu, R, h0);
                    const float m1 = __shfl_sync(0xffffffffu, m_ref, h1), r1 = __shfl_sync(0xffffffffu, R, h1);
                    l[h0] += fast_exp2(s[h0] - m0);
                    if (h1 > h0) l[h1] += fast_exp2(s[h1] - m1);
                    split3x2(fast_exp2(vx[h0] - r0), fast_exp2(vx[h1] - r1), t[j]);
                }
                // (t[j][i]: term i of heads 2 j and 2 j + 1 of the block)  head 0: bytes 0-2, head 1: 3-5, head 2: 6-8, ...
                pk[i].x = (t[0][0] & 0xffu) | (t[0][1] & 0xffu) << 8 | (t[0][2] & 0xffu) << 16 | (t[0][0] >> 8) << 24;
                pk[i].y = (t[0][1] >> 8) | (t[0][2] >> 8) << 8 | (t[1][0] & 0xffu) << 16 | (t[1][1] & 0xffu) << 24;
                pk[i].z = (t[1][2] & 0xffu) | (t[1][0] >> 8) << 8 | (t[1][1] >> 8) << 16 | (t[1][2] >> 8) << 24;
                pk[i].w = 0u;
            }
            // the P buffer was read by the P.V of tile k - 2
            if (k >= 2)
                mbar_wait_bounded(&ms.pv_done[k & 1], (uint32_t)((k >> 1) - 1 & 1), a.wait_limit_ns, abort_flag, a.status);
            uint4 *pb = reinterpret_cast<uint4 *>(p_s + (k & 1) * P_BYTES) + tid;
#pragma unroll
            for (int i = 0; i < NBLK; ++i) pb[i * kTT] = pk[i];
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&ms.p_full[k & 1]);
                mbar_arrive(&ms.sc_empty[slot]);
            }

            // ---- end of this CTA's piece of the unit: its partial, and the combine if it is the last
            if (w.i == w.nt - 1 || k == n_tiles - 1) {
#pragma unroll
                for (int h = 0; h < QPK; ++h) {
#pragma unroll
                    for (int off = 16; off >= 1; off >>= 1) l[h] += __shfl_xor_sync(0xffffffffu, l[h], off);
                    if (lane == 0) ms.l_red[warp][h] = l[h];
                }
                named_barrier(1, kSoftmaxThreads);
                mbar_wait_bounded(&ms.pv_done[k & 1], (uint32_t)(k >> 1 & 1), a.wait_limit_ns, abort_flag, a.status);
                tc_fence_after();
                const long long u = (long long)w.b * a.n_k + w.g;
                const long long first = cta_of_tile(w.P, N, Ge), last = cta_of_tile(w.P + w.nt - 1, N, Ge);
                const bool whole = first == last;  // no other CTA has a piece: straight to the output
                const long long counter = counter_of(u, first, (long long)a.batch * a.n_k, kWsCounters);
                const bool slot_ok = in_bounds(u + c, a.partial_slots, a.status);
#pragma unroll 1
                for (int h = 0; h < QPK; ++h) {
                    uint32_t r[4];
                    tmem_ld_cols<4>(t_o + (uint32_t)o_column(h, __shfl_sync(0xffffffffu, my_vl, h), w.g), r);
                    tmem_wait_ld();
                    const float o = fmaf(fmaf(__uint_as_float(r[2]), 0.03125f, __uint_as_float(r[1])), 0.03125f,
                                         __uint_as_float(r[0]));
                    const float m_h = __shfl_sync(0xffffffffu, m_ref, h), r_h = __shfl_sync(0xffffffffu, R, h);
                    const float l_h = ms.l_red[0][h] + ms.l_red[1][h] + ms.l_red[2][h] + ms.l_red[3][h];
                    const float o_rel = o * exp2f(r_h - m_h);  // relative to 2^m
                    if (whole) {
                        const long long row = (long long)w.b * a.n_q + w.g * QPK + h;
                        if (tid < DV && in_bounds(row, (long long)a.batch * a.n_q, a.status))
                            a.out[row * DV + tid] = __float2bfloat16_rn(o_rel / l_h);
                    } else if (slot_ok) {
                        float *dst = a.partials + ((size_t)(u + c) * QPK + h) * (DV + kPad);
                        if (tid < DV) __stcg(dst + tid, o_rel);
                        if (tid == 0) {
                            __stcg(dst + DV, m_h);
                            __stcg(dst + DV + 1, l_h);
                        }
                    }
                }
                if (whole) {
                    tc_fence_before();
                    named_barrier(1, kSoftmaxThreads);  // l_red is written again by the next unit
                    walker_advance<kTT>(w, a);
                    continue;
                }
                tc_fence_before();
                __threadfence();
                named_barrier(1, kSoftmaxThreads);
                if (tid == 0) {
                    const unsigned old = in_bounds(counter, kWsCounters, a.status) ? atomicAdd(a.counters + counter, 1u) : 0u;
                    ms.last_flag = old == (unsigned)(last - first) ? 1 : 0;
                }
                named_barrier(1, kSoftmaxThreads);
                if (*(volatile int *)&ms.last_flag) {
                    __threadfence();
                    const bool ok = in_bounds(u + last, a.partial_slots, a.status);
                    for (int it = tid; it < QPK * (DV / 4) && ok; it += kSoftmaxThreads) {
                        const int h2 = it / (DV / 4), d4 = it % (DV / 4);
                        auto rec = [&](long long cc) {
                            return a.partials + ((size_t)(u + cc) * QPK + h2) * (DV + kPad);
                        };
                        // records four at a time; the maximum first, unless four are all
                        float M = -INFINITY, L = 0.f;
                        if (last - first >= 4)
                            for (long long c0 = first; c0 <= last; c0 += 8) {
                                float mv[8];
#pragma unroll
                                for (int e = 0; e < 8; ++e) mv[e] = c0 + e <= last ? __ldcg(rec(c0 + e) + DV) : -INFINITY;
#pragma unroll
                                for (int e = 0; e < 8; ++e) M = fmaxf(M, mv[e]);
                            }
                        float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
                        for (long long c0 = first; c0 <= last; c0 += 4) {
                            float2 ml[4];
                            float4 xv[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                ml[e] = make_float2(-INFINITY, 0.f);
                                if (c0 + e <= last) {
                                    ml[e] = __ldcg(reinterpret_cast<const float2 *>(rec(c0 + e) + DV));
                                    xv[e] = __ldcg(reinterpret_cast<const float4 *>(rec(c0 + e)) + d4);
                                }
                            }
                            if (last - first < 4) M = fmaxf(fmaxf(ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x));
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                if (c0 + e > last) break;
                                const float f = fast_exp2(ml[e].x - M);
                                L = fmaf(f, ml[e].y, L);
                                O.x = fmaf(f, xv[e].x, O.x);
                                O.y = fmaf(f, xv[e].y, O.y);
                                O.z = fmaf(f, xv[e].z, O.z);
                                O.w = fmaf(f, xv[e].w, O.w);
                            }
                        }
                        const float inv = 1.f / L;  // L > 0: every piece has a position
                        const long long row = (long long)w.b * a.n_q + w.g * QPK + h2;
                        if (in_bounds(row, (long long)a.batch * a.n_q, a.status))
                            *reinterpret_cast<uint2 *>(a.out + row * DV + d4 * 4) =
                                make_uint2(pack_bf16x2(O.x * inv, O.y * inv), pack_bf16x2(O.z * inv, O.w * inv));
                    }
                    if (tid == 0) a.counters[counter] = 0u;
                }
                named_barrier(1, kSoftmaxThreads);
            }
            walker_advance<kTT>(w, a);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, a.tmem_cols);
    }
}

// ------------------------------------------------------------------ host side

using Kv8Fn = void (*)(CUtensorMap, CUtensorMap, Kv8Args);

template <int DK, int DV>
Kv8Fn pick_qpk(int qpk) {
    switch (qpk) {
        case 1: return decode_kv8_kernel<DK, DV, 1>;
        case 2: return decode_kv8_kernel<DK, DV, 2>;
        case 4: return decode_kv8_kernel<DK, DV, 4>;
        case 8: return decode_kv8_kernel<DK, DV, 8>;
        case 16: return decode_kv8_kernel<DK, DV, 16>;
        default: return nullptr;
    }
}

Kv8Fn pick(const diffqkv_dims_t *d) {
    const int qpk = d->n_q / d->n_k;
    if (d->d_k == 64) return d->d_v == 64 ? pick_qpk<64, 64>(qpk) : pick_qpk<64, 128>(qpk);
    return d->d_v == 64 ? pick_qpk<128, 64>(qpk) : pick_qpk<128, 128>(qpk);
}

uint32_t align_to(uint32_t x, uint32_t n) { return (x + n - 1) / n * n; }

int log2_or_minus1(int v) {
    if (v & (v - 1)) return -1;
    int l = 0;
    while ((1 << l) < v) ++l;
    return l;
}

diffqkv_status_t decode_kv8_launch(const diffqkv_dims_t *d, const diffqkv_kv8_cache_t *cache, const void *q,
                                   const int32_t *block_table, int32_t max_blocks, const int32_t *seq_lens,
                                   int32_t max_seq_len, void *out, void *workspace, size_t workspace_bytes,
                                   cudaStream_t stream) {
    diffqkv_status_t st = validate_kv8(d, cache);
    if (st != DIFFQKV_OK) return st;
    if (!q || !block_table || !seq_lens || !out || max_blocks < 1) return DIFFQKV_ERR_INVALID_ARG;
    const int P = cache->page_size;
    if ((long long)max_blocks * P > 0x7fffffffLL) return DIFFQKV_ERR_INVALID_ARG;
    Kv8Fn fn = pick(d);
    if (!fn) return DIFFQKV_ERR_UNSUPPORTED;
    if (!aligned16(q) || !aligned16(out) || (reinterpret_cast<uintptr_t>(seq_lens) & 3u) ||
        (reinterpret_cast<uintptr_t>(block_table) & 3u))
        return DIFFQKV_ERR_MISALIGNED;
    if (!workspace || workspace_bytes < decode_workspace_size(d)) return DIFFQKV_ERR_WORKSPACE;
    if (!aligned16(workspace)) return DIFFQKV_ERR_MISALIGNED;
    DeviceInfo dev;
    st = current_device_info(&dev);
    if (st != DIFFQKV_OK) return st;

    Kv8Args a;
    const int qpk = d->n_q / d->n_k, qpv = d->n_q / d->n_v;
    int span = 1;
    a.nb = 1;
    for (int g = 0; g < d->n_k; ++g) {
        const int v0 = g * qpk / qpv, v1 = ((g + 1) * qpk - 1) / qpv;
        span = std::max(span, v1 - v0 + 1);
        for (int v = v0; v <= v1; ++v) {
            const int h0 = std::max(0, v * qpv - g * qpk), h1 = std::min(qpk, (v + 1) * qpv - g * qpk) - 1;
            a.nb = std::max(a.nb, h1 / 4 - h0 / 4 + 1);
        }
    }
    a.vpg = span;
    a.q_per_v = qpv;
    const int ns = (qpk + 3) / 4 * 16, cols = 2 * ns + span * a.nb * 16;
    a.tmem_cols = 32;
    while ((int)a.tmem_cols < cols) a.tmem_cols *= 2;
    if (a.tmem_cols > 512) return DIFFQKV_ERR_UNSUPPORTED;
    // two CTAs a SM, so that one's latencies (barriers, TMEM, conversions) hide behind the other's; one where TMEM does
    // not hold two
    const int per_sm = a.tmem_cols > 256 ? 1 : 2;

    // shared memory: K ring, V ring (what is left, at most kMaxVSlots slots), P and q buffers, scales, bookkeeping
    const uint32_t v_tile = (uint32_t)(kTT * d->d_v);
    const uint32_t p_bytes = (uint32_t)(ns * kTT), q_bytes = align_to((uint32_t)(ns * d->d_k), 1024);
    a.off_v = (uint32_t)(k_stages(d->d_k) * kTT * d->d_k);
    a.sc_bytes = align_to((uint32_t)(kTT * (1 + span) + 8 * span), 16);
    const uint32_t tail = 2 * p_bytes + 2 * q_bytes + kScaleWarps * a.sc_bytes + align_to((uint32_t)sizeof(Misc), 16);
    const uint32_t room = (per_sm == 2 ? 113u : 227u) * 1024 - 1024 - a.off_v - tail;
    a.v_slots = std::min<int>(kMaxVSlots, (int)(room / v_tile));
    if (a.v_slots < 2) return DIFFQKV_ERR_UNSUPPORTED;
    a.off_p = a.off_v + (uint32_t)a.v_slots * v_tile;
    a.off_q = a.off_p + 2 * p_bytes;
    a.off_sc = a.off_q + 2 * q_bytes;
    a.off_misc = a.off_sc + kScaleWarps * a.sc_bytes;
    const uint32_t smem = a.off_p + tail + 1024;

    a.sub_rows = std::gcd(kTT, P);
    a.sub_shift = log2_or_minus1(a.sub_rows);
    a.page_size = P;
    a.page_shift = log2_or_minus1(P);
    CUtensorMap tm_k, tm_v;
    auto map = [&](CUtensorMap *m, const void *base, int dim, int heads) {
        const uint64_t dims[4] = {(uint64_t)dim, (uint64_t)heads, (uint64_t)P, (uint64_t)cache->num_pages};
        const uint64_t strides[3] = {(uint64_t)dim, (uint64_t)dim * heads, (uint64_t)dim * heads * P};
        const uint32_t box[4] = {(uint32_t)dim, 1, (uint32_t)a.sub_rows, 1};
        return make_tensor_map_u8(m, base, 4, dims, strides, box,
                                  dim == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                                  dim == 128 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_64B);
    };
    st = map(&tm_k, cache->k_pages, d->d_k, d->n_k);
    if (st == DIFFQKV_OK) st = map(&tm_v, cache->v_pages, d->d_v, d->n_v);
    if (st != DIFFQKV_OK) return st;

    uint8_t *ws = static_cast<uint8_t *>(workspace);
    const size_t units = (size_t)d->batch * d->n_k;
    a.q = static_cast<const __nv_bfloat16 *>(q);
    a.k_scales = cache->k_scales;
    a.v_scales = cache->v_scales;
    a.block_table = block_table;
    a.seq_lens = seq_lens;
    a.out = static_cast<__nv_bfloat16 *>(out);
    a.counters = reinterpret_cast<uint32_t *>(ws + kWsHeader);
    a.partials = reinterpret_cast<float *>(ws + kWsRecords);
    a.status = reinterpret_cast<int32_t *>(ws);
    a.batch = d->batch;
    a.n_q = d->n_q;
    a.n_k = d->n_k;
    a.n_v = d->n_v;
    a.t_max = max_blocks * P;
    a.max_blocks = max_blocks;
    a.num_pages = cache->num_pages;
    a.sb = cache->scale_block;
    a.partial_slots = (long long)units + kGridMax;
    a.scale_blocks = (long long)cache->num_pages * (P / cache->scale_block);
    a.scale_log2 = (float)((double)d->scale * 1.4426950408889634);
    a.wait_limit_ns = kWaitLimitNs;
    // fewer CTAs where the hint says that there are fewer tiles
    const int msl = max_seq_len >= 1 && max_seq_len <= a.t_max ? max_seq_len : a.t_max;
    const long long tiles = (long long)units * ((msl + kTT - 1) / kTT);
    a.grid = (int)std::min<long long>({tiles, (long long)dev.num_sms * per_sm, (long long)kGridMax});
    if (ensure_dynamic_smem((const void *)fn, (int)smem) != DIFFQKV_OK) return DIFFQKV_ERR_CUDA;
    fn<<<a.grid, kThreads, smem, stream>>>(tm_k, tm_v, a);
    return cudaGetLastError() == cudaSuccess ? DIFFQKV_OK : DIFFQKV_ERR_CUDA;
}

}  // namespace

}  // namespace diffqkv

extern "C" diffqkv_status_t diffqkv_decode_paged_kv8(const diffqkv_dims_t *dims, const diffqkv_kv8_cache_t *cache,
                                                     const void *q, const int32_t *block_table, int32_t max_blocks,
                                                     const int32_t *seq_lens, int32_t max_seq_len, void *out,
                                                     void *workspace, size_t workspace_bytes,
                                                     diffqkv_stream_t stream) {
    diffqkv::ApiRange nvtx_range("diffqkv_decode_paged_kv8");
    return diffqkv::decode_kv8_launch(dims, cache, q, block_table, max_blocks, seq_lens, max_seq_len, out, workspace,
                                      workspace_bytes, (cudaStream_t)stream);
}
