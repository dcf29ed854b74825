// kv8_store.cu -- new K and V rows quantised into the pages of an 8-bit cache.
//
// The cache holds e4m3 codes and one power of two 2^e per block of `sb` positions (inside a page) and
// head.  e4m3 is a floating type, so a power-of-two scale costs it no relative precision, and both
// directions of it are exact: x * 2^-e before the one rounding to e4m3, and moving a code between two
// scales (which rounds only where it falls below the smallest normal code).
//
// For every (block, head) that the call's rows touch:
//   a  = max |x| over the call's finite values in it, e_new = least e in [-120, 119] with a <= 448 * 2^e
//   lowest row written is the block's row 0:  e = e_new      (the block begins anew)
//   else:                                     e = max(e_old, e_new), and where that grew, the rows
//                                             below the lowest written one become rn(code * 2^(e_old - e))
//   code = rn_e4m3(x * 2^-e)                  (infinities, and magnitudes above 448 * 2^119, become +-448; NaN stays NaN)
// Rows above the written ones stay as they are.
//
// The call reads 2 bytes and writes 1 per element; with a prompt's rows that is what bounds it, with a decode step's
// the launch and four dependent loads.  A run is a maximal stretch of consecutive tokens in one block.  One group of lanes
// owns a (run, head), so the block's maximum needs no atomics and no second launch; the rows stay in registers between the
// maximum and the rounding (longer runs are read twice).  The first rows are requested together with the slots,
// before it is known which run they belong to: most often they are the ones.
// Shapes of group, by the rows a run can have (4 heads of 64 and 16 of 128 unless stated, inputs beyond L2):
//  * `share` warps over the runs that begin in the CTA's chunk of tokens.  One warp (CTAs of four) where it holds a block in
//    registers (16 rows of 128 or 32 of 64) and where the call has kWarpsPerSm (run, head)s an SM or more; otherwise two,
//    four or eight (CTAs of eight) up to one of the two; the maximum crosses a warp in one redux and the warps through
//    shared memory.  16384 tokens in blocks of 16: 25.5 us, 4.4 TB/s, 0.69 of the copy rate (27.7 with CTAs of
//    eight for one warp); of 64: 30 us (35.6 with four warps each), of 128: 37 (47 with eight).  1024 tokens in blocks of
//    128: 6.9 us shared, 15.2 with one warp; 4096: 13.8 against 21.6.
//    Slots come 64 tokens at a time, side by side, so that a run of up to 32 tokens is known without another load.  What keeps
//    it from the copy rate: issue slots (66% used) and the CTAs' start, two loads deep.
//  * a chunk of one token for up to kFewTokens, so that a decode step's heads and requests spread over the SMs: 16 tokens
//    3.5 us against 4.6 with chunks of 16, 256 tokens 4.5 against 5.0, but 512 tokens 6.0 against 5.0.
//  * blocks of up to kRowBlock positions in larger steps: the 8 or 16 lanes of one row take kRowVec tokens and the runs
//    that begin there.  16384 tokens: blocks of one 68 us (a warp a run: 174), of four 36 us (a warp: 53).
#include <algorithm>
#include <type_traits>

#include "internal.h"
#include "kv8.cuh"

namespace diffqkv {

namespace {

constexpr int kStoreWarps = 8;
constexpr int kRunVec = 8, kRowVec = 4;  // 16-byte loads a lane keeps, by shape of group
constexpr int kMaxTokens = 32; // tokens whose runs one CTA may lead
constexpr int kRowBlock = 4;   // blocks up to this size take a row's lanes
constexpr int kWarpsPerSm = 16;  // (run, head)s an SM from which a warp each is enough
constexpr int kFewTokens = 256;
constexpr int run_warps(bool shared) { return shared ? kStoreWarps : kStoreWarps / 2; }

struct StoreArgs {
    const uint4 *k_new, *v_new;
    uint8_t *k_pages, *v_pages, *k_scales, *v_scales;
    const int32_t *slot_map;
    int32_t *status;
    int32_t tokens, n_k, n_v, sb, sb_shift;  // sb_shift: log2(sb), or -1
    int32_t slots;                           // num_pages * page_size
    int32_t chunk;                           // tokens of one CTA
    int32_t share;                           // warps of one (run, head)
};

__device__ __forceinline__ int block_of(const StoreArgs &a, int slot) {
    return a.sb_shift >= 0 ? slot >> a.sb_shift : slot / a.sb;
}

// Slot of token t, or -1 where it names none.
__device__ __forceinline__ int slot_of(const StoreArgs &a, int t) {
    const int s = __ldg(a.slot_map + t);
    return s < a.slots ? s : -1;
}

// Larger magnitude of each of two bf16 pairs, as bits without the sign.
__device__ __forceinline__ uint32_t max_bits(uint32_t m, uint32_t w) { return __vmaxu2(m, w & 0x7fff7fffu); }

// The same without infinities and NaN.
__device__ __forceinline__ uint32_t max_finite_bits(uint32_t m, uint32_t w) {
    uint32_t lo = w & 0x7fffu, hi = (w >> 16) & 0x7fffu;
    lo = lo >= 0x7f80u ? 0u : lo;
    hi = hi >= 0x7f80u ? 0u : hi;
    return __vmaxu2(m, lo | (hi << 16));
}

// Least e in [kKv8MinExp, kKv8MaxExp] with the bf16 number of these bits (finite, no sign) <= 448 * 2^e =
// 1.75 * 2^(e + 8).
__device__ __forceinline__ int scale_exp(uint32_t bits) {
    return min(max((int)(bits >> 7) - 135 + ((bits & 0x7fu) > 0x60u ? 1 : 0), kKv8MinExp), kKv8MaxExp);
}

__device__ __forceinline__ uint2 quantise8(const uint4 &x, float f) {
    uint2 r;
    r.x = e4m3x2(bf16lo(x.x) * f, bf16hi(x.x) * f) | (e4m3x2(bf16lo(x.y) * f, bf16hi(x.y) * f) << 16);
    r.y = e4m3x2(bf16lo(x.z) * f, bf16hi(x.z) * f) | (e4m3x2(bf16lo(x.w) * f, bf16hi(x.w) * f) << 16);
    return r;
}

// Four codes times the power of two f <= 1.
__device__ __forceinline__ uint32_t move4(uint32_t codes, float f) {
    float a, b, c, d;
    f16x2_to_floats(e4m3x2_to_f16x2(codes & 0xffffu), a, b);
    f16x2_to_floats(e4m3x2_to_f16x2(codes >> 16), c, d);
    return e4m3x2(a * f, b * f) | (e4m3x2(c * f, d * f) << 16);
}

// Largest of v over the group of G lanes.
template <int G>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
    if constexpr (G == 32) return __reduce_max_sync(0xffffffffu, v);
    const uint32_t mask = ((1u << G) - 1u) << (threadIdx.x & 31 & ~(G - 1));
#pragma unroll
    for (int off = G / 2; off >= 1; off >>= 1) v = max(v, __shfl_xor_sync(mask, v, off));
    return v;
}

// One (run, head): the run's tokens t0 .. t0 + len - 1 lie in scale block `blk`, lowest row `low`.  `lane`: of the group.
// keep: the lane's first rows of the run if `kept`.  `share` groups (warps) split the rows, this one being `mine`; their
// maxima meet in `cross` (shared memory, one word a warp of the CTA) at a named barrier of theirs.
template <int D, int G, int VEC>
__device__ __forceinline__ void store_run(const StoreArgs &a, const uint4 *x, uint8_t *pages, uint8_t *scales,
                                          int heads, int head, int t0, int len, int blk, int low, int lane,
                                          uint4 (&keep)[VEC], bool kept, int share = 1, int mine = 0,
                                          uint32_t *cross = nullptr) {
    constexpr int LPR = D / 8;              // lanes of a row (8 elements each)
    const int ROWS = G / LPR * share;       // rows of one load of the groups
    const int sub = mine * (G / LPR) + lane / LPR, part = lane % LPR;
    if (!in_bounds(blk, a.slots / a.sb, a.status) || !in_bounds((long long)t0 + len - 1, a.tokens, a.status)) return;
    uint8_t *byte = scales + (size_t)blk * heads + head;
    const int old = low > 0 ? kv8_exp(*byte) : 0;
    auto row_of = [&](int i) { return x + ((size_t)(t0 + i) * heads + head) * LPR + part; };

    uint32_t m = 0;
    for (int base = sub; base < len; base += ROWS * VEC) {
        if (!kept || base != sub)
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                const int i = base + v * ROWS;
                if (i < len) keep[v] = __ldg(row_of(i));
            }
#pragma unroll
        for (int v = 0; v < VEC; ++v)
            if (base + v * ROWS < len)
                m = max_bits(max_bits(max_bits(max_bits(m, keep[v].x), keep[v].y), keep[v].z), keep[v].w);
    }
    auto all_max = [&](uint32_t v) {
        v = group_max<G>(v);
        if (share > 1) {
            const int first = ((int)threadIdx.x >> 5) - mine;
            named_barrier(1 + first / share, share * 32);
            if (lane == 0) cross[first + mine] = v;
            named_barrier(1 + first / share, share * 32);
            for (int w = 0; w < share; ++w) v = max(v, cross[first + w]);
        }
        return v;
    };
    uint32_t amax = all_max(max(m & 0xffffu, m >> 16));
    if (amax >= 0x7f80u) {  // an infinity or NaN among them: the maximum again without those
        m = 0;
        for (int i = sub; i < len; i += ROWS) {
            const uint4 r = __ldg(row_of(i));
            m = max_finite_bits(max_finite_bits(max_finite_bits(max_finite_bits(m, r.x), r.y), r.z), r.w);
        }
        amax = all_max(max(m & 0xffffu, m >> 16));
    }
    int e = scale_exp(amax);
    if (low > 0) e = max(e, old);
    const float f = exp2_int(-e);

    for (int base = sub; base < len; base += ROWS * VEC) {
        int slot[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            const int i = base + v * ROWS;
            if (i < len) {
                if (len > ROWS * VEC) keep[v] = __ldg(row_of(i));
                slot[v] = __ldg(a.slot_map + t0 + i);  // (inside the pool: it belongs to the run)
            }
        }
#pragma unroll
        for (int v = 0; v < VEC; ++v)
            if (base + v * ROWS < len && in_bounds(slot[v], a.slots, a.status))
                *reinterpret_cast<uint2 *>(pages + ((size_t)slot[v] * heads + head) * D + part * 8) =
                    quantise8(keep[v], f);
    }
    if (low > 0 && e > old) {
        const float g = exp2_int(max(old - e, -126));  // 2^-126 already takes every code to zero
        for (int r = sub; r < low && in_bounds(r, a.sb, a.status); r += ROWS) {
            uint2 *p = reinterpret_cast<uint2 *>(pages + (((size_t)blk * a.sb + r) * heads + head) * D + part * 8);
            uint2 c = *p;
            c.x = move4(c.x, g);
            c.y = move4(c.y, g);
            *p = c;
        }
    }
    if (lane == 0 && mine == 0 && (low == 0 || e != old)) *byte = (uint8_t)(e + 127);
}

template <int DK, int DV, bool SHARED>
__global__ void __launch_bounds__(run_warps(SHARED) * 32, 24 / run_warps(SHARED)) kv8_store_runs_kernel(const StoreArgs a) {
    constexpr int WARPS = run_warps(SHARED);
    __shared__ uint32_t cross[WARPS];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int share = SHARED ? a.share : 1;
    const int heads = a.n_k + a.n_v;
    // the (run, head)s of this warp: one head, the runs that begin in the CTA's chunk of tokens
    const int head = blockIdx.y * (WARPS / share) + warp / share, mine = warp % share;
    const int t_begin = blockIdx.x * a.chunk;
    uint4 keep[kRunVec];
    if (!SHARED && head < heads) {  // the chunk's rows, before the slots are there
        const bool k = head < a.n_k;
        const int lpr = k ? DK / 8 : DV / 8, n = k ? a.n_k : a.n_v, rows = 32 / lpr;
        const uint4 *x = (k ? a.k_new : a.v_new) + (size_t)(k ? head : head - a.n_k) * lpr + lane % lpr;
#pragma unroll
        for (int v = 0; v < kRunVec; ++v) {
            const int i = v * rows + lane / lpr;
            if (i < a.chunk && t_begin + i < a.tokens) keep[v] = __ldg(x + (size_t)(t_begin + i) * n * lpr);
        }
    }
    // every warp finds the runs its CTA leads: lane i has the slots of tokens t_begin + i and t_begin + 32 + i
    const int t = t_begin + lane, raw = t < a.tokens ? __ldg(a.slot_map + t) : -1;
    const int far = t + 32 < a.tokens ? slot_of(a, t + 32) : -1;
    const int ahead = lane == 0 && t > 0 ? slot_of(a, t - 1) : -1;
    if (raw >= a.slots && lane < a.chunk && warp == 0 && blockIdx.y == 0) record_error(a.status, DIFFQKV_ERR_DEVICE_PAGE);
    const int slot = raw < a.slots ? raw : -1, blk = slot >= 0 ? block_of(a, slot) : -1;
    int before = __shfl_up_sync(0xffffffffu, blk, 1);
    if (lane == 0) before = ahead >= 0 ? block_of(a, ahead) : -1;
    const bool leads = lane < a.chunk && blk >= 0 && before != blk;
    if (head >= heads) return;
    for (unsigned left = __ballot_sync(0xffffffffu, leads); left; left &= left - 1) {
        const int src = __ffs(left) - 1;
        const int t0 = t_begin + src;
        const int run_blk = __shfl_sync(0xffffffffu, blk, src);
        // the run's length and lowest row, 32 tokens at a time; a block's rows are all that a run can have
        int len = 0, low = a.sb;
        for (bool open = true; open; len += 32) {
            const int tt = t0 + len + lane;
            int s;
            if (len == 0) {
                const int x = __shfl_sync(0xffffffffu, slot, src + lane & 31), y = __shfl_sync(0xffffffffu, far, src + lane & 31);
                s = src + lane < 32 ? x : y;
            } else {
                s = tt < a.tokens ? slot_of(a, tt) : -1;
            }
            const unsigned row = (unsigned)(s - run_blk * a.sb);
            const unsigned out = __ballot_sync(0xffffffffu, s < 0 || row >= (unsigned)a.sb);
            const int n = out ? __ffs(out) - 1 : 32;
            low = min(low, (int)__reduce_min_sync(0xffffffffu, lane < n ? row : 0x7fffffffu));
            open = n == 32 && len + 32 < a.sb;
            if (n < 32) len += n - 32;
        }
        const bool kept = !SHARED && src == 0 && len <= a.chunk;
        if (head < a.n_k)
            store_run<DK, 32>(a, a.k_new, a.k_pages, a.k_scales, a.n_k, head, t0, len, run_blk, low, lane, keep, kept, share,
                              mine, cross);
        else
            store_run<DV, 32>(a, a.v_new, a.v_pages, a.v_scales, a.n_v, head - a.n_k, t0, len, run_blk, low, lane, keep, kept,
                              share, mine, cross);
    }
}

// One group of D / 8 lanes per head and kRowVec tokens: the runs that begin among them.
template <int D>
__device__ __forceinline__ void store_rows(const StoreArgs &a, const uint4 *x, uint8_t *pages, uint8_t *scales, int heads,
                                           unsigned cta, bool flag) {
    constexpr int LPR = D / 8, VEC = kRowVec;
    const unsigned group = (cta * (kStoreWarps * 32u) + threadIdx.x) / LPR;
    const int t0 = (int)(group / (unsigned)heads) * VEC, head = (int)(group % (unsigned)heads);
    if (t0 >= a.tokens) return;
    auto row = [&](int t) { return __ldg(x + ((size_t)t * heads + head) * LPR + threadIdx.x % LPR); };
    uint4 rows[VEC];  // before the slots are there
#pragma unroll
    for (int v = 0; v < VEC; ++v)
        if (t0 + v < a.tokens) rows[v] = row(t0 + v);
    int slot[VEC], blk[VEC + 2];  // blk[v + 1]: block of token t0 + v
#pragma unroll
    for (int v = -1; v <= VEC; ++v) {
        const int t = t0 + v, raw = t >= 0 && t < a.tokens ? __ldg(a.slot_map + t) : -1;
        if (v >= 0 && v < VEC) {
            slot[v] = raw;
            if (raw >= a.slots && flag && head == 0) record_error(a.status, DIFFQKV_ERR_DEVICE_PAGE);
        }
        blk[v + 1] = raw >= 0 && raw < a.slots ? block_of(a, raw) : -1;
    }
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
        const int b = blk[v + 1];
        if (b < 0 || blk[v] == b) continue;
        int len = 1, low = slot[v] - b * a.sb;
#pragma unroll
        for (int w = v + 1; w < VEC; ++w)
            if (len == w - v && blk[w + 1] == b) {
                low = min(low, slot[w] - b * a.sb);
                ++len;
            }
        if (len == VEC - v && blk[VEC + 1] == b)  // on behind these tokens
            for (int t = t0 + VEC, s; t < a.tokens && (s = slot_of(a, t)) >= 0 && block_of(a, s) == b; ++t) {
                low = min(low, s - b * a.sb);
                ++len;
            }
        uint4 keep[VEC];
#pragma unroll
        for (int w = 0; w < VEC; ++w)
            if (w < len) keep[w] = v + w < VEC ? rows[v + w] : row(t0 + v + w);
        store_run<D, LPR>(a, x, pages, scales, heads, head, t0 + v, len, b, low, (int)threadIdx.x % LPR, keep, true);
    }
}

// The first k_ctas CTAs: K, the others: V.
template <int DK, int DV>
__global__ void __launch_bounds__(kStoreWarps * 32) kv8_store_rows_kernel(const StoreArgs a, unsigned k_ctas) {
    if (blockIdx.x < k_ctas)
        store_rows<DK>(a, a.k_new, a.k_pages, a.k_scales, a.n_k, blockIdx.x, true);
    else
        store_rows<DV>(a, a.v_new, a.v_pages, a.v_scales, a.n_v, blockIdx.x - k_ctas, false);
}

template <int DK, int DV>
void store_launch(const StoreArgs &a, cudaStream_t stream) {
    if (a.sb <= kRowBlock && a.tokens > kFewTokens) {
        auto ctas = [&](int heads, int d) {
            const long long threads = ((long long)a.tokens + kRowVec - 1) / kRowVec * heads * (d / 8);
            return (unsigned)((threads + kStoreWarps * 32 - 1) / (kStoreWarps * 32));
        };
        const unsigned k = ctas(a.n_k, DK), v = ctas(a.n_v, DV);
        kv8_store_rows_kernel<DK, DV><<<k + v, kStoreWarps * 32, 0, stream>>>(a, k);
        return;
    }
    const int per_cta = run_warps(a.share > 1) / a.share;
    const dim3 grid((a.tokens + a.chunk - 1) / a.chunk, (a.n_k + a.n_v + per_cta - 1) / per_cta);
    if (a.share > 1)
        kv8_store_runs_kernel<DK, DV, true><<<grid, run_warps(true) * 32, 0, stream>>>(a);
    else
        kv8_store_runs_kernel<DK, DV, false><<<grid, run_warps(false) * 32, 0, stream>>>(a);
}

diffqkv_status_t kv8_store_launch(const diffqkv_dims_t *d, const diffqkv_kv8_cache_t *c, const void *k_new,
                                  const void *v_new, const int32_t *slot_map, int32_t tokens, int32_t *status,
                                  cudaStream_t stream) {
    diffqkv_status_t st = validate_kv8(d, c);
    if (st != DIFFQKV_OK) return st;
    if (tokens < 0) return DIFFQKV_ERR_INVALID_ARG;
    if (tokens == 0) return DIFFQKV_OK;
    if (!k_new || !v_new || !slot_map) return DIFFQKV_ERR_INVALID_ARG;
    if ((long long)d->n_k + d->n_v > 65535) return DIFFQKV_ERR_UNSUPPORTED;  // grid
    if ((long long)tokens * std::max(d->n_k, d->n_v) * 16 > 0x7fffffffLL) return DIFFQKV_ERR_UNSUPPORTED;  // thread index
    if (!aligned16(k_new) || !aligned16(v_new) || (reinterpret_cast<uintptr_t>(slot_map) & 3u) ||
        (reinterpret_cast<uintptr_t>(status) & 3u))
        return DIFFQKV_ERR_MISALIGNED;
    DeviceInfo dev;
    st = current_device_info(&dev);
    if (st != DIFFQKV_OK) return st;

    StoreArgs a;
    a.k_new = static_cast<const uint4 *>(k_new);
    a.v_new = static_cast<const uint4 *>(v_new);
    a.k_pages = static_cast<uint8_t *>(c->k_pages);
    a.v_pages = static_cast<uint8_t *>(c->v_pages);
    a.k_scales = c->k_scales;
    a.v_scales = c->v_scales;
    a.slot_map = slot_map;
    a.status = status ? status : dev.status_word;
    a.tokens = tokens;
    a.n_k = d->n_k;
    a.n_v = d->n_v;
    a.sb = c->scale_block;
    a.sb_shift = -1;
    if ((a.sb & (a.sb - 1)) == 0)
        for (a.sb_shift = 0; (1 << a.sb_shift) < a.sb;) ++a.sb_shift;
    a.slots = c->num_pages * c->page_size;
    // a CTA's chunk is about a block of tokens, one token where there are few; the warps of a (run, head) hold a block
    a.chunk = tokens <= kFewTokens ? 1 : std::min(kMaxTokens, std::max(16, a.sb));
    a.share = 1;
    if (tokens > kFewTokens)
        while (a.share < kStoreWarps && a.share * 32 * kRunVec * 8 / std::max(d->d_k, d->d_v) < a.sb &&
               (long long)tokens * (d->n_k + d->n_v) / a.sb * a.share < kWarpsPerSm * dev.num_sms)
            a.share *= 2;
    if (d->d_k == 64)
        d->d_v == 64 ? store_launch<64, 64>(a, stream) : store_launch<64, 128>(a, stream);
    else
        d->d_v == 64 ? store_launch<128, 64>(a, stream) : store_launch<128, 128>(a, stream);
    return cudaGetLastError() == cudaSuccess ? DIFFQKV_OK : DIFFQKV_ERR_CUDA;
}

}  // namespace

diffqkv_status_t validate_kv8(const diffqkv_dims_t *d, const diffqkv_kv8_cache_t *c) {
    const diffqkv_status_t st = validate_dims(d);
    if (st != DIFFQKV_OK) return st;
    if (!c || !c->k_pages || !c->v_pages || !c->k_scales || !c->v_scales || c->num_pages < 1 || c->page_size < 1 ||
        c->scale_block < 1 || c->page_size % c->scale_block != 0)
        return DIFFQKV_ERR_INVALID_ARG;
    if ((d->d_k != 64 && d->d_k != 128) || (d->d_v != 64 && d->d_v != 128)) return DIFFQKV_ERR_UNSUPPORTED;
    if (c->page_size % 8 != 0) return DIFFQKV_ERR_UNSUPPORTED;
    if ((long long)c->num_pages * c->page_size > 0x7fffffffLL) return DIFFQKV_ERR_UNSUPPORTED;
    if (!aligned16(c->k_pages) || !aligned16(c->v_pages)) return DIFFQKV_ERR_MISALIGNED;
    return DIFFQKV_OK;
}

}  // namespace diffqkv

extern "C" diffqkv_status_t diffqkv_kv8_store(const diffqkv_dims_t *dims, const diffqkv_kv8_cache_t *cache,
                                              const void *k_new, const void *v_new, const int32_t *slot_map,
                                              int32_t tokens, int32_t *device_status_word, diffqkv_stream_t stream) {
    diffqkv::ApiRange nvtx_range("diffqkv_kv8_store");
    return diffqkv::kv8_store_launch(dims, cache, k_new, v_new, slot_map, tokens, device_status_word,
                                     (cudaStream_t)stream);
}
