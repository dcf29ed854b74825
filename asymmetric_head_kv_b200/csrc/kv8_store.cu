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
// The call reads 2 bytes and writes 1 per element; with a prompt's rows that is what bounds it.  A run is
// a maximal stretch of consecutive tokens in one block; one warp owns a (run, head), so the block's
// maximum needs no atomics and no second launch: the warp keeps up to kVec 16-byte loads of the run's
// rows in registers between the maximum and the rounding (a run of 32 rows of 64 or 16 of 128), and
// reads longer runs twice (the second time out of L1 / L2).  The maximum is taken on the bf16 bit patterns
// (two 16-bit maxima an instruction) and crosses the warp in one redux.
#include <algorithm>

#include "internal.h"
#include "kv8.cuh"

namespace diffqkv {

namespace {

constexpr int kStoreWarps = 8;
constexpr int kVec = 8;        // 16-byte loads a lane keeps
constexpr int kMaxTokens = 16; // tokens whose runs one CTA may lead

struct StoreArgs {
    const uint4 *k_new, *v_new;
    uint8_t *k_pages, *v_pages, *k_scales, *v_scales;
    const int32_t *slot_map;
    int32_t *status;
    int32_t tokens, n_k, n_v, sb, sb_shift;  // sb_shift: log2(sb), or -1
    int32_t slots;                           // num_pages * page_size
    int32_t chunk;                           // tokens of one CTA
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

// One (run, head): the run's tokens t0 .. t0 + len - 1 lie in scale block `blk`, lowest row `low`.
template <int D>
__device__ __forceinline__ void store_run(const StoreArgs &a, const uint4 *x, uint8_t *pages, uint8_t *scales,
                                          int heads, int head, int t0, int len, int blk, int low, int lane) {
    constexpr int LPR = D / 8;      // lanes of a row (8 elements each)
    constexpr int ROWS = 32 / LPR;  // rows of one warp-wide load
    const int sub = lane / LPR, part = lane % LPR;
    uint8_t *byte = scales + (size_t)blk * heads + head;
    const int old = low > 0 ? kv8_exp(*byte) : 0;
    auto row_of = [&](int i) { return x + ((size_t)(t0 + i) * heads + head) * LPR + part; };

    uint4 keep[kVec];
    uint32_t m = 0;
    for (int base = 0; base < len; base += ROWS * kVec) {
#pragma unroll
        for (int v = 0; v < kVec; ++v) {
            const int i = base + v * ROWS + sub;
            keep[v] = i < len ? __ldg(row_of(i)) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int v = 0; v < kVec; ++v)
            m = max_bits(max_bits(max_bits(max_bits(m, keep[v].x), keep[v].y), keep[v].z), keep[v].w);
    }
    uint32_t amax = __reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16));
    if (amax >= 0x7f80u) {  // an infinity or NaN among them: the maximum again without those
        m = 0;
        for (int i = sub; i < len; i += ROWS) {
            const uint4 r = __ldg(row_of(i));
            m = max_finite_bits(max_finite_bits(max_finite_bits(max_finite_bits(m, r.x), r.y), r.z), r.w);
        }
        amax = __reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16));
    }
    int e = scale_exp(amax);
    if (low > 0) e = max(e, old);
    const float f = exp2_int(-e);

    for (int base = 0; base < len; base += ROWS * kVec) {
        if (len > ROWS * kVec) {
#pragma unroll
            for (int v = 0; v < kVec; ++v) {
                const int i = base + v * ROWS + sub;
                if (i < len) keep[v] = __ldg(row_of(i));
            }
        }
#pragma unroll
        for (int v = 0; v < kVec; ++v) {
            const int i = base + v * ROWS + sub;
            if (i >= len) continue;
            const int slot = slot_of(a, t0 + i);
            *reinterpret_cast<uint2 *>(pages + ((size_t)slot * heads + head) * D + part * 8) = quantise8(keep[v], f);
        }
    }
    if (low > 0 && e > old) {
        const float g = exp2_int(max(old - e, -126));  // 2^-126 already takes every code to zero
        for (int r = sub; r < low; r += ROWS) {
            uint2 *p = reinterpret_cast<uint2 *>(pages + (((size_t)blk * a.sb + r) * heads + head) * D + part * 8);
            uint2 c = *p;
            c.x = move4(c.x, g);
            c.y = move4(c.y, g);
            *p = c;
        }
    }
    if (lane == 0 && (low == 0 || e != old)) *byte = (uint8_t)(e + 127);
}

template <int DK, int DV>
__global__ void __launch_bounds__(kStoreWarps * 32) kv8_store_kernel(const StoreArgs a) {
    const int lane = threadIdx.x & 31;
    const int warp = (threadIdx.x >> 5) + kStoreWarps * blockIdx.y;
    const int warps = kStoreWarps * gridDim.y;
    const int heads = a.n_k + a.n_v;
    const int t_begin = blockIdx.x * a.chunk;
    // every warp finds the runs its CTA leads: lane i looks at token t_begin + i
    const int t = t_begin + lane;
    int slot = -1, blk = -1;
    bool leads = false;
    if (lane < a.chunk && t < a.tokens) {
        const int raw = __ldg(a.slot_map + t);
        if (raw >= a.slots && warp == 0) record_error(a.status, DIFFQKV_ERR_DEVICE_PAGE);
        slot = raw < a.slots ? raw : -1;
        if (slot >= 0) {
            blk = block_of(a, slot);
            const int before = t > 0 ? slot_of(a, t - 1) : -1;
            leads = before < 0 || block_of(a, before) != blk;
        }
    }
    int pair = warp;  // (run, head) pairs go round the warps
    for (unsigned left = __ballot_sync(0xffffffffu, leads); left; left &= left - 1) {
        const int src = __ffs(left) - 1;
        if (pair >= heads) {
            pair -= heads;
            continue;
        }
        const int t0 = t_begin + src;
        const int run_blk = __shfl_sync(0xffffffffu, blk, src);
        // the run's length and lowest row, 32 tokens at a time
        int len = 0, low = a.sb;
        for (bool open = true; open; len += 32) {
            const int tt = t0 + len + lane;
            const int s = tt < a.tokens ? slot_of(a, tt) : -1;
            const bool in = s >= 0 && block_of(a, s) == run_blk;
            const unsigned out = __ballot_sync(0xffffffffu, !in);
            const int n = out ? __ffs(out) - 1 : 32;
            low = min(low, (int)__reduce_min_sync(0xffffffffu, lane < n ? (unsigned)(s - run_blk * a.sb) : 0x7fffffffu));
            if (n < 32) {
                len += n - 32;
                open = false;
            }
        }
        for (; pair < heads; pair += warps) {
            if (pair < a.n_k)
                store_run<DK>(a, a.k_new, a.k_pages, a.k_scales, a.n_k, pair, t0, len, run_blk, low, lane);
            else
                store_run<DV>(a, a.v_new, a.v_pages, a.v_scales, a.n_v, pair - a.n_k, t0, len, run_blk, low, lane);
        }
        pair -= heads;
    }
}

using StoreFn = void (*)(StoreArgs);

diffqkv_status_t kv8_store_launch(const diffqkv_dims_t *d, const diffqkv_kv8_cache_t *c, const void *k_new,
                                  const void *v_new, const int32_t *slot_map, int32_t tokens, int32_t *status,
                                  cudaStream_t stream) {
    diffqkv_status_t st = validate_kv8(d, c);
    if (st != DIFFQKV_OK) return st;
    if (tokens < 0) return DIFFQKV_ERR_INVALID_ARG;
    if (tokens == 0) return DIFFQKV_OK;
    if (!k_new || !v_new || !slot_map) return DIFFQKV_ERR_INVALID_ARG;
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
    // few tokens: one CTA for each token and eight heads, so that every warp has one pair; many: the
    // chunk covers a block's tokens and the warps go round its heads
    const int heads = d->n_k + d->n_v;
    a.chunk = std::min(kMaxTokens, std::max(1, tokens / (4 * dev.num_sms)));
    const int gx = (tokens + a.chunk - 1) / a.chunk;
    const int gy = (heads + kStoreWarps - 1) / kStoreWarps;
    if (gy > 65535) return DIFFQKV_ERR_UNSUPPORTED;
    StoreFn fn = d->d_k == 64 ? (d->d_v == 64 ? kv8_store_kernel<64, 64> : kv8_store_kernel<64, 128>)
                              : (d->d_v == 64 ? kv8_store_kernel<128, 64> : kv8_store_kernel<128, 128>);
    fn<<<dim3(gx, gy), kStoreWarps * 32, 0, stream>>>(a);
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
