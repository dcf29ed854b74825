// page_map.cu -- block tables and slot maps of a serving step, from the requests' lengths.
//
// Request b holds s_b cached positions in pages of P and adds n_b.  With exclusive sums over the
// requests, qs_b = sum n and off_b = sum (ceil((s + n) / P) - ceil(s / P)),
//   table[b, ceil(s_b / P) + i] = free[off_b + i],  and token i of request b, row qs_b + i of the
//   step's token buffer, sits at position p = s_b + i, slot table[b, p / P] * P + p % P.
//
// One launch.  The work is two sums over the requests and a few bytes a token, so what bounds it is
// the launch and the latency of a handful of dependent loads; a second launch, or CTAs that wait on
// one another for a carried sum, would cost more than every CTA redoing the sums (8 bytes a request
// out of L2).  Each thread sums a run of consecutive requests, a block scan of the runs' sums stays in
// shared memory, and a token or page finds its request by a binary search over the runs and a walk
// inside one.  No CTA reads what another writes: the slot of a token in a new page comes from the
// free list, not from the table entry.
// Up to kManyThreads requests a thread has one request (ONE), and what the tokens need of it (its length, its pages, the
// page that it fills first, and the head of the free list) is fetched beside the sums and kept in shared memory: the map of a
// decode step then has two dependent global loads in a row instead of five: 512 requests with a token each 5.6 us against
// 6.1 without, 256 requests of up to 127 tokens 4.8 against 5.3 (both with four tokens a thread).
// CTAs of kFewThreads threads up to as many requests, of kManyThreads beyond: 256 requests of up to 127 tokens 4.8 us against
// 6.1 with the larger CTAs.
// A thread maps one token while the buffer is small enough (each token is a search of its own then, side by side): 64
// requests with a token each 3.0 us against 4.0 with four a thread, 256 requests of up to 127 tokens 3.4 against 4.5,
// a buffer of 160000 rows 4.5 against 4.7.  Beyond, four, which share a search and a 16-byte store: 270000 rows 4.75 us
// against 5.05, 2^20 rows of 1024 requests 7.2 against 8.8.
#include "common.cuh"
#include "internal.h"

namespace diffqkv {

namespace {

constexpr int kFewThreads = 256, kManyThreads = 1024;
constexpr int kMapTokens = 4;  // consecutive tokens a thread maps in large buffers (one 16-byte store per output)

struct PageMapArgs {
    const int32_t *seq_lens, *new_lens, *free_pages;
    int32_t *block_table, *query_start, *slot_map, *positions, *total_lens, *pages_used, *status;
    int32_t batch, max_blocks, page_size, page_shift, num_pages, num_free, capacity;
    int32_t per;  // requests of one thread's run
};

struct Request {
    int s, n;      // cached positions and new tokens, after the checks
    int have, take;  // pages it holds and pages it takes
};

__device__ __forceinline__ int page_of(const PageMapArgs &a, int x) {
    return a.page_shift >= 0 ? x >> a.page_shift : x / a.page_size;
}

// Request b after the checks: lengths outside [0, max_blocks * page_size] add nothing.
__device__ __forceinline__ Request load_request(const PageMapArgs &a, int b, bool dropped, bool flag) {
    const int cap = a.max_blocks * a.page_size;
    const int s = __ldg(a.seq_lens + b), n = __ldg(a.new_lens + b);
    Request r;
    r.s = min(max(s, 0), cap);
    const bool bad = s < 0 || s > cap || n < 0 || n > cap - s;
    if (bad && flag) record_error(a.status, DIFFQKV_ERR_DEVICE_SEQLEN);
    r.n = bad || dropped ? 0 : n;
    auto pages = [&](int x) {
        const int p = page_of(a, x);
        return p + (x != p * a.page_size);
    };
    r.have = pages(r.s);
    r.take = pages(r.s + r.n) - r.have;
    return r;
}

// Largest i in [0, n) with v[i] <= x (v ascending, v[0] <= x).
__device__ __forceinline__ int last_not_above(const int *v, int n, int x) {
    int lo = 0;
    while (n > 1) {
        const int half = n >> 1;
        if (v[lo + half] <= x) lo += half;
        n -= half;
    }
    return lo;
}

// A pool page, or -1 (flagged) for an entry outside the pool.
__device__ __forceinline__ int checked_page(const PageMapArgs &a, int page) {
    if (page >= 0 && page < a.num_pages) return page;
    record_error(a.status, DIFFQKV_ERR_DEVICE_PAGE);
    return -1;
}

// Whether the table has an entry lp of request b (checked build).
__device__ __forceinline__ bool in_table(const PageMapArgs &a, int b, int lp) {
    return in_bounds(b, a.batch, a.status) && in_bounds(lp, a.max_blocks, a.status);
}
__device__ __forceinline__ int held_entry(const PageMapArgs &a, int b, int lp) {
    return in_table(a, b, lp) ? a.block_table[(size_t)b * a.max_blocks + lp] : -1;
}

// ONE: at most THREADS requests, one a thread.
// TOKENS: consecutive tokens of a thread.
template <int THREADS, bool ONE, int TOKENS>
__global__ void __launch_bounds__(THREADS) page_map_kernel(const PageMapArgs a) {
    constexpr int WARPS = THREADS / 32;
    __shared__ int tok_s[THREADS], pag_s[THREADS];  // tokens and pages before each run
    __shared__ long long warp_t[WARPS], warp_p[WARPS];
    __shared__ int len_s[ONE ? THREADS : 1], page_s[ONE ? THREADS : 1], free_s[THREADS];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int b0 = min(a.batch, tid * a.per), b1 = min(a.batch, b0 + a.per);
    const bool first_cta = blockIdx.x == 0;

    free_s[tid] = tid < a.num_free ? __ldg(a.free_pages + tid) : -1;
    long long t = 0, p = 0;
    Request own{0, 0, 0, 0};
    for (int b = b0; b < b1; ++b) {
        own = load_request(a, b, false, first_cta);
        t += own.n;
        p += own.take;
    }
    int own_page = -1;  // pool page of the position after the cached ones, where that page is held
    if (ONE && b0 < b1 && own.n > 0 && page_of(a, own.s) < own.have)
        own_page = held_entry(a, b0, page_of(a, own.s));
    long long it = t, ip = p;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const long long yt = __shfl_up_sync(0xffffffffu, it, off), yp = __shfl_up_sync(0xffffffffu, ip, off);
        if (lane >= off) {
            it += yt;
            ip += yp;
        }
    }
    if (lane == 31) {
        warp_t[warp] = it;
        warp_p[warp] = ip;
    }
    __syncthreads();
    // every warp scans the warps' sums
    long long wt = lane < WARPS ? warp_t[lane] : 0, wp = lane < WARPS ? warp_p[lane] : 0;
#pragma unroll
    for (int off = 1; off < WARPS; off <<= 1) {
        const long long yt = __shfl_up_sync(0xffffffffu, wt, off), yp = __shfl_up_sync(0xffffffffu, wp, off);
        if (lane >= off) {
            wt += yt;
            wp += yp;
        }
    }
    const long long all_t = __shfl_sync(0xffffffffu, wt, WARPS - 1), all_p = __shfl_sync(0xffffffffu, wp, WARPS - 1);
    const long long bt = __shfl_sync(0xffffffffu, wt, max(warp - 1, 0)), bp = __shfl_sync(0xffffffffu, wp, max(warp - 1, 0));
    // a step that does not fit the token buffer or the free list is dropped as a whole
    const bool no_room = all_t > a.capacity;
    const bool dropped = no_room || all_p > a.num_free;
    if (dropped && first_cta && tid == 0)
        record_error(a.status, no_room ? DIFFQKV_ERR_DEVICE_SEQLEN : DIFFQKV_ERR_DEVICE_PAGE);
    const int tokens = dropped ? 0 : (int)all_t, pages = dropped ? 0 : (int)all_p;
    const int t_before = dropped ? 0 : (int)((warp ? bt : 0) + it - t), p_before = dropped ? 0 : (int)((warp ? bp : 0) + ip - p);
    tok_s[tid] = t_before;
    pag_s[tid] = p_before;
    if (ONE) {
        len_s[tid] = own.s;
        page_s[tid] = own_page;
    }

    // per-request outputs: run i belongs to CTA i mod grid
    if (tid % gridDim.x == blockIdx.x) {
        int at = t_before;
        for (int b = b0; b < b1; ++b) {
            if (!ONE) own = load_request(a, b, false, false);
            if (dropped) own.n = 0;
            a.query_start[b] = at;
            a.total_lens[b] = own.s + own.n;
            at += own.n;
        }
    }
    if (first_cta && tid == 0) {
        a.query_start[a.batch] = tokens;
        a.pages_used[0] = pages;
    }
    __syncthreads();
    const int runs = ONE ? a.batch : (a.batch + a.per - 1) / a.per;
    const int stride = gridDim.x * THREADS;
    auto held_pages = [&](int s) {
        const int q = page_of(a, s);
        return q + (s != q * a.page_size);
    };
    auto free_page = [&](int k) {
        if (!in_bounds(k, a.num_free, a.status)) return -1;
        return k < THREADS ? free_s[k] : __ldg(a.free_pages + k);
    };

    // table entries of the pages taken
    for (int k = blockIdx.x * THREADS + tid; k < pages; k += stride) {
        const int run = last_not_above(pag_s, runs, k);
        int b = run * a.per, off = pag_s[run], have;
        if (ONE) {
            have = held_pages(len_s[run]);
        } else {
            Request r = load_request(a, b, false, false);
            while (k >= off + r.take && in_bounds(b + 1, a.batch, a.status)) {
                off += r.take;
                r = load_request(a, ++b, false, false);
            }
            have = r.have;
        }
        if (in_table(a, b, have + (k - off)))
            a.block_table[(size_t)b * a.max_blocks + have + (k - off)] = checked_page(a, free_page(k));
    }

    // slots and positions, TOKENS consecutive tokens a thread
    for (long long i0 = (long long)(blockIdx.x * THREADS + tid) * TOKENS; i0 < a.capacity;
         i0 += (long long)stride * TOKENS) {
        int slot[TOKENS], pos[TOKENS];
#pragma unroll
        for (int e = 0; e < TOKENS; ++e) slot[e] = pos[e] = -1;
        if (i0 < tokens) {
            int run = last_not_above(tok_s, runs, (int)i0);
            int b = run * a.per, at = tok_s[run], off = pag_s[run], s, have, end;
            auto open = [&] {  // the request's length, pages and end (ONE)
                s = len_s[run];
                have = held_pages(s);
                at = tok_s[run];
                off = pag_s[run];
                end = run + 1 < runs ? tok_s[run + 1] : tokens;
            };
            Request r{0, 0, 0, 0};
            if (ONE)
                open();
            else {
                r = load_request(a, b, false, false);
                s = r.s;
                have = r.have;
                end = at + r.n;
            }
            int seen = -1, page = -1;  // logical page last looked up, and its pool page
#pragma unroll
            for (int e = 0; e < TOKENS; ++e) {
                const int i = (int)i0 + e;
                if (i >= tokens) break;
                while (i >= end && in_bounds(b + 1, a.batch, a.status)) {
                    seen = -1;
                    if (ONE) {
                        b = ++run;
                        open();
                    } else {
                        at = end;
                        off += r.take;
                        r = load_request(a, ++b, false, false);
                        s = r.s;
                        have = r.have;
                        end = at + r.n;
                    }
                }
                pos[e] = s + (i - at);
                const int lp = page_of(a, pos[e]);
                if (lp != seen) {
                    seen = lp;
                    page = checked_page(a, lp >= have                  ? free_page(off + (lp - have))
                                           : ONE && lp == page_of(a, s) ? page_s[run]
                                                                        : held_entry(a, b, lp));
                }
                if (page >= 0) slot[e] = page * a.page_size + (pos[e] - lp * a.page_size);
            }
        }
        if (TOKENS == 4 && i0 + TOKENS <= a.capacity) {
            *reinterpret_cast<int4 *>(a.slot_map + i0) = make_int4(slot[0], slot[1 % TOKENS], slot[2 % TOKENS], slot[3 % TOKENS]);
            if (a.positions) *reinterpret_cast<int4 *>(a.positions + i0) = make_int4(pos[0], pos[1 % TOKENS], pos[2 % TOKENS], pos[3 % TOKENS]);
        } else {
            for (int e = 0; e < TOKENS && i0 + e < a.capacity; ++e) {
                a.slot_map[i0 + e] = slot[e];
                if (a.positions) a.positions[i0 + e] = pos[e];
            }
        }
    }
}

diffqkv_status_t page_map_launch(int32_t batch, const int32_t *seq_lens, const int32_t *new_lens,
                                 int32_t *block_table, int32_t max_blocks, int32_t page_size, int32_t num_pages,
                                 const int32_t *free_pages, int32_t num_free, int32_t capacity, int32_t *query_start,
                                 int32_t *slot_map, int32_t *positions, int32_t *total_lens, int32_t *pages_used,
                                 int32_t *status, cudaStream_t stream) {
    if (batch < 1 || !seq_lens || !new_lens || !block_table || max_blocks < 1 || page_size < 1 || num_pages < 1 ||
        num_free < 0 || (num_free > 0 && !free_pages) || capacity < 0 || (capacity > 0 && !slot_map) || !query_start ||
        !total_lens || !pages_used)
        return DIFFQKV_ERR_INVALID_ARG;
    if ((long long)max_blocks * page_size > 0x7fffffffLL || (long long)num_pages * page_size > 0x7fffffffLL ||
        batch > (1 << 24))
        return DIFFQKV_ERR_UNSUPPORTED;
    const void *words[] = {seq_lens, new_lens, block_table, free_pages, query_start, total_lens, pages_used, status};
    for (const void *w : words)
        if (reinterpret_cast<uintptr_t>(w) & 3u) return DIFFQKV_ERR_MISALIGNED;
    if (!aligned16(slot_map) || !aligned16(positions)) return DIFFQKV_ERR_MISALIGNED;
    // outputs apart from inputs and from one another: CTAs that redo the sums would read another one's results
    struct Range {
        const void *p;
        long long words;
    };
    const Range in[] = {{seq_lens, batch}, {new_lens, batch}, {free_pages, num_free}};
    const Range out[] = {{block_table, (long long)batch * max_blocks}, {query_start, batch + 1}, {slot_map, capacity},
                         {positions, capacity}, {total_lens, batch}, {pages_used, 1}};
    auto meet = [](const Range &x, const Range &y) {
        const uintptr_t a = reinterpret_cast<uintptr_t>(x.p), b = reinterpret_cast<uintptr_t>(y.p);
        return x.p && y.p && a < b + 4 * (uintptr_t)y.words && b < a + 4 * (uintptr_t)x.words;
    };
    for (size_t i = 0; i < sizeof out / sizeof *out; ++i) {
        for (const Range &x : in)
            if (meet(out[i], x)) return DIFFQKV_ERR_INVALID_ARG;
        for (size_t j = 0; j < i; ++j)
            if (meet(out[i], out[j])) return DIFFQKV_ERR_INVALID_ARG;
    }
    DeviceInfo dev;
    const diffqkv_status_t st = current_device_info(&dev);
    if (st != DIFFQKV_OK) return st;

    PageMapArgs a;
    a.seq_lens = seq_lens;
    a.new_lens = new_lens;
    a.free_pages = free_pages;
    a.block_table = block_table;
    a.query_start = query_start;
    a.slot_map = slot_map;
    a.positions = positions;
    a.total_lens = total_lens;
    a.pages_used = pages_used;
    a.status = status ? status : dev.status_word;
    a.batch = batch;
    a.max_blocks = max_blocks;
    a.page_size = page_size;
    a.num_pages = num_pages;
    a.num_free = num_free;
    a.capacity = capacity;
    a.page_shift = -1;
    if ((page_size & (page_size - 1)) == 0)
        for (a.page_shift = 0; (1 << a.page_shift) < page_size;) ++a.page_shift;
    const int threads = batch <= kFewThreads ? kFewThreads : kManyThreads;
    a.per = (batch + threads - 1) / threads;
    // CTAs as many as the SMs hold, fewer where one sweep over the tokens takes fewer; a token a thread up to one and a
    // half such sweeps
    const long long most = (long long)dev.num_sms * (threads == kFewThreads ? 4 : 1);
    const int tok = 2LL * capacity <= 3LL * most * threads ? 1 : kMapTokens;
    const long long want = ((long long)capacity + threads * tok - 1) / (threads * tok);
    const int grid = (int)(want < 1 ? 1 : want > most ? most : want);
    auto launch = [&](auto one, auto four) { (tok == 1 ? one : four)<<<grid, threads, 0, stream>>>(a); };
    if (batch <= kFewThreads)
        launch(page_map_kernel<kFewThreads, true, 1>, page_map_kernel<kFewThreads, true, kMapTokens>);
    else if (batch <= kManyThreads)
        launch(page_map_kernel<kManyThreads, true, 1>, page_map_kernel<kManyThreads, true, kMapTokens>);
    else
        launch(page_map_kernel<kManyThreads, false, 1>, page_map_kernel<kManyThreads, false, kMapTokens>);
    return cudaGetLastError() == cudaSuccess ? DIFFQKV_OK : DIFFQKV_ERR_CUDA;
}

}  // namespace

}  // namespace diffqkv

extern "C" diffqkv_status_t diffqkv_page_map(int32_t batch, const int32_t *seq_lens, const int32_t *new_lens,
                                             int32_t *block_table, int32_t max_blocks, int32_t page_size,
                                             int32_t num_pages, const int32_t *free_pages, int32_t num_free,
                                             int32_t capacity, int32_t *query_start, int32_t *slot_map,
                                             int32_t *positions, int32_t *total_lens, int32_t *pages_used,
                                             int32_t *device_status_word, diffqkv_stream_t stream) {
    diffqkv::ApiRange nvtx_range("diffqkv_page_map");
    return diffqkv::page_map_launch(batch, seq_lens, new_lens, block_table, max_blocks, page_size, num_pages, free_pages,
                                    num_free, capacity, query_start, slot_map, positions, total_lens, pages_used,
                                    device_status_word, (cudaStream_t)stream);
}
