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
#include "common.cuh"
#include "internal.h"

namespace diffqkv {

namespace {

constexpr int kMapThreads = 512;
constexpr int kMapTokens = 4;  // consecutive tokens a thread maps (one 16-byte store per output)

struct PageMapArgs {
    const int32_t *seq_lens, *new_lens, *free_pages;
    int32_t *block_table, *query_start, *slot_map, *positions, *total_lens, *pages_used, *status;
    int32_t batch, max_blocks, page_size, num_pages, num_free, capacity;
    int32_t per;  // requests of one thread's run
};

struct Request {
    int s, n;      // cached positions and new tokens, after the checks
    int have, take;  // pages it holds and pages it takes
};

// Request b after the checks: lengths outside [0, max_blocks * page_size] add nothing.
__device__ __forceinline__ Request load_request(const PageMapArgs &a, int b, bool dropped, bool flag) {
    const int cap = a.max_blocks * a.page_size;
    const int s = __ldg(a.seq_lens + b), n = __ldg(a.new_lens + b);
    Request r;
    r.s = min(max(s, 0), cap);
    const bool bad = s < 0 || s > cap || n < 0 || n > cap - s;
    if (bad && flag) record_error(a.status, DIFFQKV_ERR_DEVICE_SEQLEN);
    r.n = bad || dropped ? 0 : n;
    r.have = r.s / a.page_size + (r.s % a.page_size != 0);
    const int t = r.s + r.n;
    r.take = t / a.page_size + (t % a.page_size != 0) - r.have;
    return r;
}

// Largest i in [0, n) with v[i] <= x (v ascending, v[0] <= x).
__device__ __forceinline__ int last_not_above(const long long *v, int n, long long x) {
    int lo = 0;
    while (n > 1) {
        const int half = n >> 1;
        if (v[lo + half] <= x) lo += half;
        n -= half;
    }
    return lo;
}

__global__ void __launch_bounds__(kMapThreads) page_map_kernel(const PageMapArgs a) {
    __shared__ long long tok_s[kMapThreads + 1];  // tokens before each run
    __shared__ long long pag_s[kMapThreads + 1];  // pages taken before each run
    __shared__ long long warp_t[kMapThreads / 32], warp_p[kMapThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int b0 = min(a.batch, tid * a.per), b1 = min(a.batch, b0 + a.per);
    const bool first_cta = blockIdx.x == 0;

    long long t = 0, p = 0;
    for (int b = b0; b < b1; ++b) {
        const Request r = load_request(a, b, false, first_cta);
        t += r.n;
        p += r.take;
    }
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
    long long bt = 0, bp = 0;
    for (int w = 0; w < warp; ++w) {
        bt += warp_t[w];
        bp += warp_p[w];
    }
    tok_s[tid] = bt + it - t;
    pag_s[tid] = bp + ip - p;
    if (tid == kMapThreads - 1) {
        tok_s[kMapThreads] = bt + it;
        pag_s[kMapThreads] = bp + ip;
    }
    __syncthreads();
    // a step that does not fit the token buffer or the free list is dropped as a whole
    const bool no_room = tok_s[kMapThreads] > a.capacity;
    const bool dropped = no_room || pag_s[kMapThreads] > a.num_free;
    if (dropped && first_cta && tid == 0)
        record_error(a.status, no_room ? DIFFQKV_ERR_DEVICE_SEQLEN : DIFFQKV_ERR_DEVICE_PAGE);
    const int tokens = dropped ? 0 : (int)tok_s[kMapThreads];
    const int pages = dropped ? 0 : (int)pag_s[kMapThreads];

    // per-request outputs: run i belongs to CTA i mod grid
    if (tid % gridDim.x == blockIdx.x) {
        int at = dropped ? 0 : (int)tok_s[tid];
        for (int b = b0; b < b1; ++b) {
            const Request r = load_request(a, b, dropped, false);
            a.query_start[b] = at;
            a.total_lens[b] = r.s + r.n;
            at += r.n;
        }
    }
    if (first_cta && tid == 0) {
        a.query_start[a.batch] = tokens;
        a.pages_used[0] = pages;
    }
    const int runs = (a.batch + a.per - 1) / a.per;
    const int stride = gridDim.x * kMapThreads;

    // table entries of the pages taken
    for (int k = blockIdx.x * kMapThreads + tid; k < pages; k += stride) {
        const int run = last_not_above(pag_s, runs, k);
        int b = run * a.per;
        long long off = pag_s[run];
        Request r = load_request(a, b, false, false);
        while (k >= off + r.take) {
            off += r.take;
            r = load_request(a, ++b, false, false);
        }
        int page = __ldg(a.free_pages + k);
        if (page < 0 || page >= a.num_pages) {
            record_error(a.status, DIFFQKV_ERR_DEVICE_PAGE);
            page = -1;
        }
        a.block_table[(size_t)b * a.max_blocks + r.have + (int)(k - off)] = page;
    }

    // slots and positions, kMapTokens consecutive tokens a thread
    for (long long i0 = (long long)(blockIdx.x * kMapThreads + tid) * kMapTokens; i0 < a.capacity;
         i0 += (long long)stride * kMapTokens) {
        int slot[kMapTokens], pos[kMapTokens];
#pragma unroll
        for (int e = 0; e < kMapTokens; ++e) slot[e] = pos[e] = -1;
        if (i0 < tokens) {
            const int run = last_not_above(tok_s, runs, i0);
            int b = run * a.per;
            long long at = tok_s[run];
            long long off = pag_s[run];
            Request r = load_request(a, b, false, false);
            int seen = -1, page = -1;  // logical page last looked up, and its pool page
#pragma unroll
            for (int e = 0; e < kMapTokens; ++e) {
                const long long i = i0 + e;
                if (i >= tokens) break;
                while (i >= at + r.n) {
                    at += r.n;
                    off += r.take;
                    r = load_request(a, ++b, false, false);
                    seen = -1;
                }
                pos[e] = r.s + (int)(i - at);
                const int lp = pos[e] / a.page_size;
                if (lp != seen) {
                    seen = lp;
                    page = lp < r.have ? a.block_table[(size_t)b * a.max_blocks + lp]
                                       : __ldg(a.free_pages + off + (lp - r.have));
                    if (page < 0 || page >= a.num_pages) {
                        record_error(a.status, DIFFQKV_ERR_DEVICE_PAGE);
                        page = -1;
                    }
                }
                if (page >= 0) slot[e] = page * a.page_size + pos[e] % a.page_size;
            }
        }
        if (i0 + kMapTokens <= a.capacity) {
            *reinterpret_cast<int4 *>(a.slot_map + i0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
            if (a.positions) *reinterpret_cast<int4 *>(a.positions + i0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
        } else {
            for (int e = 0; i0 + e < a.capacity; ++e) {
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
    a.per = (batch + kMapThreads - 1) / kMapThreads;
    // enough CTAs for one sweep over the tokens, at most two a SM
    const long long want = ((long long)capacity + kMapThreads * kMapTokens - 1) / (kMapThreads * kMapTokens);
    const long long most = 2LL * dev.num_sms;
    const int grid = (int)(want < 1 ? 1 : want > most ? most : want);
    page_map_kernel<<<grid, kMapThreads, 0, stream>>>(a);
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
