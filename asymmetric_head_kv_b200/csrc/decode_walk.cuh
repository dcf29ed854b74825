// decode_walk.cuh -- the tile walk shared by the split/combine decode kernels.
//
// A work unit is (batch b, K head g).  The tiles of all units are concatenated in (b, g) order and cut
// into equal contiguous ranges, one per CTA, so a range may begin or end inside a unit.
#pragma once

#include "common.cuh"

namespace diffqkv {

// Position of the tile walk: unit (b, g), tile i of nt, first global tile P.
struct Walker {
    int b, g, i, nt, T;
    long long P;
};

__device__ __forceinline__ int clamp_len(int v, int t_max) { return v < 0 ? 0 : (v > t_max ? t_max : v); }

// Args: seq_lens, batch, n_k, t_max.
template <int TT, class Args>
__device__ __forceinline__ void walker_advance(Walker &w, const Args &a) {
    if (++w.i < w.nt) return;
    w.P += w.nt;
    w.i = 0;
    if (++w.g < a.n_k) return;
    w.g = 0;
    for (;;) {
        if (++w.b >= a.batch) { w.nt = 0; return; }
        w.T = clamp_len(__ldg(a.seq_lens + w.b), a.t_max);
        w.nt = (w.T + TT - 1) / TT;
        if (w.nt > 0) return;
    }
}

// CTA that owns global tile t when N tiles are cut into G equal ranges
// [floor(c N / G), floor((c+1) N / G)).
__device__ __forceinline__ long long cta_of_tile(long long t, long long N, long long G) {
    return ((t + 1) * G - 1) / N;
}

// Counter (of `counters`) in which the CTAs of a unit that more than one of them has a piece of count these pieces: the
// unit's own where there are as many counters as units, else that of the unit's first CTA.  A CTA is that for one such
// unit at most, the one its range ends inside of.
__device__ __forceinline__ long long counter_of(long long u, long long first, long long units, int counters) {
    return units <= counters ? u : first;
}

// Run by one warp: total tile count N and the unit holding the first tile of CTA c of G, into
// scan_s = {N, P0, b0 << 32 | g0, i0}.  CTA 0 flags lengths outside [0, t_max] (status).
template <int TT, class Args>
__device__ __forceinline__ void walker_scan(const Args &a, long long c, long long G, int lane, long long *scan_s) {
    long long acc = 0;
    for (int base = 0; base < a.batch; base += 32) {
        const int b = base + lane;
        int nt = 0;
        if (b < a.batch) {
            const int raw = __ldg(a.seq_lens + b);
            if (c == 0 && (raw < 0 || raw > a.t_max)) record_error(a.status, DIFFQKV_ERR_DEVICE_SEQLEN);
            nt = (clamp_len(raw, a.t_max) + TT - 1) / TT;
        }
        long long incl = (long long)nt * a.n_k;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += y;
        }
        acc += __shfl_sync(0xffffffffu, incl, 31);
    }
    const long long N = acc;
    // never more CTAs than tiles: every CTA range is then non-empty
    const long long Ge = N < G ? N : G;
    const long long t_begin = (c < Ge) ? (c * N) / Ge : N;
    long long P0 = 0;
    int b0 = a.batch, g0 = 0, i0 = 0;
    acc = 0;
    bool found = false;
    for (int base = 0; base < a.batch && !found && N > 0; base += 32) {
        const int b = base + lane;
        const int nt = b < a.batch ? (clamp_len(__ldg(a.seq_lens + b), a.t_max) + TT - 1) / TT : 0;
        const long long w = (long long)nt * a.n_k;
        long long incl = w;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += y;
        }
        const long long excl = incl - w;
        const bool hit = b < a.batch && nt > 0 && acc + excl <= t_begin && t_begin < acc + incl;
        const unsigned m = __ballot_sync(0xffffffffu, hit);
        if (m) {
            const int L = __ffs(m) - 1;
            const long long start = __shfl_sync(0xffffffffu, acc + excl, L);
            const int ntL = __shfl_sync(0xffffffffu, nt, L);
            const long long within = t_begin - start;
            b0 = base + L;
            g0 = (int)(within / ntL);
            i0 = (int)(within % ntL);
            P0 = start + (long long)g0 * ntL;
            found = true;
        }
        acc += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) {
        scan_s[0] = N;
        scan_s[1] = P0;
        scan_s[2] = ((long long)b0 << 32) | (unsigned)g0;
        scan_s[3] = i0;
    }
}

}  // namespace diffqkv
