"""Seeded 8-bit paged caches for the tests of the calls that read them."""
import numpy as np
import torch

import oracle
from oracle import kv8


def pools(num_pages, page, sb, shape, seed, spread=2):
    """(k_pages, v_pages, k_scales, v_scales): normal codes, scale exponents within +-spread of 2^-6, on the CPU."""
    g = torch.Generator().manual_seed(seed)
    out = []
    for n, d in ((shape.n_k, shape.d_k), (shape.n_v, shape.d_v)):
        x = torch.randn((num_pages, page, n, d), generator=g) * 64
        out.append(x.clamp(-448, 448).to(torch.float8_e4m3fn))
    for n in (shape.n_k, shape.n_v):
        out.append((121 + torch.randint(-spread, spread + 1, (num_pages, page // sb, n), generator=g)).to(torch.uint8))
    return out


def tables(lens, page, max_blocks, seed, spare=2):
    """(num_pages, block_table): distinct pages in random order, -1 where unused."""
    held = [-(-int(t) // page) for t in lens]
    num_pages = sum(held) + spare
    perm = torch.randperm(num_pages, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    table = torch.full((len(lens), max_blocks), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(held):
        table[b, :n] = perm[at:at + n]
        at += n
    return num_pages, table


def queries(rows, shape, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn((rows, shape.n_q, shape.d_k), generator=g).to(torch.bfloat16)


def stale(codes, table, lens, page):
    """Copies of the pools with every row that no sequence holds set to the NaN code."""
    out = []
    for c in codes:
        raw = torch.full_like(c.view(torch.uint8), 0x7F)
        for b, n in enumerate(lens):
            for p0 in range(0, int(n), page):
                pg, k = int(table[b, p0 // page]), min(page, int(n) - p0)
                raw[pg, :k] = c.view(torch.uint8)[pg, :k]
        out.append(raw.view(torch.float8_e4m3fn))
    return out


def dequant(p):
    """bf16 pools of the same values (exact)."""
    return kv8.dequant(p[0], p[2]), kv8.dequant(p[1], p[3])


def attention_tolerance(ref, mag, scores, smag, vmax):
    """What decode outputs [B, n_q, d_v] may be off by, element by element.

    out = sum_j p_j v_j with bf16 output: its rounding, 2^-8 |out| (and 2^-16 for the double counting of it).  The three
    e4m3 terms of a weight p_j 2^(its V block's exponent) hold 12 bits, so sum_j p_j |v_j| times 2^-12, as much again for
    the fp32 sums of terms, rows and splits: 2^-11; or 2^-28 of the largest such weight (at most p_max 2^(largest
    exponent), codes are at most 448): positions * 2^-28 * p_max * vmax.  A score's fp32 sum over d elements in the
    block-addition model of the tensor cores is off by at most d 2^-23 (1 + 1/16) of S = sum |q k| scale, and moves its
    weight, and through the row sum every weight, by that much: 2 * 128 * 2^-23 * 1.0625 * S <= 2^-14.9 S.

    ``mag``: sum_j p_j |v_j|; ``scores``: list of [n_q, positions]; ``smag`` [B, n_q]: largest S; ``vmax`` [B, n_q]: 448 *
    2^(largest exponent)."""
    tol = (2 ** -8 + 2 ** -16) * np.abs(ref) + (2 ** -11 + 2 ** -14.9 * smag[:, :, None]) * mag
    for b, s in enumerate(scores):
        if s.shape[1]:
            p = np.exp(s - s.max(1, keepdims=True))
            tol[b] += (s.shape[1] * 2.0 ** -28 / p.sum(1) * vmax[b])[:, None]
    return tol


def check_decode(out, q, p, table, lens, scale, what=""):
    """Decode output against the fp64 oracle on the pools ``p`` (codes and scales), by :func:`attention_tolerance`."""
    k, v = dequant(p)
    ref = oracle.decode_paged(q, k, v, table, lens, scale)
    mag = oracle.decode_paged(q, k, v.abs(), table, lens, scale)
    rows = oracle.gather_paged(k, table, lens).double()
    B, n_q, _ = q.shape
    n_k, n_v = k.shape[2], v.shape[2]
    scores, smag, vmax = [], np.zeros((B, n_q)), np.zeros((B, n_q))
    for b, n in enumerate(int(t) for t in lens):
        kb = rows[b, :n].repeat_interleave(n_q // n_k, 1)
        scores.append((torch.einsum("hd,jhd->hj", q[b].double(), kb) * scale).numpy())
        smag[b] = (torch.einsum("hd,jhd->hj", q[b].double().abs(), kb.abs()) * scale).amax(1).numpy() if n else 0.0
        held = table[b, :-(-n // v.shape[1])].long()
        e = kv8.exponents(p[3][held]).max(axis=(0, 1), initial=-120)
        vmax[b] = 448.0 * np.exp2(np.repeat(e, n_q // n_v).astype(np.float64))
    tol = attention_tolerance(ref, mag, scores, smag, vmax)
    got = out.double().cpu().numpy()
    assert np.isfinite(got).all(), what
    over = np.abs(got - ref) - tol
    assert over.max(initial=-1.0) <= 0, f"{what}: {over.max()} over at {np.unravel_index(over.argmax(), over.shape)}"


def check_prefill(out, q, start, p, table, lens, scale, what=""):
    """Prefill rows [tokens, n_q, d_v] against the fp64 formula on the pools ``p``: row r of request b (rows start[b] ..
    start[b + 1] - 1) sits at position lens[b] - n_b + r.

    Tolerance: the bf16 rounding, 2^-8 |out|; f16 weights, 2^-11 of each (and 2^-31 of the largest, absolutely), as
    much again for fp32 sums and the exponentials: 2^-10 * sum_j p_j |v_j| + positions * 2^-31 p_max max|v|; V rows in f16
    below the range its exponent reference leaves: 2^-25 of the largest exponent; a score's error as in
    :func:`attention_tolerance`."""
    k, v = dequant(p)
    n_q = q.shape[1]
    n_k, n_v = k.shape[2], v.shape[2]
    got = out.double().cpu().numpy()
    kg, vg = oracle.gather_paged(k, table, lens).double(), oracle.gather_paged(v, table, lens).double()
    for b, n in enumerate(int(t) for t in lens):
        rows = int(start[b + 1]) - int(start[b])
        if rows == 0:
            continue
        pos = torch.arange(n - rows, n)
        held = table[b, :-(-n // v.shape[1])].long()
        e = kv8.exponents(p[3][held]).max(axis=(0, 1), initial=-120)
        for h in range(n_q):
            qh = q[start[b]:start[b + 1], h].double()
            kh, vh = kg[b, :n, h // (n_q // n_k)], vg[b, :n, h // (n_q // n_v)]
            s = (qh @ kh.T * scale).masked_fill(torch.arange(n)[None] > pos[:, None], float("-inf"))
            w = torch.softmax(s, 1)
            ref, mag = w @ vh, w @ vh.abs()
            smag = ((qh.abs() @ kh.abs().T) * scale).masked_fill(torch.isinf(s), 0).amax(1, keepdim=True)
            top = 2.0 ** float(e[h // (n_q // n_v)])
            tol = (2 ** -8 + 2 ** -16) * ref.abs() + (2 ** -10 + 2 ** -14.9 * smag) * mag + 2 ** -25 * top + \
                (pos + 1)[:, None] * 2.0 ** -31 * w.amax(1, keepdim=True) * 448 * top
            g = torch.from_numpy(got[start[b]:start[b + 1], h])
            assert torch.isfinite(g).all(), f"{what} request {b} head {h}"
            over = ((g - ref).abs() - tol).max().item()
            assert over <= 0, f"{what} request {b} head {h}: {over} over"
