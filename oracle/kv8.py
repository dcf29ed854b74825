"""Definitions of the 8-bit paged cache and of the page bookkeeping, in plain Python and numpy -- TEST
INFRASTRUCTURE ONLY (see the package docstring).

A cache element is code * 2^(byte - 127), code an e4m3 number.  Every such value is a bf16 number (4 significant
bits, exponents inside bf16's), so attention over an 8-bit cache is the fp64 oracle over the bf16 pools that
:func:`dequant` returns, with no rounding in between.
"""
from __future__ import annotations

import numpy as np
import torch

E_MIN, E_MAX = -120, 119


def code_values() -> np.ndarray:
    """Value of each of the 256 e4m3 codes (bias 7, no infinities, 0x7f and 0xff NaN)."""
    v = np.empty(256)
    for c in range(256):
        sign, e, m = (-1.0 if c & 128 else 1.0), (c >> 3) & 15, c & 7
        if e == 15 and m == 7:
            v[c] = np.nan
        else:
            v[c] = sign * (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
    return v


_VALUES = code_values()
_POS = _VALUES[:127]  # ascending magnitudes 0 .. 448


def encode(x) -> np.ndarray:
    """Nearest e4m3 code of each value, ties to the even code; |x| > 448 saturates, NaN is 0x7f."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(np.where(np.isnan(x), 0.0, x)), 448.0)
    hi = np.clip(np.searchsorted(_POS, a, side="left"), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _POS[lo], _POS[hi] - a
    take_lo = (dl < dh) | ((dl == dh) & (lo % 2 == 0))
    code = np.where(take_lo, lo, hi).astype(np.uint8) | np.where(np.signbit(x), 0x80, 0).astype(np.uint8)
    return np.where(np.isnan(x), 0x7F, code).astype(np.uint8)


def codes_of(pages) -> np.ndarray:
    return pages.detach().cpu().view(torch.uint8).numpy()


def exponents(scales) -> np.ndarray:
    s = scales.detach().cpu().numpy() if isinstance(scales, torch.Tensor) else np.asarray(scales)
    return np.clip(s.astype(np.int64) - 127, E_MIN, E_MAX)


def dequant(pages, scales) -> torch.Tensor:
    """bf16 pool [num_pages, page_size, heads, d] of the values an 8-bit pool stands for (exact)."""
    c, e = codes_of(pages), exponents(scales)
    sb = c.shape[1] // e.shape[1]
    v = _VALUES[c] * np.exp2(np.repeat(e, sb, axis=1)[:, :, :, None].astype(np.float64))
    out = torch.from_numpy(v).to(torch.bfloat16)
    assert np.array_equal(out.double().numpy(), v, equal_nan=True)
    return out


def least_exponent(amax: float) -> int:
    """Least e in [E_MIN, E_MAX] with amax <= 448 * 2^e (E_MAX where there is none)."""
    e = E_MIN
    while e < E_MAX and amax > 448.0 * 2.0 ** e:
        e += 1
    return e


def store(codes: np.ndarray, scales: np.ndarray, x, slots) -> None:
    """Writes rows x [T, heads, d] (values) into uint8 codes [pages, P, heads, d] and scale bytes
    [pages, P / sb, heads], in place, by the definition: block by block, head by head."""
    x = np.asarray(x, np.float64)
    pages, P, heads, _ = codes.shape
    sb = P // scales.shape[1]
    groups = {}
    for t, s in enumerate(int(v) for v in slots):
        if 0 <= s < pages * P:
            groups.setdefault(s // sb, []).append((s % sb, t))
    for blk, members in groups.items():
        page, part = divmod(blk, P // sb)
        low = min(r for r, _ in members)
        for h in range(heads):
            rows = np.stack([x[t, h] for _, t in members])
            fin = np.abs(rows[np.isfinite(rows)])
            e = least_exponent(float(fin.max(initial=0.0)))
            if low > 0:
                old = int(np.clip(int(scales[page, part, h]) - 127, E_MIN, E_MAX))
                e = max(e, old)
                if e > old:
                    at = slice(part * sb, part * sb + low)
                    codes[page, at, h] = encode(_VALUES[codes[page, at, h]] * 2.0 ** (old - e))
                    scales[page, part, h] = e + 127
            else:
                scales[page, part, h] = e + 127
            for r, t in members:
                codes[page, part * sb + r, h] = encode(x[t, h] * 2.0 ** -e)


def page_map(seq_lens, new_lens, table, free_pages, page_size, num_pages, capacity):
    """Returns dict(block_table, query_start, slot_map, positions, total_lens, pages_used, status)."""
    table = np.array(table, np.int64)
    cap_pos = table.shape[1] * page_size
    status = 0

    def flag(code):
        nonlocal status
        status = status or code

    s, n = [], []
    for a, b in zip(map(int, seq_lens), map(int, new_lens)):
        bad = a < 0 or a > cap_pos or b < 0 or a + b > cap_pos
        if bad:
            flag(7)
        s.append(min(max(a, 0), cap_pos))
        n.append(0 if bad else b)
    pages = lambda v: -(-v // page_size)  # noqa: E731
    taken = sum(pages(a + b) - pages(a) for a, b in zip(s, n))
    if sum(n) > capacity or taken > len(free_pages):
        flag(7 if sum(n) > capacity else 10)
        n = [0] * len(n)
    slot, pos, start, used = [], [], [0], 0
    for b, (a, m) in enumerate(zip(s, n)):
        held = pages(a)
        for i in range(held, pages(a + m)):
            p = int(free_pages[used])
            used += 1
            if not 0 <= p < num_pages:
                flag(10)
                p = -1
            table[b, i] = p
        for i in range(m):
            p = int(table[b, (a + i) // page_size])
            if not 0 <= p < num_pages:
                flag(10)
                p = -1
            pos.append(a + i)
            slot.append(-1 if p < 0 else p * page_size + (a + i) % page_size)
        start.append(start[-1] + m)
    pad = [-1] * (capacity - len(slot))
    return dict(block_table=table, query_start=np.array(start), slot_map=np.array(slot + pad, np.int64),
                positions=np.array(pos + pad, np.int64), total_lens=np.array([a + m for a, m in zip(s, n)]),
                pages_used=np.array([used]), status=status)
