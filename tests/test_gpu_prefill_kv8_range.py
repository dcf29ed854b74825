"""Prefill over an 8-bit cache whose scales lie many powers of two apart: codes and scales are applied exactly, whatever
their neighbours' are."""
import pytest
import torch

import asymmetric_head_kv_b200 as ak
import oracle
from kv8_inputs import dequant, pools, queries, tables
from oracle import kv8
from workloads import Shape

pytestmark = pytest.mark.gpu


def _outliers(shape, length, at, rise, seed, k_byte=123, low=110):
    """Pools whose V blocks (16 positions) lie at exponent low - 127, but for block(s) ``at``, ``rise`` above: their keys
    are -448 2^(k_byte - 127) in every element, which a query without negative elements scores far below the others."""
    num, table = tables([length], 16, -(-length // 16), seed)
    p = pools(num, 16, 16, shape, seed, 1)
    p[3][:] = low
    for i in at:
        pg = int(table[0, i])
        p[0].view(torch.uint8)[pg] = 0xFE
        p[2][pg] = k_byte
        p[3][pg] = low + rise
    return p, table


def _run(p, table, q, start, lens, scale, dev):
    i32 = lambda x: torch.as_tensor(x, dtype=torch.int32).to(dev)  # noqa: E731
    return ak.prefill_paged_kv8(q.to(dev), i32(start), *[t.to(dev) for t in p], i32(table), i32(lens), scale=scale)


def _check(out, q, start, p, table, lens, scale):
    """Against the fp64 formula.  The terms of kv8_inputs.check_prefill but the two that take the cache's largest scale: K and
    V are exact here, and a weight (its V block's scale included) that f16 holds as a subnormal is off by 2^-25 where the
    reference is held at 2^7, the reference being at most 2^8 above the largest weight of a real position: 2^-24 of
    that, for each position and up to 448."""
    k, v = dequant(p)
    n_q, P = q.shape[1], v.shape[1]
    n_k, n_v, sb = k.shape[2], v.shape[2], P // p[3].shape[1]
    got = out.double().cpu()
    assert torch.isfinite(got[:start[-1]]).all()
    kg, vg = oracle.gather_paged(k, table, lens).double(), oracle.gather_paged(v, table, lens).double()
    for b, n in enumerate(lens):
        rows = slice(start[b], start[b + 1])
        pos = torch.arange(n - (start[b + 1] - start[b]), n)
        j = torch.arange(n)
        e = torch.from_numpy(kv8.exponents(p[3]))[table[b, j // P].long(), j % P // sb].double()  # [n, n_v]
        for h in range(n_q):
            qh = q[rows, h].double()
            kh, vh = kg[b, :n, h // (n_q // n_k)], vg[b, :n, h // (n_q // n_v)]
            s = (qh @ kh.T * scale).masked_fill(j[None] > pos[:, None], float("-inf"))
            w = torch.softmax(s, 1)
            ref, mag = w @ vh, w @ vh.abs()
            smag = ((qh.abs() @ kh.abs().T) * scale).masked_fill(torch.isinf(s), 0).amax(1, keepdim=True)
            top = (w * torch.exp2(e[:, h // (n_q // n_v)])).amax(1, keepdim=True)
            tol = (2 ** -8 + 2 ** -16) * ref.abs() + (2 ** -10 + 2 ** -14.9 * smag) * mag + \
                (pos + 1)[:, None] * 2.0 ** -24 * 448 * top
            over = ((got[rows, h] - ref).abs() - tol).max().item()
            assert over <= 0, f"request {b} head {h}: {over} over"


@pytest.mark.parametrize("rise", [8, 9, 14, 23, 24, 25, 30, 33, 48, 80, 120])
@pytest.mark.parametrize("at", [[0], [3], [1, 70]])
def test_a_weightless_block_of_large_scale_costs_nothing(cuda_device, rise, at):
    for shape, rows, length in ((Shape(4, 2, 4, 64, 128), 300, 1200), (Shape(2, 1, 2, 128, 64), 1150, 1150),
                                (Shape(2, 2, 1, 64, 64), 40, 3000)):
        p, table = _outliers(shape, length, at, rise, seed=rise)
        q = queries(rows, shape, 1).abs()
        out = _run(p, table, q, [0, rows], [length], shape.scale, cuda_device)
        _check(out, q, [0, rows], p, table, [length], shape.scale)


@pytest.mark.parametrize("sb", [16, 1])
def test_scales_over_the_whole_range(cuda_device, sb):
    for seed, shape in ((1, Shape(4, 1, 4, 64, 128)), (2, Shape(4, 2, 2, 128, 64)), (3, Shape(2, 1, 2, 64, 64))):
        lens, rows = [700, 2000], [700, 5]
        num, table = tables(lens, 16, 125, seed)
        p = pools(num, 16, sb, shape, seed, 1)
        g = torch.Generator().manual_seed(seed)
        p[3][:] = torch.randint(20, 200, p[3].shape, generator=g).to(torch.uint8)
        p[2][:] = torch.randint(90, 124, p[2].shape, generator=g).to(torch.uint8)
        q = queries(sum(rows), shape, seed)
        out = _run(p, table, q, [0, 700, 705], lens, shape.scale, cuda_device)
        _check(out, q, [0, 700, 705], p, table, lens, shape.scale)


@pytest.mark.parametrize("below", [15, 16, 20, 25, 36, 60])
def test_keys_far_below_others_of_their_tile(cuda_device, below):
    """K blocks 2^below under their tile's largest, with scores of order one there: the queries are large, and the large
    block's keys zero."""
    shape, length = Shape(2, 1, 2, 64, 64), 150
    num, table = tables([length], 16, 10, 1)
    p = pools(num, 16, 16, shape, 1, 0)
    p[2][:] = 127 - below
    for i in (0, 7):
        p[2][int(table[0, i])] = 127
        p[0].view(torch.uint8)[int(table[0, i])] = 0
    q = (queries(length, shape, 1).float() * 2.0 ** (below - 6)).to(torch.bfloat16)
    out = _run(p, table, q, [0, length], [length], 0.125, cuda_device)
    _check(out, q, [0, length], p, table, [length], 0.125)


def test_queries_that_are_not_finite_beside_mixed_tiles(cuda_device):
    """Their rows are NaN, the others as they were."""
    shape, length = Shape(2, 1, 2, 64, 128), 200
    p, table = _outliers(shape, length, [1, 6], 40, seed=1)
    q = queries(length, shape, 1).abs()
    clean = _run(p, table, q, [0, length], [length], shape.scale, cuda_device)
    q[17, 0, 3], q[150, 1, 60] = float("inf"), float("nan")
    out = _run(p, table, q, [0, length], [length], shape.scale, cuda_device)
    want = torch.zeros_like(clean, dtype=torch.bool)
    want[17, 0], want[150, 1] = True, True
    assert torch.equal(torch.isnan(out), want) and torch.equal(out[~want], clean[~want])
