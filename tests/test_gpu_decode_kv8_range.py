"""Decode over an 8-bit cache whose scales lie many powers of two apart, where the large one carries no weight.

The reference of a head's weights is the largest p_j 2^(V exponent of j) of a real position, so a V block of large
scale costs the others nothing where its scores make it weightless."""
import numpy as np
import pytest
import torch

import asymmetric_head_kv_b200 as ak
import oracle
from kv8_inputs import attention_tolerance, dequant, pools, queries, tables
from oracle import kv8
from workloads import DIFFQKV, Shape

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


def _check_decode(out, q, p, table, n, scale):
    """One sequence of n positions against fp64.  As kv8_inputs.attention_tolerance, but that the weights' absolute term,
    positions * 2^-28 * 448, is taken of the largest p_j 2^(exponent of j) over the positions, not of the largest p times
    the largest scale: the reference of the split is that maximum over the positions so far, never above it."""
    k, v = dequant(p)
    lens, n_q = [n], q.shape[1]
    ref = oracle.decode_paged(q, k, v, table, lens, scale)
    mag = oracle.decode_paged(q, k, v.abs(), table, lens, scale)
    kb = oracle.gather_paged(k, table, lens).double()[0, :n].repeat_interleave(n_q // k.shape[2], 1)
    s = (torch.einsum("hd,jhd->hj", q[0].double(), kb) * scale).numpy()
    smag = (torch.einsum("hd,jhd->hj", q[0].double().abs(), kb.abs()) * scale).amax(1).numpy()
    sb = v.shape[1] // p[3].shape[1]
    j = torch.arange(n)
    e = kv8.exponents(p[3])[table[0, j // v.shape[1]].numpy(), (j % v.shape[1] // sb).numpy()]  # [n, n_v]
    w = np.exp(s - s.max(1, keepdims=True)) * np.exp2(np.repeat(e, n_q // v.shape[2], 1).T.astype(np.float64))
    tol = attention_tolerance(ref, mag, [s], smag[None], 448.0 * w.max(1)[None])
    over = np.abs(out.double().cpu().numpy() - ref) - tol
    assert over.max() <= 0, f"{over.max()} over at {np.unravel_index(over.argmax(), over.shape)}"
    assert np.abs(ref).max(axis=2).min() > 0


@pytest.mark.parametrize("rise", [0, 16, 24, 28, 31, 32, 33, 48, 64, 120])
@pytest.mark.parametrize("at", [[0], [3], [70]], ids=["first tile", "same tile", "later tile"])
def test_decode_keeps_its_bits_beside_a_weightless_block(cuda_device, rise, at):
    for shape, length in ((Shape(16, 4, 16, 64, 128), 64 if at == [3] else 1200), (Shape(8, 8, 2, 128, 64), 1300)):
        p, table = _outliers(shape, length, at, rise, seed=rise)
        q = queries(1, shape, 1).abs()
        out = ak.decode_paged_kv8(q.to(cuda_device), *[t.to(cuda_device) for t in p], table.to(cuda_device),
                                  torch.tensor([length], dtype=torch.int32, device=cuda_device), scale=shape.scale)
        _check_decode(out, q, p, table, length, shape.scale)


def test_decode_with_scales_over_the_whole_range(cuda_device):
    """Every block's V exponent and its keys' drawn apart, heads of one K head on V heads of their own."""
    for seed, shape in ((1, DIFFQKV), (2, Shape(16, 2, 8, 64, 128)), (3, Shape(16, 1, 16, 64, 64))):
        length = 2000
        num, table = tables([length], 16, 125, seed)
        p = pools(num, 16, 16, shape, seed, 1)
        g = torch.Generator().manual_seed(seed)
        p[3][:] = torch.randint(20, 200, p[3].shape, generator=g).to(torch.uint8)
        p[2][:] = torch.randint(116, 124, p[2].shape, generator=g).to(torch.uint8)
        q = queries(1, shape, seed)
        out = ak.decode_paged_kv8(q.to(cuda_device), *[t.to(cuda_device) for t in p], table.to(cuda_device),
                                  torch.tensor([length], dtype=torch.int32, device=cuda_device), scale=shape.scale)
        _check_decode(out, q, p, table, length, shape.scale)
