"""Pins of the 8-bit cache's oracle: the e4m3 table, the rounding, the scale rule and the page bookkeeping."""
import numpy as np
import pytest
import torch

import oracle
from oracle import kv8


def test_code_table_is_e4m3():
    v = kv8.code_values()
    ref = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(v, ref, equal_nan=True)


def test_encode_rounds_to_nearest_even():
    x = torch.randn(20000, generator=torch.Generator().manual_seed(0)).double() * 40
    x = torch.cat([x.clamp(-448, 448), x * 1e-4, torch.linspace(-448, 448, 4097, dtype=torch.float64)])
    got = kv8.encode(x.numpy())
    want = x.float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    # torch rounds the binary32 value; these are exact in it
    same = x.float().double().numpy() == x.numpy()
    assert same.sum() > 4000
    assert np.array_equal(got[same], want[same])
    assert kv8.encode([500.0, -np.inf, np.nan, 17.0, 19.0, 2.0 ** -10, 3 * 2.0 ** -10]).tolist() == \
        [0x7E, 0xFE, 0x7F, kv8.encode(16.0), kv8.encode(20.0), 0, 2]


@pytest.mark.parametrize("amax,e", [(448.0, 0), (448.5, 1), (449.0, 1), (1.75, -8), (1.7578125, -7), (0.0, -120),
                                    (2.0 ** -133, -120), (2.9e38, 119), (3.38e38, 119)])
def test_scale_rule(amax, e):
    assert kv8.least_exponent(amax) == e


def test_store_by_hand():
    codes = np.zeros((2, 8, 1, 2), np.uint8)
    scales = np.full((2, 2, 1), 127, np.uint8)
    kv8.store(codes, scales, [[[448.0, 1.0]], [[-7.0, 2.0]]], [8, 9])       # page 1, rows 0 and 1 of block 0
    assert scales[1, 0, 0] == 127 and (kv8._VALUES[codes[1, :2, 0]] == [[448, 1], [-7, 2]]).all()
    kv8.store(codes, scales, [[[896.0, 32.0]]], [10])                        # row 2 doubles the scale
    assert scales[1, 0, 0] == 128 and (kv8._VALUES[codes[1, :3, 0]] == [[224, 0.5], [-3.5, 1], [448, 16]]).all()
    kv8.store(codes, scales, [[[1.0, 2.0]]], [8])                            # row 0 begins the block anew
    assert scales[1, 0, 0] == 127 - 7 and (kv8._VALUES[codes[1, 0, 0]] == [128, 256]).all()
    assert scales[1, 1, 0] == 127 and not codes[0].any() and not codes[1, 4:].any()


def test_dequantised_pool_is_bf16_at_every_code_and_scale():
    codes = torch.arange(256, dtype=torch.uint8).repeat(1, 8, 1, 1).view(torch.float8_e4m3fn)
    for byte in (0, 7, 60, 127, 200, 247, 255):
        kv8.dequant(codes, torch.full((1, 1, 1), byte, dtype=torch.uint8))   # asserts exactness


def test_page_map_by_hand():
    r = kv8.page_map([3, 0, 4], [2, 0, 5], [[5, -1, -1], [-1, -1, -1], [6, -1, -1]], [9, 8, 7], 4, 10, 9)
    assert r["block_table"].tolist() == [[5, 9, -1], [-1, -1, -1], [6, 8, 7]]
    assert r["query_start"].tolist() == [0, 2, 2, 7] and r["total_lens"].tolist() == [5, 0, 9]
    assert r["slot_map"].tolist() == [23, 36, 32, 33, 34, 35, 28, -1, -1]
    assert r["positions"].tolist() == [3, 4, 4, 5, 6, 7, 8, -1, -1]
    assert r["pages_used"].tolist() == [3] and r["status"] == 0
    short = kv8.page_map([3, 0], [2, 1], [[5, -1], [-1, -1]], [9], 4, 10, 8)
    assert short["status"] == 10 and short["block_table"].tolist() == [[5, -1], [-1, -1]]
    assert short["slot_map"].tolist() == [-1] * 8 and short["total_lens"].tolist() == [3, 0]


def test_attention_over_dequantised_pools():
    """The 8-bit attention's reference is the fp64 oracle over bf16 pools that hold the same values."""
    g = torch.Generator().manual_seed(3)
    codes = torch.randint(0, 127, (3, 8, 2, 64), generator=g, dtype=torch.uint8).view(torch.float8_e4m3fn)
    scales = torch.randint(110, 122, (3, 2, 2), generator=g, dtype=torch.uint8)
    pool = kv8.dequant(codes, scales)
    want = codes.double() * torch.exp2(scales.double() - 127).repeat_interleave(4, 1)[..., None]
    assert torch.equal(pool.double(), want)
    q = torch.randn((1, 4, 64), generator=g).to(torch.bfloat16)
    table = torch.tensor([[2, 0, 1]], dtype=torch.int32)
    out = oracle.decode_paged(q, pool, pool, table, [21], 0.01)
    rows = want[[2, 0, 1]].reshape(24, 2, 64)[:21]
    for h in range(4):
        w = torch.softmax(q[0, h].double() @ rows[:, h // 2].T * 0.01, 0)
        assert np.allclose(out[0, h], (w @ rows[:, h // 2]).numpy(), atol=1e-12)
