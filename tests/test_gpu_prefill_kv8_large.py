"""Prefill over 8-bit pools beyond 2^31 bytes."""
import pytest
import torch

import asymmetric_head_kv_b200 as ak
import workloads as wl
from kv8_inputs import check_prefill, pools, queries, tables

pytestmark = pytest.mark.gpu


def test_cache_past_32_bit_offsets(cuda_device):
    """Sequences whose pages lie behind 2^31 bytes of both pools, and behind 2^32 of V's, equal the same rows in small
    pools: whole units, and units cut into pieces."""
    dev, shape, page = cuda_device, wl.DIFFQKV, 64
    lens, rows = [500, 3000], [300, 5]
    num, table = tables(lens, page, 47, 1, spare=0)
    host = pools(num, page, 16, shape, 1)
    small = [t.to(dev) for t in host]
    big_n = 2 ** 31 // (page * 4 * 64) + num + 20
    big = ak.kv8_pools(big_n, page, 4, 16, 64, 128, scale_block=16, device=dev)
    off = big_n - num
    for b, s in zip(big, small):
        b.view(torch.uint8)[off:] = s.view(torch.uint8)
    assert off * page * 4 * 64 >= 2 ** 31 and off * page * 16 * 128 >= 2 ** 32
    for pick in ([0], [1], [0, 1]):
        n, r = [lens[i] for i in pick], [rows[i] for i in pick]
        start = [sum(r[:i]) for i in range(len(r) + 1)]
        q = queries(start[-1], shape, 2)
        i32 = lambda x: torch.as_tensor(x, dtype=torch.int32).to(dev)  # noqa: E731
        args = q.to(dev), i32(start)
        out = ak.prefill_paged_kv8(*args, *small, i32(table[pick]), i32(n), scale=shape.scale)
        check_prefill(out, q, start, host, table[pick], n, shape.scale)
        far = torch.where(table[pick] >= 0, table[pick] + off, -1)
        assert torch.equal(ak.prefill_paged_kv8(*args, *big, i32(far), i32(n), scale=shape.scale), out)
