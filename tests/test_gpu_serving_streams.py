"""What the serving calls allocate themselves belongs to the stream they run on: a call on a side stream neither waits
for, nor races with, the current stream's work on the same allocator pool."""
import pytest
import torch

import asymmetric_head_kv_b200 as ak
from asymmetric_head_kv_b200 import _capi
from kv8_inputs import pools, queries, tables
from workloads import Shape

pytestmark = pytest.mark.gpu


def _behind_other_work(call, side, dev):
    """Runs call(side) while the current stream holds freed, non-zero memory and is busy."""
    dirty = [torch.full((n,), 0x5A, dtype=torch.uint8, device=dev) for n in (1 << 16, 1 << 20, 1 << 23, 1 << 25)]
    torch.cuda._sleep(40_000_000)  # some 20 ms
    del dirty
    out = call(side)
    side.synchronize()
    out = [t.clone() for t in out]
    torch.cuda.synchronize()
    return out


def test_buffers_of_a_call_belong_to_its_stream(cuda_device):
    dev, shape, lens = cuda_device, Shape(4, 1, 4, 64, 128), [4000, 900]
    num, table = tables(lens, 16, 250, 1)
    p = [t.to(dev) for t in pools(num, 16, 16, shape, 1)]
    td, ld = table.to(dev), torch.tensor(lens, dtype=torch.int32, device=dev)
    q, rows = queries(2, shape, 1).to(dev), queries(40, shape, 2).to(dev)
    start = torch.tensor([0, 33, 40], dtype=torch.int32, device=dev)
    free = torch.arange(num, dtype=torch.int32, device=dev)
    ones = torch.ones_like(ld)
    word = torch.zeros(1, dtype=torch.int32, device=dev)  # (request 0 is at its table's end: flagged, adds nothing)

    def decode(s):
        return [ak.decode_paged_kv8(q, *p, td, ld, stream=s)]

    def prefill(s):
        return [ak.prefill_paged_kv8(rows, start, *p, td, ld, stream=s)]

    def mapping(s):
        return list(ak.page_map(ld, ones, td.clone() if s is None else spare, free, 16, num, capacity=7, status=word,
                                stream=s))

    side = torch.cuda.Stream(device=dev)
    for call in (decode, prefill, mapping):
        want = [t.clone() for t in call(None)]
        spare = td.clone()
        torch.cuda.synchronize()
        call(side)  # (its memory is there: the call below is not held up by an allocation)
        spare = td.clone()
        torch.cuda.synchronize()
        got = _behind_other_work(call, side, dev)
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    assert word.item() == _capi.DEVICE_SEQLEN and ak.device_status() == 0
