"""Block tables and slot maps built on the GPU, against the plain definition (whole numbers: equal)."""
import pytest
import torch

import asymmetric_head_kv_b200 as ak
from asymmetric_head_kv_b200 import _capi
from oracle import kv8

pytestmark = pytest.mark.gpu


def _i32(x, dev):
    return torch.as_tensor(x, dtype=torch.int32).to(dev)


def _check(s, n, table, free, page, num_pages, capacity, dev, expect=0):
    want = kv8.page_map(s, n, table, free, page, num_pages, capacity)
    bt = _i32(table, dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    got = ak.page_map(_i32(s, dev), _i32(n, dev), bt, _i32(free, dev), page, num_pages, capacity=capacity, status=status)
    assert status.item() == expect == want["status"]
    for name, t in zip(("query_start", "slot_map", "positions", "total_lens", "pages_used"), got):
        assert t.cpu().tolist() == want[name].tolist(), name
    assert bt.cpu().tolist() == want["block_table"].tolist()


def _step(batch, hi, new_hi, page, seed, spare=3):
    g = torch.Generator().manual_seed(seed)
    s = torch.randint(0, hi + 1, (batch,), generator=g)
    n = torch.randint(0, new_hi + 1, (batch,), generator=g)
    held, need = -(-s // page), -(-(s + n) // page)
    num_pages = int(need.sum()) + spare
    perm = torch.randperm(num_pages, generator=g).tolist()
    mb = max(1, -(-(hi + new_hi) // page))
    table = [[-1] * mb for _ in range(batch)]
    at = 0
    for b in range(batch):
        for i in range(int(held[b])):
            table[b][i] = perm[at]
            at += 1
    return s.tolist(), n.tolist(), table, perm[at:], num_pages


@pytest.mark.parametrize("batch,hi,new_hi,page", [
    (1, 0, 1, 16), (1, 100, 1, 16), (1, 0, 5000, 8), (3, 33, 7, 1), (17, 500, 40, 24), (511, 60, 9, 16), (512, 60, 9, 16),
    (513, 60, 9, 16), (1500, 300, 30, 32), (2, 7, 0, 16),
    (256, 90, 300, 16), (257, 90, 300, 16), (1023, 40, 90, 8), (1024, 40, 90, 24), (1025, 40, 90, 8),
])
def test_against_the_definition(cuda_device, batch, hi, new_hi, page):
    s, n, table, free, num_pages = _step(batch, hi, new_hi, page, batch * 7 + page)
    for extra in (0, 1, 2, 3, 777):
        _check(s, n, table, free, page, num_pages, sum(n) + extra, cuda_device)


@pytest.mark.parametrize("batch,hi,new_hi,page", [(7, 100, 60000, 16), (300, 90, 1500, 24), (1500, 300, 300, 32)])
def test_large_buffers(cuda_device, batch, hi, new_hi, page):
    """Buffers beyond the size up to which a thread maps one token: four, with ends of every remainder."""
    s, n, table, free, num_pages = _step(batch, hi, new_hi, page, batch)
    for capacity in (sum(n) + 230000, sum(n) + 230001, sum(n) + 230003):
        _check(s, n, table, free, page, num_pages, capacity, cuda_device)


def test_many_requests_with_long_stretches_of_empty_ones(cuda_device):
    batch, page = 5000, 16
    n = [0] * batch
    n[0], n[2500], n[4999] = 1, 70, 33
    s = [0] * batch
    s[2500] = 15
    table = [[-1] * 8 for _ in range(batch)]
    table[2500][0] = 11
    _check(s, n, table, [1, 2, 3, 4, 5, 6, 7, 8, 9, 10], page, 20, 120, cuda_device)


@pytest.mark.parametrize("what", ["buffer", "pages", "negative", "too_long", "bad_held", "bad_free"])
def test_what_does_not_fit_is_flagged(cuda_device, what):
    s, n, table, free, num_pages = _step(9, 90, 20, 16, 5)
    s[4], n[4] = 13, 9   # a request that writes into a held page and takes one
    held = -(-13 // 16)
    table[4] = [num_pages - 1] * held + [-1] * (len(table[4]) - held)
    free = free + [0, 1, 2]
    cap, expect = sum(n) + 5, _capi.DEVICE_PAGE
    if what == "buffer":
        cap, expect = sum(n) - 1, _capi.DEVICE_SEQLEN
    elif what == "pages":
        free = free[:1]
    elif what == "negative":
        s[2], expect = -4, _capi.DEVICE_SEQLEN
    elif what == "too_long":
        n[7], expect = 10 ** 9, _capi.DEVICE_SEQLEN
    elif what == "bad_held":
        table[4][0] = num_pages
    else:
        free[0] = -7
    _check(s, n, table, free, 16, num_pages, max(cap, 0), cuda_device, expect)


def test_a_dropped_step_leaves_the_table(cuda_device):
    dev = cuda_device
    bt = torch.full((2, 4), -5, dtype=torch.int32, device=dev)
    bt[0, 0] = 1
    keep = bt.clone()
    qs, slots, pos, total, used = ak.page_map(_i32([3, 0], dev), _i32([30, 5], dev), bt, _i32([2], dev), 16, 8,
                                              capacity=64, status=torch.zeros(1, dtype=torch.int32, device=dev))
    assert torch.equal(bt, keep) and used.item() == 0 and total.tolist() == [3, 0] and qs.tolist() == [0, 0, 0]
    assert (slots == -1).all() and (pos == -1).all()


def test_captured_and_replayed_on_its_own_stream(cuda_device):
    dev = cuda_device
    s, n, table, free, num_pages = _step(40, 200, 30, 16, 9)
    seq, new, bt, fr = (_i32(v, dev) for v in (s, n, table, free))
    outs = [torch.empty(k, dtype=torch.int32, device=dev) for k in (41, sum(n), sum(n), 40, 1)]
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        ak.page_map(seq, new, bt, fr, 16, num_pages, *outs, status=status)
    for lens in (s, list(reversed(s))):
        held = [-(-v // 16) for v in lens]
        t2 = [[0] * h + [-1] * (len(table[0]) - h) for h in held]
        want = kv8.page_map(lens, n, t2, free + list(range(num_pages)), 16, num_pages, sum(n))
        if int(want["pages_used"][0]) > len(free):
            continue
        seq.copy_(_i32(lens, dev))
        bt.copy_(_i32(t2, dev))
        g.replay()
        torch.cuda.synchronize()
        assert outs[1].tolist() == want["slot_map"].tolist() and bt.tolist() == want["block_table"].tolist()


def test_refusals(cuda_device):
    dev = cuda_device
    a = dict(seq_lens=_i32([1], dev), new_lens=_i32([1], dev), block_table=_i32([[0, -1]], dev), free_pages=_i32([1], dev),
             page_size=16, num_pages=4, capacity=4)
    with pytest.raises(TypeError):
        ak.page_map(**{**a, "seq_lens": a["seq_lens"].long()})
    with pytest.raises(ValueError):
        ak.page_map(**{**a, "new_lens": _i32([1, 2], dev)})
    with pytest.raises(ValueError):
        ak.page_map(**{**a, "block_table": _i32([0], dev)})
    with pytest.raises(ValueError):
        ak.page_map(**{**a, "capacity": None})
    with pytest.raises(ValueError):
        ak.page_map(**{**a, "free_pages": torch.tensor([1], dtype=torch.int32)})
    with pytest.raises(ak.DiffqkvError) as e:
        ak.page_map(**{**a, "page_size": 0})
    assert e.value.status == _capi.INVALID_ARG
    with pytest.raises(ak.DiffqkvError) as e:
        ak.page_map(**{**a, "capacity": None}, slot_map=torch.empty(9, dtype=torch.int32, device=dev)[1:])
    assert e.value.status == _capi.MISALIGNED
