"""One workspace, zero-filled once, for calls of any shape and of every operator that shares its layout (header, 2048
counters, records): each equals, bit for bit, the same call on a fresh workspace."""
import pytest
import torch

import asymmetric_head_kv_b200 as ak
import oracle
import workloads as wl
from kv8_inputs import check_decode, check_prefill, pools, queries, tables
from parity import assert_parity
from workloads import Shape

pytestmark = pytest.mark.gpu

HEAD = 256 + 4 * 2048  # bytes that a call which completes leaves zero


def _decode_kv8(dev, shape, lens, seed):
    num, table = tables(lens, 16, -(-max(lens) // 16), seed)
    p = [t.to(dev) for t in pools(num, 16, 16, shape, seed)]
    q, td, ld = queries(len(lens), shape, seed).to(dev), table.to(dev), torch.tensor(lens, dtype=torch.int32, device=dev)

    def call(ws, out):
        return ak.decode_paged_kv8(q, *p, td, ld, scale=shape.scale, workspace=ws, out=out)
    return call, (len(lens), shape.n_q, shape.d_v)


def _prefill_kv8(dev, shape, rows, lens, seed):
    num, table = tables(lens, 16, -(-max(lens) // 16), seed)
    p = [t.to(dev) for t in pools(num, 16, 16, shape, seed)]
    td, ld = table.to(dev), torch.tensor(lens, dtype=torch.int32, device=dev)
    start = torch.tensor([sum(rows[:i]) for i in range(len(rows) + 1)], dtype=torch.int32, device=dev)
    q = queries(sum(rows), shape, seed).to(dev)

    def call(ws, out):
        return ak.prefill_paged_kv8(q, start, *p, td, ld, scale=shape.scale, workspace=ws, out=out)
    return call, (sum(rows), shape.n_q, shape.d_v)


def _decode(dev, shape, lens, seed):
    d = wl.random_decode_inputs(len(lens), max(lens), shape, seed=seed, seq_lens=lens)
    q, k, v, ld = (d[n].to(dev) for n in ("q", "k_cache", "v_cache", "seq_lens"))

    def call(ws, out):
        return ak.decode(q, k, v, ld, scale=d["scale"], workspace=ws, out=out)
    return call, (len(lens), shape.n_q, shape.d_v)


def _calls(dev, kind):
    sigma = wl.DIFFQKV
    long_one, many, few = [20000], [1000 - i for i in range(64)], [5000, 700, 3]
    if kind == "decode_kv8":
        return [_decode_kv8(dev, sigma, n, i) for i, n in enumerate((long_one, many, few, many))]
    if kind == "decode":
        return [_decode(dev, sigma, n, i) for i, n in enumerate((long_one, many, few, many))]
    cut = Shape(4, 1, 4, 64, 128)
    return [_decode_kv8(dev, sigma, long_one, 0), _prefill_kv8(dev, cut, [40, 3], [4000, 900], 1),
            _decode(dev, sigma, many, 2), _prefill_kv8(dev, Shape(2, 2, 1, 128, 64), [300], [5000], 3),
            _decode_kv8(dev, sigma, many, 4), _decode(dev, wl.GQA_CONTROL, few, 5),
            _decode_kv8(dev, Shape(16, 16, 16, 128, 128), many, 6), _prefill_kv8(dev, cut, [40, 3], [4000, 900], 1)]


@pytest.mark.parametrize("kind", ["decode_kv8", "decode", "mixed"])
def test_one_workspace_for_every_call(cuda_device, kind):
    dev = cuda_device
    one = torch.zeros(64 << 20, dtype=torch.uint8, device=dev)
    for i, (call, shape) in enumerate(_calls(dev, kind)):
        outs = []
        for ws in (one, torch.zeros(64 << 20, dtype=torch.uint8, device=dev)):
            out = torch.full(shape, float("nan"), dtype=torch.bfloat16, device=dev)
            call(ws, out)
            assert ak.workspace_status(ws) == 0
            outs.append(out)
        assert not torch.isnan(outs[1]).any()
        assert torch.equal(outs[0], outs[1]), f"call {i}"
    assert not one[:HEAD].any()


def _many_lens(n):
    return torch.randint(0, 400, (n,), generator=torch.Generator().manual_seed(3)).tolist()


def test_more_units_than_counters_kv8(cuda_device):
    """Beyond 2048 (sequence, K head)s a split unit counts its pieces in the counter of its first CTA."""
    dev, shape, lens = cuda_device, Shape(8, 4, 8, 64, 64), _many_lens(600)
    num, table = tables(lens, 16, 25, 1)
    p = pools(num, 16, 16, shape, 1)
    q = queries(len(lens), shape, 2)
    ws = ak.decode_workspace(ak.make_dims(600, 8, 4, 8, 64, 64, shape.scale), device=dev)
    ld = torch.tensor(lens, dtype=torch.int32, device=dev)
    outs = [ak.decode_paged_kv8(q.to(dev), *[t.to(dev) for t in p], table.to(dev), ld, scale=shape.scale, workspace=ws)
            for _ in range(2)]
    assert ak.workspace_status(ws) == 0 and not ws[:HEAD].any() and torch.equal(outs[0], outs[1])
    check_decode(outs[0], q, p, table, lens, shape.scale)


@pytest.mark.parametrize("grid", [0, 2048])
def test_more_units_than_counters(cuda_device, grid):
    dev, lens = cuda_device, _many_lens(600)
    d = wl.random_decode_inputs(600, 400, Shape(8, 4, 8, 64, 64), seed=4, seq_lens=lens)
    ws = ak.decode_workspace(d["q"], d["k_cache"], d["v_cache"], device=dev)
    tuning = {"grid_ctas": grid, "stages": 0, "ctas_per_sm": 0} if grid else None
    for _ in range(2):
        out = ak.decode(d["q"].to(dev), d["k_cache"].to(dev), d["v_cache"].to(dev), d["seq_lens"].to(dev),
                        scale=d["scale"], workspace=ws, tuning=tuning)
        assert ak.workspace_status(ws) == 0 and not ws[:HEAD].any()
        assert_parity(out, oracle.decode(d["q"], d["k_cache"], d["v_cache"], d["seq_lens"], d["scale"]), f"grid {grid}")


def test_prefill_after_a_decode_of_the_same_cache(cuda_device):
    """The two calls of a server's step share a workspace and still match the definition."""
    dev, shape, lens = cuda_device, Shape(4, 1, 4, 64, 128), [4000, 900]
    num, table = tables(lens, 16, 250, 1)
    p = pools(num, 16, 16, shape, 1)
    gp, td, ld = [t.to(dev) for t in p], table.to(dev), torch.tensor(lens, dtype=torch.int32, device=dev)
    q, rows, start = queries(2, shape, 1), queries(40, shape, 2), torch.tensor([0, 33, 40], dtype=torch.int32, device=dev)
    dims = ak.make_dims(2, 4, 1, 4, 64, 128, shape.scale)
    ws = max((ak.decode_workspace(dims, device=dev), ak.prefill_paged_kv8_workspace(dims, dev)), key=torch.Tensor.numel)
    for _ in range(2):
        out = ak.decode_paged_kv8(q.to(dev), *gp, td, ld, scale=shape.scale, workspace=ws)
        check_decode(out, q, p, table, lens, shape.scale)
        out = ak.prefill_paged_kv8(rows.to(dev), start, *gp, td, ld, scale=shape.scale, workspace=ws)
        check_prefill(out, rows, [0, 33, 40], p, table, lens, shape.scale)
    assert ak.workspace_status(ws) == 0
