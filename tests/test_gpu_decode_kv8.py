"""Decode over an 8-bit paged cache against the fp64 oracle on bf16 pools that hold the same values.

The tolerance is derived in kv8_inputs.attention_tolerance.  (The fp32-weight paths' rule has an absolute cap
of 2e-2 for outputs of order one; rows of an 8-bit pool reach 448 * 2^-4 here, and the rounding of a bf16 output between 8
and 16 alone is up to 2^-5 = 3.1e-2.)"""
import pytest
import torch

import asymmetric_head_kv_b200 as ak
import workloads as wl
from asymmetric_head_kv_b200 import _capi
from kv8_inputs import check_decode, pools, queries, stale, tables
from oracle import kv8
from workloads import Shape

pytestmark = pytest.mark.gpu

SHAPES = {
    "diffqkv": wl.DIFFQKV, "gqa": wl.GQA_CONTROL, "sigma": wl.SIGMA_1P5B_PAPER,
    "mha64": Shape(8, 8, 8, 64, 64), "mqa": Shape(16, 1, 1, 64, 64), "mqa128": Shape(16, 1, 16, 128, 128),
    "wide_k": Shape(16, 8, 2, 128, 64), "unaligned": Shape(24, 12, 8, 64, 128), "two": Shape(16, 2, 8, 64, 128),
    "two_v_wide": Shape(8, 2, 4, 128, 64),
}


def _run(p, q, table, lens, scale, dev, expect=0, **kw):
    gp = [t.to(dev) for t in p]
    B, n_q, d_k = q.shape
    dims = ak.make_dims(B, n_q, p[0].shape[2], p[1].shape[2], d_k, p[1].shape[3], scale)
    ws = ak.decode_workspace(dims, device=dev)
    out = ak.decode_paged_kv8(q.to(dev), *gp, table.to(dev), torch.as_tensor(lens, dtype=torch.int32).to(dev),
                              scale=scale, workspace=ws, **kw)
    assert ak.workspace_status(ws) == expect
    assert not ws[256:256 + 4 * B * p[0].shape[2]].any()
    return out


def _case(shape, lens, page, sb, dev, seed=0, spread=2, max_blocks=None, **kw):
    mb = max_blocks or max(1, max(-(-int(t) // page) for t in lens))
    num, table = tables(lens, page, mb, seed)
    p = pools(num, page, sb, shape, seed, spread)
    q = queries(len(lens), shape, seed + 1)
    out = _run([*stale(p[:2], table, lens, page), *p[2:]], q, table, lens, shape.scale, dev, **kw)
    check_decode(out, q, p, table, lens, shape.scale)


@pytest.mark.parametrize("name", SHAPES)
@pytest.mark.parametrize("lens", [[1], [127, 128, 129, 0, 1], [700, 1301]], ids=str)
def test_shapes_and_lengths(cuda_device, name, lens):
    _case(SHAPES[name], lens, 16, 16, cuda_device, seed=len(lens))


@pytest.mark.parametrize("page,sb", [(8, 8), (8, 1), (24, 8), (24, 3), (32, 4), (64, 64), (128, 32), (256, 256), (40, 40)])
def test_pages_and_scale_blocks(cuda_device, page, sb):
    _case(wl.DIFFQKV, [page * 3 + 5, 1, page, 333], page, sb, cuda_device, seed=page)


def test_many_short_and_one_long(cuda_device):
    lens = [int(x) for x in torch.randint(0, 200, (70,), generator=torch.Generator().manual_seed(0))] + [9000]
    _case(wl.DIFFQKV, lens, 16, 16, cuda_device, seed=2)


def test_long_context_in_many_splits(cuda_device):
    _case(Shape(4, 1, 4, 64, 128), [40001], 64, 16, cuda_device, seed=3)


@pytest.mark.parametrize("hint", [1, 50, 700])
def test_length_hint_never_changes_the_result(cuda_device, hint):
    _case(wl.DIFFQKV, [700, 300], 16, 16, cuda_device, max_seq_len=hint)


@pytest.mark.parametrize("spread", [6, 10])
def test_scales_far_apart(cuda_device, spread):
    """Scales over a factor of 2^12 and 2^20: scores of several thousand, weights on a handful of positions.  The
    queries are shrunk by 2^-spread, so that the scores stay of order one at the larger scales."""
    shape = wl.DIFFQKV
    lens = [900, 77]
    num, table = tables(lens, 16, 60, 4)
    p = pools(num, 16, 16, shape, 4, spread)
    q = (queries(2, shape, 5).float() * 2.0 ** -spread).to(torch.bfloat16)
    out = _run(p, q, table, lens, shape.scale, cuda_device)
    check_decode(out, q, p, table, lens, shape.scale, "scales far apart")


def test_growing_scores_rescale_the_output(cuda_device):
    """Each tile's scores exceed the last one's by more than the slack, then V's scales grow the same way."""
    shape = Shape(4, 1, 4, 64, 128)
    lens = [128 * 9 + 3]
    num, table = tables(lens, 16, 73, 0)
    p = pools(num, 16, 16, shape, 1, 0)
    order = table[0].long()
    for i in range(73):
        p[2][order[i]] = 118 + i // 16      # K scales double every other tile
        p[3][order[i]] = 110 + i // 8       # V scales every tile
    q = queries(1, shape, 2)
    out = _run(p, q, table, lens, shape.scale, cuda_device)
    check_decode(out, q, p, table, lens, shape.scale, "rescales")


@pytest.mark.parametrize("gain", [2.0 ** -60, 1e-3, 1e3, 2.0 ** 60])
def test_query_sizes(cuda_device, gain):
    shape = wl.DIFFQKV
    num, table = tables([500], 16, 32, 1)
    p = pools(num, 16, 16, shape, 1)
    q = (queries(1, shape, 3).float() * gain).to(torch.bfloat16)
    scale = 0.125 / gain
    out = _run(p, q, table, [500], scale, cuda_device)
    check_decode(out, q, p, table, [500], scale, f"gain {gain}")


def test_query_elements_far_apart(cuda_device):
    """Elements of a query over 2^-20 .. 1 of the largest: what the terms drop is below 2^-26 of the largest."""
    shape = wl.DIFFQKV
    num, table = tables([300], 16, 19, 1)
    p = pools(num, 16, 16, shape, 1)
    q = queries(1, shape, 3).float() * torch.exp2(-torch.arange(64).float() / 3)
    q = q.to(torch.bfloat16)
    out = _run(p, q, table, [300], 1.0, cuda_device)
    check_decode(out, q, p, table, [300], 1.0, "spread query")


def test_nan_in_a_held_row_reaches_its_heads_only(cuda_device):
    shape = wl.DIFFQKV
    num, table = tables([200], 16, 13, 1)
    p = pools(num, 16, 16, shape, 1)
    clean = _run(p, queries(1, shape, 1), table, [200], shape.scale, cuda_device)
    p[0].view(torch.uint8)[int(table[0, 3]), 2, 1, 5] = 0x7F     # K head 1: query heads 4..7
    p[1].view(torch.uint8)[int(table[0, 1]), 0, 9, 100] = 0xFF   # V head 9: query head 9, element 100
    out = _run(p, queries(1, shape, 1), table, [200], shape.scale, cuda_device)
    nan = torch.isnan(out[0].float()).cpu()
    want = torch.zeros((16, 128), dtype=torch.bool)
    want[4:8] = True
    want[9, 100] = True
    assert torch.equal(nan, want)
    assert torch.equal(out[0].cpu()[~want], clean[0].cpu()[~want])


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_a_query_that_is_not_finite_gives_nan(cuda_device, value):
    shape = wl.DIFFQKV
    num, table = tables([200], 16, 13, 1)
    p = pools(num, 16, 16, shape, 1)
    q = queries(1, shape, 1)
    q[0, 6, 9] = value
    out = _run(p, q, table, [200], shape.scale, cuda_device)
    nan = torch.isnan(out[0].float()).cpu()
    assert nan[6].all() and int(nan.sum()) == 128


def test_bad_entries_and_lengths_are_flagged(cuda_device):
    shape = wl.DIFFQKV
    num, table = tables([200, 40], 16, 13, 1)
    p = pools(num, 16, 16, shape, 1)
    q = queries(2, shape, 1)
    good = _run(p, q, table, [200, 40], shape.scale, cuda_device)
    bad = table.clone()
    bad[0, 5] = num
    out = _run(p, q, bad, [200, 40], shape.scale, cuda_device, expect=_capi.DEVICE_PAGE)
    assert torch.equal(out[1], good[1])
    out = _run(p, q, table, [200, -3], shape.scale, cuda_device, expect=_capi.DEVICE_SEQLEN)
    assert torch.equal(out[0], good[0]) and not out[1].any()
    full = torch.where(table < 0, torch.zeros_like(table), table)
    out = _run(p, q, full, [13 * 16 + 9, 40], shape.scale, cuda_device, expect=_capi.DEVICE_SEQLEN)
    assert torch.equal(out, _run(p, q, full, [13 * 16, 40], shape.scale, cuda_device))


def test_shared_pages_and_repeated_calls_are_bit_identical(cuda_device):
    shape = wl.DIFFQKV
    num, table = tables([900], 16, 57, 1)
    p = [t.to(cuda_device) for t in pools(num, 16, 16, shape, 1)]
    table = table.repeat(3, 1).to(cuda_device)
    q = queries(1, shape, 1).repeat(3, 1, 1).to(cuda_device)
    lens = torch.tensor([900, 900, 900], dtype=torch.int32, device=cuda_device)
    ws = ak.decode_workspace(ak.make_dims(3, 16, 4, 16, 64, 128, 1.0), device=cuda_device)
    a = ak.decode_paged_kv8(q, *p, table, lens, workspace=ws)
    for _ in range(3):
        assert torch.equal(ak.decode_paged_kv8(q, *p, table, lens, workspace=ws), a)


def test_streams_and_graphs(cuda_device):
    """Two streams with workspaces of their own, then a captured call replayed on new inputs."""
    dev, shape = cuda_device, wl.DIFFQKV
    lens = [800, 333]
    num, table = tables(lens, 16, 60, 1)
    p = [t.to(dev) for t in pools(num, 16, 16, shape, 1)]
    dims = ak.make_dims(2, 16, 4, 16, 64, 128, 1.0)
    td, ld = table.to(dev), torch.tensor(lens, dtype=torch.int32, device=dev)
    qs = [queries(2, shape, s).to(dev) for s in (1, 2)]
    wss = [ak.decode_workspace(dims, device=dev) for _ in range(2)]
    want = [ak.decode_paged_kv8(q, *p, td, ld, workspace=wss[0]).clone() for q in qs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = [torch.empty_like(want[0]) for _ in range(2)]
    for _ in range(20):
        for i in range(2):
            ak.decode_paged_kv8(qs[i], *p, td, ld, workspace=wss[i], out=outs[i], stream=streams[i])
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])
    g = torch.cuda.CUDAGraph()
    q = qs[0].clone()
    with torch.cuda.graph(g):
        ak.decode_paged_kv8(q, *p, td, ld, workspace=wss[0], out=outs[0])
    q.copy_(qs[1])
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[1])


def test_cache_past_32_bit_offsets(cuda_device):
    """A sequence whose pages lie behind 2^31 bytes of both pools equals the same rows in a small pool."""
    dev, shape, page = cuda_device, wl.DIFFQKV, 64
    lens = [500]
    num, table = tables(lens, page, 8, 1, spare=0)
    small = [t.to(dev) for t in pools(num, page, 16, shape, 1)]
    big_n = 2 ** 31 // (page * 4 * 64) + 20
    big = ak.kv8_pools(big_n, page, 4, 16, 64, 128, scale_block=16, device=dev)
    off = big_n - num
    for b, s in zip(big, small):
        b.view(torch.uint8)[off:] = s.view(torch.uint8)
    q, ld = queries(1, shape, 2).to(dev), torch.tensor(lens, dtype=torch.int32, device=dev)
    a = ak.decode_paged_kv8(q, *small, table.to(dev), ld)
    assert torch.equal(ak.decode_paged_kv8(q, *big, (table + off).to(dev), ld), a)


def test_steps_of_a_generation(cuda_device):
    """page_map, kv8_store and decode_paged_kv8 over several steps, as a server runs them, against the oracle on
    the pools the definition writes."""
    dev, shape, page, B = cuda_device, wl.DIFFQKV, 16, 3
    num, mb = 40, 12
    gpu = ak.kv8_pools(num, page, 4, 16, 64, 128, device=dev)
    host = [(p.cpu().view(torch.uint8).numpy(), s.cpu().numpy()) for p, s in ((gpu[0], gpu[2]), (gpu[1], gpu[3]))]
    table = torch.full((B, mb), -1, dtype=torch.int32, device=dev)
    lens = torch.zeros(B, dtype=torch.int32, device=dev)
    free = list(range(num))[::-1]
    g = torch.Generator().manual_seed(0)
    ws = ak.decode_workspace(ak.make_dims(B, 16, 4, 16, 64, 128, 1.0), device=dev)
    for step, new in enumerate([[50, 1, 100], [1, 1, 1], [1, 1, 1], [1, 20, 0], [1, 1, 1]]):
        T = sum(new) + step
        _, slots, _, total, used = ak.page_map(lens, torch.tensor(new, dtype=torch.int32, device=dev), table,
                                               torch.tensor(free, dtype=torch.int32, device=dev), page, num, capacity=T)
        free = free[int(used):]
        k = torch.randn((T, 4, 64), generator=g).mul_(1.5 ** step).to(torch.bfloat16)
        v = torch.randn((T, 16, 128), generator=g).mul_(1.5 ** step).to(torch.bfloat16)
        ak.kv8_store(k.to(dev), v.to(dev), slots, *gpu)
        for x, (codes, scales) in zip((k, v), host):
            kv8.store(codes, scales, x.double().numpy(), slots.cpu().tolist())
        lens = total
        q = queries(B, shape, step)
        out = ak.decode_paged_kv8(q.to(dev), *gpu, table, lens, workspace=ws)
        assert ak.workspace_status(ws) == 0 and ak.device_status() == 0
        pool = [torch.from_numpy(c).view(torch.float8_e4m3fn) for c, _ in host] + [torch.from_numpy(s) for _, s in host]
        check_decode(out, q, pool, table.cpu(), lens.cpu(), 0.125, f"step {step}")


def test_refusals(cuda_device):
    dev, shape = cuda_device, wl.DIFFQKV
    num, table = tables([40], 16, 3, 1)
    p = [t.to(dev) for t in pools(num, 16, 16, shape, 1)]
    q, ld, td = queries(1, shape, 1).to(dev), torch.tensor([40], dtype=torch.int32, device=dev), table.to(dev)
    with pytest.raises(TypeError):
        ak.decode_paged_kv8(q.float(), *p, td, ld)
    with pytest.raises(ValueError):
        ak.decode_paged_kv8(q[:, :, :32], *p, td, ld)
    with pytest.raises(ValueError):
        ak.decode_paged_kv8(q, *p, td, ld[:0])
    with pytest.raises(ak.DiffqkvError) as e:
        ak.decode_paged_kv8(q[:, :12].contiguous(), *p, td, ld)
    assert e.value.status == _capi.INVALID_ARG       # 12 query heads over 16 V heads
    with pytest.raises(ak.DiffqkvError) as e:
        ak.decode_paged_kv8(q, *p, td, ld, workspace=torch.zeros(256, dtype=torch.uint8, device=dev))
    assert e.value.status == _capi.WORKSPACE
    with pytest.raises(ak.DiffqkvError) as e:
        ak.decode_paged_kv8(q, *p, td, ld, scale=0.0)
    assert e.value.status == _capi.INVALID_ARG
