"""Ragged causal prefill over an 8-bit paged cache against the fp64 formula; tolerance derived in
kv8_inputs.check_prefill."""
import pytest
import torch

import asymmetric_head_kv_b200 as ak
import workloads as wl
from asymmetric_head_kv_b200 import _capi
from kv8_inputs import check_prefill, pools, queries, stale, tables
from workloads import Shape

pytestmark = pytest.mark.gpu

SHAPES = {
    "diffqkv": wl.DIFFQKV, "gqa": wl.GQA_CONTROL, "sigma": wl.SIGMA_1P5B_PAPER, "mha64": Shape(8, 8, 8, 64, 64),
    "mqa": Shape(16, 1, 1, 64, 64), "wide_k": Shape(16, 8, 2, 128, 64), "unaligned": Shape(24, 12, 8, 64, 128),
    "three": Shape(6, 2, 3, 128, 128),
}


def _run(p, q, start, table, lens, scale, dev, expect=0, out=None, **kw):
    n_q, d_k = q.shape[1:]
    dims = ak.make_dims(len(lens), n_q, p[0].shape[2], p[1].shape[2], d_k, p[1].shape[3], scale)
    ws = ak.prefill_paged_kv8_workspace(dims, dev)
    i32 = lambda x: torch.as_tensor(x, dtype=torch.int32).to(dev)  # noqa: E731
    out = ak.prefill_paged_kv8(q.to(dev), i32(start), *[t.to(dev) for t in p], table.to(dev), i32(lens), scale=scale,
                               workspace=ws, out=out, **kw)
    assert ak.workspace_status(ws) == expect
    assert not ws[:256 + 640].any()
    return out


def _starts(rows):
    s = [0]
    for n in rows:
        s.append(s[-1] + n)
    return s


def _case(shape, rows, lens, page, sb, dev, seed=0, spread=2, q_gain=1.0, **kw):
    num, table = tables(lens, page, max(1, max(-(-int(t) // page) for t in lens)), seed)
    p = pools(num, page, sb, shape, seed, spread)
    start = _starts(rows)
    q = (queries(start[-1], shape, seed + 1).float() * q_gain).to(torch.bfloat16)
    out = _run([*stale(p[:2], table, lens, page), *p[2:]], q, start, table, lens, shape.scale, dev, **kw)
    check_prefill(out, q, start, p, table, lens, shape.scale)
    return out


@pytest.mark.parametrize("name", SHAPES)
@pytest.mark.parametrize("rows,lens", [([1], [1]), ([300, 1, 0, 129], [300, 64, 5, 200]), ([17], [700])], ids=str)
def test_shapes(cuda_device, name, rows, lens):
    _case(SHAPES[name], rows, lens, 16, 16, cuda_device, seed=len(rows))


@pytest.mark.parametrize("rows", [1, 63, 64, 65, 127, 128, 129, 255, 256, 257, 513])
@pytest.mark.parametrize("prefix", [0, 1, 191])
def test_row_counts_and_prefixes(cuda_device, rows, prefix):
    _case(Shape(2, 1, 2, 64, 128), [rows], [rows + prefix], 16, 16, cuda_device, seed=rows)


@pytest.mark.parametrize("page,sb", [(8, 8), (8, 1), (24, 8), (24, 3), (32, 4), (64, 64), (128, 32), (256, 256), (40, 40)])
def test_pages_and_scale_blocks(cuda_device, page, sb):
    _case(Shape(4, 2, 4, 64, 128), [page + 3, 90], [page * 3 + 5, 333], page, sb, cuda_device, seed=page)


def test_many_requests(cuda_device):
    g = torch.Generator().manual_seed(0)
    rows = torch.randint(0, 40, (70,), generator=g).tolist()
    lens = [r + int(x) for r, x in zip(rows, torch.randint(0, 100, (70,), generator=g))]
    _case(Shape(4, 1, 4, 64, 64), rows, lens, 16, 16, cuda_device, seed=5)


@pytest.mark.parametrize("rows,length", [(1, 5000), (5, 9001), (130, 3000), (200, 2112)])
def test_few_rows_over_a_long_context_are_split(cuda_device, rows, length):
    _case(Shape(4, 1, 4, 64, 128), [rows], [length], 64, 16, cuda_device, seed=rows)
    _case(Shape(2, 2, 1, 128, 128), [rows], [length // 2], 64, 64, cuda_device, seed=rows + 1)


@pytest.mark.parametrize("rows,lens", [([256, 5, 0, 130], [4100, 7000, 64, 131]), ([600], [600]), ([600], [5000]),
                                       ([1] * 32, [65 + 40 * i for i in range(32)]),
                                       ([1] * 33, [65 + 40 * i for i in range(33)]), ([0, 3], [0, 2000])], ids=str)
def test_ragged_batches_are_cut(cuda_device, rows, lens):
    """Few heads, so that units are cut into many pieces: blocks with fewer tiles than pieces, requests of very different
    lengths, empty ones."""
    _case(Shape(4, 1, 4, 64, 128), rows, lens, 16, 16, cuda_device)


@pytest.mark.parametrize("spread", [6, 10])
def test_scales_far_apart(cuda_device, spread):
    _case(wl.DIFFQKV, [90], [900], 16, 16, cuda_device, seed=4, spread=spread, q_gain=2.0 ** -spread)


def test_zero_rows_with_the_smallest_scale(cuda_device):
    """Blocks of zeros at the least exponent among ordinary ones, for K and for V."""
    shape = Shape(4, 2, 4, 64, 128)
    lens = [400]
    num, table = tables(lens, 16, 25, 3)
    p = pools(num, 16, 16, shape, 3)
    for i in range(2, 25, 3):
        pg = int(table[0, i])
        for c, s in ((p[0], p[2]), (p[1], p[3])):
            c.view(torch.uint8)[pg] = 0
            s[pg] = 7
    q = queries(100, shape, 1)
    out = _run(p, q, [0, 100], table, lens, shape.scale, cuda_device)
    check_prefill(out, q, [0, 100], p, table, lens, shape.scale)


def test_growing_scores_and_scales_rescale_the_output(cuda_device):
    shape = Shape(4, 1, 4, 64, 128)
    lens = [64 * 19 + 3]
    num, table = tables(lens, 16, 77, 0)
    p = pools(num, 16, 16, shape, 1, 0)
    for i in range(77):
        p[2][table[0, i].long()] = 118 + i // 16
        p[3][table[0, i].long()] = 110 + i // 8
    q = queries(200, shape, 2)
    out = _run(p, q, [0, 200], table, lens, shape.scale, cuda_device)
    check_prefill(out, q, [0, 200], p, table, lens, shape.scale)


@pytest.mark.parametrize("gain", [2.0 ** -60, 1e-3, 1e3, 2.0 ** 60])
def test_query_sizes(cuda_device, gain):
    shape = wl.DIFFQKV
    num, table = tables([300], 16, 19, 1)
    p = pools(num, 16, 16, shape, 1)
    q = (queries(150, shape, 3).float() * gain).to(torch.bfloat16)
    out = _run(p, q, [0, 150], table, [300], 0.125 / gain, cuda_device)
    check_prefill(out, q, [0, 150], p, table, [300], 0.125 / gain)


def test_rows_of_zeros_and_tiny_scales(cuda_device):
    """A zero query weights its positions alike, whatever the scale's exponent."""
    shape = Shape(2, 1, 2, 64, 64)
    num, table = tables([130], 16, 9, 1)
    p = pools(num, 16, 16, shape, 1)
    p[2][:] = 7
    q = torch.zeros((130, 2, 64), dtype=torch.bfloat16)
    out = _run(p, q, [0, 130], table, [130], 1.0, cuda_device)
    check_prefill(out, q, [0, 130], p, table, [130], 1.0)


def test_decode_rows_agree_with_decode(cuda_device):
    """One row per request is a decode step: both calls on the same cache, within their tolerances."""
    dev, shape = cuda_device, wl.DIFFQKV
    lens = [700, 64, 1, 333]
    num, table = tables(lens, 16, 44, 1)
    p = pools(num, 16, 16, shape, 1)
    q = queries(4, shape, 2)
    out = _run(p, q, [0, 1, 2, 3, 4], table, lens, shape.scale, dev)
    check_prefill(out, q, [0, 1, 2, 3, 4], p, table, lens, shape.scale)
    ld = torch.tensor(lens, dtype=torch.int32, device=dev)
    dec = ak.decode_paged_kv8(q.to(dev), *[t.to(dev) for t in p], table.to(dev), ld, scale=shape.scale)
    assert (out.double() - dec.double()).norm() <= 2 ** -7 * dec.double().norm()


def test_rows_behind_the_last_request_are_left_alone(cuda_device):
    dev, shape = cuda_device, Shape(4, 2, 4, 64, 128)
    lens = [90, 40]
    num, table = tables(lens, 16, 6, 1)
    p = pools(num, 16, 16, shape, 1)
    q = queries(140, shape, 2)
    out = torch.full((140, 4, 128), 7.0, dtype=torch.bfloat16, device=dev)
    _run(p, q, [0, 90, 110], table, lens, shape.scale, dev, out=out)
    assert (out[110:] == 7).all()
    check_prefill(out[:110], q[:110], [0, 90, 110], p, table, lens, shape.scale)


def test_nan_in_later_positions_stays_out_of_earlier_rows(cuda_device):
    """A NaN key is masked from the rows before it; a NaN value may reach the 255 rows before it and no others."""
    shape = Shape(2, 1, 2, 64, 128)
    num, table = tables([700], 16, 44, 1)
    p = pools(num, 16, 16, shape, 1)
    q = queries(700, shape, 2)
    clean = _run(p, q, [0, 700], table, [700], shape.scale, cuda_device)
    p[0].view(torch.uint8)[int(table[0, 500 // 16]), 500 % 16, 0, 9] = 0x7F
    out = _run(p, q, [0, 700], table, [700], shape.scale, cuda_device)
    assert torch.equal(out[:500], clean[:500]) and torch.isnan(out[500:]).all()
    p[0].view(torch.uint8)[int(table[0, 500 // 16]), 500 % 16, 0, 9] = 0
    p[1].view(torch.uint8)[int(table[0, 300 // 16]), 300 % 16, 1, 5] = 0x7F
    out = _run(p, q, [0, 700], table, [700], shape.scale, cuda_device)
    nan = torch.isnan(out)
    assert nan[300:, 1, 5].all() and not nan[:300 - 255].any()
    nan[:, 1, 5] = False
    assert not nan.any()


def test_bad_inputs_are_flagged_and_clamped(cuda_device):
    dev, shape = cuda_device, Shape(4, 2, 4, 64, 128)
    lens = [90, 40]
    num, table = tables(lens, 16, 6, 1)
    p = pools(num, 16, 16, shape, 1)
    q = queries(60, shape, 2)
    good = _run(p, q, [0, 30, 60], table, lens, shape.scale, dev)
    bad = table.clone()
    bad[0, 2] = -1
    out = _run(p, q, [0, 30, 60], bad, lens, shape.scale, dev, expect=_capi.DEVICE_PAGE)
    assert torch.equal(out[30:], good[30:])
    out = _run(p, q, [0, 30, 90], table, lens, shape.scale, dev, expect=_capi.DEVICE_SEQLEN)   # past the rows of q
    assert torch.equal(out, good)
    zeros = torch.zeros_like(good)
    out = _run(p, q, [0, 30, 60], table, [90, 12], shape.scale, dev, expect=_capi.DEVICE_SEQLEN, out=zeros.clone())
    assert torch.equal(out[:30], good[:30]) and not out[30:48].any() and torch.isfinite(out.float()).all()
    out = _run(p, q, [0, 30, 60], table, [90, -5], shape.scale, dev, expect=_capi.DEVICE_SEQLEN, out=zeros.clone())
    assert not out[30:].any()
    out = _run(p, q, [0, 30, 20], table, lens, shape.scale, dev, expect=_capi.DEVICE_SEQLEN, out=zeros.clone())
    assert torch.equal(out[:30], good[:30]) and not out[30:].any()


def test_streams_graphs_and_repeats(cuda_device):
    dev, shape = cuda_device, wl.DIFFQKV
    for rows, lens in (([400, 70], [600, 900]), ([3], [4000])):
        start = _starts(rows)
        num, table = tables(lens, 16, 260, 1)
        p = [t.to(dev) for t in pools(num, 16, 16, shape, 1)]
        td, ld, sd = table.to(dev), torch.tensor(lens, dtype=torch.int32, device=dev), \
            torch.tensor(start, dtype=torch.int32, device=dev)
        dims = ak.make_dims(len(lens), 16, 4, 16, 64, 128, 1.0)
        qs = [queries(start[-1], shape, s).to(dev) for s in (1, 2)]
        wss = [ak.prefill_paged_kv8_workspace(dims, dev) for _ in range(2)]
        want = [ak.prefill_paged_kv8(x, sd, *p, td, ld, workspace=wss[0]).clone() for x in qs]
        streams, outs = [torch.cuda.Stream() for _ in range(2)], [torch.empty_like(want[0]) for _ in range(2)]
        torch.cuda.synchronize()
        for _ in range(8):
            for i in range(2):
                ak.prefill_paged_kv8(qs[i], sd, *p, td, ld, workspace=wss[i], out=outs[i], stream=streams[i])
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])
        g = torch.cuda.CUDAGraph()
        x = qs[0].clone()
        with torch.cuda.graph(g):
            ak.prefill_paged_kv8(x, sd, *p, td, ld, workspace=wss[0], out=outs[0])
        x.copy_(qs[1])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want[1])


def test_refusals(cuda_device):
    dev, shape = cuda_device, wl.DIFFQKV
    num, table = tables([40], 16, 3, 1)
    p = [t.to(dev) for t in pools(num, 16, 16, shape, 1)]
    q, td = queries(5, shape, 1).to(dev), table.to(dev)
    ld, sd = torch.tensor([40], dtype=torch.int32, device=dev), torch.tensor([0, 5], dtype=torch.int32, device=dev)
    for bad in (dict(q=q.float()), dict(q=q[:, :, :32]), dict(sd=sd[:1]), dict(ld=ld.long()), dict(td=td[0])):
        a = dict(q=q, sd=sd, td=td, ld=ld)
        a.update(bad)
        with pytest.raises((TypeError, ValueError)):
            ak.prefill_paged_kv8(a["q"], a["sd"], *p, a["td"], a["ld"])
    with pytest.raises(ak.DiffqkvError) as e:
        ak.prefill_paged_kv8(q, sd, *p, td, ld, workspace=torch.zeros(256, dtype=torch.uint8, device=dev))
    assert e.value.status == _capi.WORKSPACE
    with pytest.raises(ak.DiffqkvError) as e:
        ak.prefill_paged_kv8(q[:0], sd, *p, td, ld)
    assert e.value.status == _capi.INVALID_ARG
