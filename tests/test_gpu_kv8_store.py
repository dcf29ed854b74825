"""The quantising cache write against the definition: codes and scale bytes are equal, byte for byte, the rest of
the pool included."""
import pytest
import torch

import asymmetric_head_kv_b200 as ak
from asymmetric_head_kv_b200 import _capi
from oracle import kv8

pytestmark = pytest.mark.gpu

SHAPES = {"diffqkv": (4, 16, 64, 128), "gqa": (16, 16, 128, 128), "mqa": (1, 1, 64, 64), "k_wide": (3, 2, 128, 64)}


class Pools:
    """An 8-bit cache on the GPU and its mirror, written by the definition."""

    def __init__(self, num_pages, page, sb, shape, dev, seed=0):
        n_k, n_v, d_k, d_v = shape
        g = torch.Generator().manual_seed(seed)
        self.host = []
        for n, d in ((n_k, d_k), (n_v, d_v)):
            self.host.append((torch.randint(0, 256, (num_pages, page, n, d), generator=g, dtype=torch.uint8),
                              torch.randint(100, 140, (num_pages, page // sb, n), generator=g, dtype=torch.uint8)))
        (kc, ks), (vc, vs) = self.host
        self.gpu = [kc.to(dev).view(torch.float8_e4m3fn), vc.to(dev).view(torch.float8_e4m3fn), ks.to(dev), vs.to(dev)]
        self.dev, self.shape = dev, shape

    def rows(self, T, seed, gain=1.0):
        n_k, n_v, d_k, d_v = self.shape
        g = torch.Generator().manual_seed(seed)
        return [(torch.randn((T, n, d), generator=g) * gain).to(torch.bfloat16) for n, d in ((n_k, d_k), (n_v, d_v))]

    def store(self, k, v, slots, expect=0):
        status = torch.zeros(1, dtype=torch.int32, device=self.dev)
        ak.kv8_store(k.to(self.dev), v.to(self.dev), torch.as_tensor(slots, dtype=torch.int32).to(self.dev), *self.gpu,
                     status=status)
        assert status.item() == expect
        for x, (codes, scales) in zip((k, v), self.host):
            kv8.store(codes.numpy(), scales.numpy(), x.double().numpy(), slots)
        self.check()

    def check(self):
        for i, (codes, scales) in enumerate(self.host):
            got = self.gpu[i].view(torch.uint8).cpu()
            bad = (got != codes).nonzero()
            assert bad.numel() == 0, (i, bad[:5].tolist())
            assert torch.equal(self.gpu[2 + i].cpu(), scales), i


def _slots(page, page_ids, start, n):
    return [page_ids[p // page] * page + p % page for p in range(start, start + n)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("page,sb", [(16, 16), (8, 1), (24, 8), (32, 4), (64, 64), (128, 32), (24, 3)])
def test_chunks_then_single_rows(cuda_device, shape, page, sb):
    """A prompt's rows, a chunk that begins inside a block, then single rows whose sizes grow and shrink."""
    p = Pools(40, page, sb, SHAPES[shape], cuda_device, seed=page + sb)
    ids = torch.randperm(40, generator=torch.Generator().manual_seed(1)).tolist()
    at = 0
    for i, n in enumerate((page * 2 + 5, 1, 37)):
        p.store(*p.rows(n, i), _slots(page, ids, at, n))
        at += n
    for i, gain in enumerate((1.0, 30.0, 0.01, 900.0, 1e-3)):
        p.store(*p.rows(1, 50 + i, gain), _slots(page, ids, at, 1))
        at += 1


def test_ragged_batch_with_padding(cuda_device):
    """Rows of several requests, padding between and behind them, a slot outside the pool."""
    p = Pools(30, 16, 16, SHAPES["diffqkv"], cuda_device)
    slots = _slots(16, [4, 9], 13, 12) + [-1, -1] + _slots(16, [2], 0, 1) + _slots(16, [7, 3, 8], 5, 30) + [-1] * 7
    p.store(*p.rows(len(slots), 3), slots)
    p.store(*p.rows(3, 4), [30 * 16, 5, 2 ** 31 - 1], expect=_capi.DEVICE_PAGE)


@pytest.mark.parametrize("T", [1, 2, 31, 32, 33, 591, 592, 1183, 5000])
def test_token_counts(cuda_device, T):
    p = Pools(-(-T // 32) + 1, 32, 8, SHAPES["mqa"], cuda_device)
    p.store(*p.rows(T, T), list(range(3, T + 3)))


def test_a_block_longer_than_the_registers(cuda_device):
    p = Pools(3, 512, 512, SHAPES["k_wide"], cuda_device)
    p.store(*p.rows(700, 1), list(range(100, 800)))


@pytest.mark.parametrize("shape", ["diffqkv", "k_wide"])
@pytest.mark.parametrize("T,page,sb", [(300, 128, 128), (700, 256, 256), (2000, 64, 64), (5000, 32, 32), (6000, 128, 64),
                                       (9000, 64, 64), (3000, 24, 12)])
def test_long_blocks_shared_and_whole(cuda_device, shape, T, page, sb):
    """Runs that begin and end anywhere, by one warp (long and short of its registers), two, four and eight."""
    pages = T // page + 12
    p = Pools(pages, page, sb, SHAPES[shape], cuda_device, seed=T)
    ids = torch.randperm(pages, generator=torch.Generator().manual_seed(T)).tolist()
    slots, at, n = [], 0, 1
    while len(slots) < T:  # requests on pages of their own, each from a row of its own, a skipped token between them
        n = min(n * 3 % 997 + 1, T - len(slots))
        start = (5 * n) % page if len(ids) - at > -(-(n + page) // page) else 0
        need = -(-(start + n) // page)
        if at + need > len(ids):
            break
        slots += _slots(page, ids[at:at + need], start, n) + [-1]
        at += need
    slots += [-1] * (T - len(slots))
    p.store(*p.rows(len(slots), 3), slots)


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan"), 3.3e38, 2.0 ** -133, 0.0])
def test_special_values(cuda_device, value):
    p = Pools(4, 16, 16, SHAPES["diffqkv"], cuda_device)
    k, v = p.rows(10, 2)
    k[3, 1, 5] = value
    v[9] = value
    p.store(k, v, list(range(10)))
    k, v = p.rows(2, 3, 1e-2)
    k[0, 2, 63] = value
    p.store(k, v, [10, 11])


def test_largest_scale_jump(cuda_device):
    """A block of the smallest scale, then a row that takes it to the largest: the old rows become zero."""
    p = Pools(2, 8, 8, SHAPES["mqa"], cuda_device)
    k, v = p.rows(2, 1, 0.0)
    p.store(k, v, [0, 1])
    k, v = p.rows(1, 1)
    k[0, 0, 0] = v[0, 0, 0] = 3e38
    p.store(k, v, [2])


def test_no_tokens(cuda_device):
    p = Pools(2, 8, 8, SHAPES["mqa"], cuda_device)
    p.store(*p.rows(0, 1), [])
    p.store(*p.rows(5, 1), [-1] * 5)


def test_offsets_past_32_bits(cuda_device):
    """A V pool of more than 2^31 bytes: rows at its end land there and nowhere else."""
    page, shape = 64, (1, 16, 64, 128)
    num = 2 ** 31 // (page * 16 * 128) + 40
    dev = cuda_device
    pools = ak.kv8_pools(num, page, *shape, scale_block=16, device=dev)
    k = torch.ones((20, 1, 64), dtype=torch.bfloat16, device=dev)
    v = torch.full((20, 16, 128), 3.0, dtype=torch.bfloat16, device=dev)
    first = (num - 1) * page + 10
    ak.kv8_store(k, v, torch.arange(first, first + 20, dtype=torch.int32, device=dev), *pools)
    vp = pools[1].view(torch.uint8)
    assert int((vp != 0).sum()) == 20 * 16 * 128 and (vp[num - 1, 10:30] != 0).all()


def test_refusals(cuda_device):
    dev = cuda_device
    k_pages, v_pages, ks, vs = ak.kv8_pools(4, 16, 2, 4, 64, 128, device=dev)
    k = torch.zeros((3, 2, 64), dtype=torch.bfloat16, device=dev)
    v = torch.zeros((3, 4, 128), dtype=torch.bfloat16, device=dev)
    slots = torch.arange(3, dtype=torch.int32, device=dev)
    ak.kv8_store(k, v, slots, k_pages, v_pages, ks, vs)
    for bad in (dict(k=k.float()), dict(v=v[:, :2]), dict(slots=slots.long()), dict(kp=k_pages.view(torch.uint8)),
                dict(ks=ks[:, :, :1]), dict(vs=vs.cpu()), dict(slots=slots.cpu())):
        a = dict(k=k, v=v, slots=slots, kp=k_pages, vp=v_pages, ks=ks, vs=vs)
        a.update(bad)
        with pytest.raises((TypeError, ValueError)):
            ak.kv8_store(*a.values())
    odd = ak.kv8_pools(4, 12, 2, 4, 64, 128, device=dev)
    with pytest.raises(ak.DiffqkvError) as e:
        ak.kv8_store(k, v, slots, *odd)
    assert e.value.status == _capi.UNSUPPORTED
    with pytest.raises(ValueError):
        ak.kv8_pools(4, 16, 2, 4, 64, 128, scale_block=5)


def test_a_step_from_lengths_to_the_cache(cuda_device):
    """page_map and kv8_store one after another on another stream, captured: the map's slots go straight in."""
    dev, page = cuda_device, 16
    p = Pools(64, page, 16, SHAPES["diffqkv"], dev)
    seq = torch.tensor([17, 0, 40], dtype=torch.int32, device=dev)
    new = torch.tensor([1, 50, 9], dtype=torch.int32, device=dev)
    table = torch.full((3, 8), -1, dtype=torch.int32)
    table[0, :2] = torch.tensor([60, 61])
    table[2, :3] = torch.tensor([50, 51, 52])
    free = torch.arange(10, 30, dtype=torch.int32, device=dev)
    k, v = p.rows(64, 8)
    kd, vd, bt = k.to(dev), v.to(dev), table.to(dev)
    outs = [torch.empty(n, dtype=torch.int32, device=dev) for n in (4, 64, 64, 3, 1)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ak.page_map(seq, new, bt, free, page, 64, *outs)
        ak.kv8_store(kd, vd, outs[1], *p.gpu)
    g.replay()
    torch.cuda.synchronize()
    want = kv8.page_map([17, 0, 40], [1, 50, 9], table.tolist(), list(range(10, 30)), page, 64, 64)
    assert outs[1].tolist() == want["slot_map"].tolist()
    for x, (codes, scales) in zip((k, v), p.host):
        kv8.store(codes.numpy(), scales.numpy(), x.double().numpy(), want["slot_map"])
    p.check()
