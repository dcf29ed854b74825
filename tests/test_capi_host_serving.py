"""Argument checks of the serving entry points that need no GPU: every refusal comes before anything is launched."""
import ctypes

import pytest
import torch

import asymmetric_head_kv_b200 as ak
from asymmetric_head_kv_b200 import _capi
from asymmetric_head_kv_b200.build import build


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()


def dims(**kw):
    base = dict(batch=2, n_q=16, n_k=4, n_v=16, d_k=64, d_v=128, scale=0.125)
    base.update(kw)
    return ak.make_dims(**base)


def cache(**kw):
    base = dict(k_pages=0x10000, v_pages=0x20000, k_scales=0x30000, v_scales=0x40000, num_pages=8, page_size=16,
                scale_block=16)
    base.update(kw)
    return _capi.Kv8Cache(**base)


def page_map(**kw):
    a = dict(batch=2, seq_lens=0x100, new_lens=0x200, block_table=0x300, max_blocks=4, page_size=16, num_pages=8,
             free_pages=0x400, num_free=3, capacity=9, query_start=0x500, slot_map=0x600, positions=0x700,
             total_lens=0x800, pages_used=0x900, status=None, stream=None)
    a.update(kw)
    return _capi.lib().diffqkv_page_map(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(batch=0), _capi.INVALID_ARG), (dict(seq_lens=None), _capi.INVALID_ARG), (dict(new_lens=None), _capi.INVALID_ARG),
    (dict(block_table=None), _capi.INVALID_ARG), (dict(max_blocks=0), _capi.INVALID_ARG),
    (dict(page_size=0), _capi.INVALID_ARG), (dict(num_pages=0), _capi.INVALID_ARG), (dict(num_free=-1), _capi.INVALID_ARG),
    (dict(free_pages=None), _capi.INVALID_ARG), (dict(capacity=-1), _capi.INVALID_ARG),
    (dict(slot_map=None), _capi.INVALID_ARG), (dict(query_start=None), _capi.INVALID_ARG),
    (dict(total_lens=None), _capi.INVALID_ARG), (dict(pages_used=None), _capi.INVALID_ARG),
    (dict(max_blocks=2 ** 30, page_size=16), _capi.UNSUPPORTED), (dict(num_pages=2 ** 30, page_size=16), _capi.UNSUPPORTED),
    (dict(batch=2 ** 25), _capi.UNSUPPORTED), (dict(seq_lens=0x102), _capi.MISALIGNED),
    (dict(slot_map=0x604), _capi.MISALIGNED), (dict(positions=0x708), _capi.MISALIGNED), (dict(status=0x2), _capi.MISALIGNED),
])
def test_page_map_refuses(kw, code):
    assert page_map(**kw) == code


CACHE_REFUSALS = [
    (dict(), dict(k_pages=None), _capi.INVALID_ARG), (dict(), dict(v_scales=None), _capi.INVALID_ARG),
    (dict(), dict(num_pages=0), _capi.INVALID_ARG), (dict(), dict(scale_block=0), _capi.INVALID_ARG),
    (dict(), dict(scale_block=5), _capi.INVALID_ARG), (dict(), dict(page_size=12, scale_block=12), _capi.UNSUPPORTED),
    (dict(), dict(num_pages=2 ** 28), _capi.UNSUPPORTED), (dict(), dict(k_pages=0x10008), _capi.MISALIGNED),
    (dict(n_k=3), dict(), _capi.INVALID_ARG), (dict(scale=0.0), dict(), _capi.INVALID_ARG),
    (dict(d_k=96), dict(), _capi.UNSUPPORTED), (dict(d_v=256), dict(), _capi.UNSUPPORTED),
]


def store(d, c, k=0x1000, v=0x2000, slots=0x3000, tokens=3, status=None):
    return _capi.lib().diffqkv_kv8_store(d, c, k, v, slots, tokens, status, None)


def decode(d, c, q=0x1000, table=0x2000, mb=4, lens=0x3000, out=0x4000, ws=0x5000, n=1 << 30):
    return _capi.lib().diffqkv_decode_paged_kv8(d, c, q, table, mb, lens, 0, out, ws, n, None)


def prefill(d, c, q=0x1000, start=0x1800, tokens=5, table=0x2000, mb=4, lens=0x3000, out=0x4000, ws=0x5000, n=1 << 30):
    return _capi.lib().diffqkv_prefill_paged_kv8(d, c, q, start, tokens, table, mb, lens, out, ws, n, None)


@pytest.mark.parametrize("call", [store, decode, prefill])
@pytest.mark.parametrize("dim_kw,cache_kw,code", CACHE_REFUSALS)
def test_a_bad_cache_is_refused(call, dim_kw, cache_kw, code):
    assert call(dims(**dim_kw), cache(**cache_kw)) == code
    assert call(None, cache()) == _capi.INVALID_ARG
    assert call(dims(), None) == _capi.INVALID_ARG


def test_store_refuses():
    d, c = dims(), cache()
    assert store(d, c, tokens=-1) == _capi.INVALID_ARG
    assert store(d, c, k=None) == _capi.INVALID_ARG
    assert store(d, c, slots=None) == _capi.INVALID_ARG
    assert store(d, c, v=0x2008) == _capi.MISALIGNED
    assert store(d, c, slots=0x3002) == _capi.MISALIGNED
    assert store(d, c, k=None, v=None, slots=None, tokens=0) == _capi.OK      # nothing to do


def test_decode_refuses():
    d, c = dims(), cache()
    assert decode(d, c, q=None) == _capi.INVALID_ARG
    assert decode(d, c, mb=0) == _capi.INVALID_ARG
    assert decode(d, c, mb=2 ** 28) == _capi.INVALID_ARG
    assert decode(dims(n_q=96, n_k=4, n_v=16), c) == _capi.UNSUPPORTED        # 24 query heads per K head
    assert decode(d, c, out=0x4008) == _capi.MISALIGNED
    assert decode(d, c, table=0x2002) == _capi.MISALIGNED
    assert decode(d, c, ws=None) == _capi.WORKSPACE
    assert decode(d, c, n=16) == _capi.WORKSPACE


def test_prefill_refuses():
    d, c = dims(), cache()
    assert prefill(d, c, tokens=0) == _capi.INVALID_ARG
    assert prefill(d, c, start=None) == _capi.INVALID_ARG
    assert prefill(d, c, mb=2 ** 28) == _capi.INVALID_ARG
    assert prefill(d, c, q=0x1004) == _capi.MISALIGNED
    assert prefill(d, c, start=0x1802) == _capi.MISALIGNED
    assert prefill(d, c, ws=None) == _capi.WORKSPACE
    assert prefill(d, c, n=4096) == _capi.WORKSPACE
    size = _capi.lib().diffqkv_prefill_paged_kv8_workspace_size
    assert size(d) > 4096 and size(dims(d_v=64)) < size(d) and size(dims(n_k=3)) == 0 and size(None) == 0
    assert size(dims(batch=500)) == size(d)                                   # reusable whatever the batch


def test_host_tensors_are_refused_before_any_device_work():
    i32, bf16 = torch.int32, torch.bfloat16
    z = torch.zeros
    kp, vp, ks, vs = ak.kv8_pools(4, 16, 4, 16, 64, 128, device="cpu")
    with pytest.raises(ValueError):
        ak.page_map(z(2, dtype=i32), z(2, dtype=i32), z((2, 4), dtype=i32), z(3, dtype=i32), 16, 8, capacity=4)
    with pytest.raises(ValueError):
        ak.kv8_store(z((3, 4, 64), dtype=bf16), z((3, 16, 128), dtype=bf16), z(3, dtype=i32), kp, vp, ks, vs)
    with pytest.raises(ValueError):
        ak.decode_paged_kv8(z((1, 16, 64), dtype=bf16), kp, vp, ks, vs, z((1, 4), dtype=i32), z(1, dtype=i32))
    with pytest.raises(ValueError):
        ak.prefill_paged_kv8(z((3, 16, 64), dtype=bf16), z(2, dtype=i32), kp, vp, ks, vs, z((1, 4), dtype=i32),
                             z(1, dtype=i32))
    with pytest.raises((TypeError, ValueError)):  # whichever of the wrong arguments is looked at first
        ak.kv8_store(None, None, None, kp, vp, ks, vs)


def test_the_extension_refuses_calls_before_it_is_bound():
    from asymmetric_head_kv_b200 import _serving as bound
    with pytest.raises(TypeError):
        bound.page_map(1, 2)
    with pytest.raises(ValueError):
        bound.bind(0, 0, 0, 0)


def test_pools():
    kp, vp, ks, vs = ak.kv8_pools(5, 32, 2, 3, 64, 128, scale_block=8, device="cpu")
    assert kp.shape == (5, 32, 2, 64) and vp.shape == (5, 32, 3, 128) and kp.dtype == torch.float8_e4m3fn
    assert ks.shape == (5, 4, 2) and vs.shape == (5, 4, 3) and (ks == 127).all()
    assert ctypes.sizeof(_capi.Kv8Cache) == 4 * 8 + 3 * 4 + 4
