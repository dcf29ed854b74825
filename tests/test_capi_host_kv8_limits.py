"""Sizes at which the 8-bit cache's calls begin to refuse, as the header states them."""
import pytest

import asymmetric_head_kv_b200 as ak
from asymmetric_head_kv_b200 import _capi
from asymmetric_head_kv_b200.build import build


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()


def dims(n_q, n_k, n_v):
    return ak.make_dims(2, n_q, n_k, n_v, 64, 128, 0.125)


CACHE = _capi.Kv8Cache(0x10000, 0x20000, 0x30000, 0x40000, 8, 16, 16)


@pytest.mark.parametrize("ratio", [3, 5, 6, 7, 12, 15, 24, 32])
def test_decode_refuses_other_ratios_of_heads(ratio):
    d = dims(2 * ratio, 2, 2)
    assert _capi.lib().diffqkv_decode_paged_kv8(d, CACHE, 0x1000, 0x2000, 4, 0x3000, 0, 0x4000, 0x5000, 1 << 40,
                                                None) == _capi.UNSUPPORTED


@pytest.mark.parametrize("heads,tokens", [((16, 4, 16), 2 ** 27 // 16), ((2, 2, 1), 2 ** 26), ((1, 1, 1), 2 ** 27),
                                          ((65534, 2, 65534), 1), ((32768, 32768, 32768), 1)])
def test_the_write_refuses_more_rows_than_it_has_threads_for(heads, tokens):
    assert _capi.lib().diffqkv_kv8_store(dims(*heads), CACHE, 0x1000, 0x2000, 0x3000, tokens, None,
                                         None) == _capi.UNSUPPORTED
