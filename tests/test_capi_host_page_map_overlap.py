"""Page-map outputs that overlap inputs or one another are refused: every CTA redoes the sums over the requests, so one
that wrote over them would change another's."""
import pytest

import asymmetric_head_kv_b200 as ak  # noqa: F401  (the package loads the library)
from asymmetric_head_kv_b200 import _capi
from asymmetric_head_kv_b200.build import build


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()


ARGS = dict(batch=4, seq_lens=0x1000, new_lens=0x2000, block_table=0x3000, max_blocks=8, page_size=16, num_pages=8,
            free_pages=0x4000, num_free=16, capacity=64, query_start=0x5000, slot_map=0x6000, positions=0x7000,
            total_lens=0x8000, pages_used=0x9000, status=None, stream=None)
WORDS = dict(seq_lens=4, new_lens=4, block_table=32, free_pages=16, query_start=5, slot_map=64, positions=64, total_lens=4,
             pages_used=1)
OUT = ("block_table", "query_start", "slot_map", "positions", "total_lens", "pages_used")


def call(**kw):
    return _capi.lib().diffqkv_page_map(*dict(ARGS, **kw).values())


@pytest.mark.parametrize("out", OUT)
@pytest.mark.parametrize("other", WORDS)
def test_overlaps_are_refused(out, other):
    if out == other:
        return
    step = 16 if out in ("slot_map", "positions") else 4
    assert call(**{out: ARGS[other]}) == _capi.INVALID_ARG
    # the output's last word on the other's first, and its first on the other's last
    low, high = ARGS[other] - 4 * (WORDS[out] - 1), ARGS[other] + 4 * (WORDS[other] - 1)
    assert call(**{out: -(-low // step) * step}) == _capi.INVALID_ARG
    assert call(**{out: high // step * step}) == _capi.INVALID_ARG


def test_neighbours_are_not():
    """Side by side, and the inputs among themselves, is fine: the call gets as far as looking for a device."""
    ok = call()
    assert ok != _capi.INVALID_ARG
    assert call(new_lens=ARGS["seq_lens"]) == ok
    assert call(total_lens=ARGS["seq_lens"] + 16) == ok and call(query_start=ARGS["new_lens"] - 20) == ok
    assert call(positions=None) == ok
    assert call(slot_map=ARGS["free_pages"] + 64) == ok
