"""Page-map outputs that overlap inputs or one another are refused: every CTA redoes the sums over the requests, so one
that wrote over them would change another's."""
import pytest
import torch

import asymmetric_head_kv_b200 as ak
from asymmetric_head_kv_b200 import _capi
from asymmetric_head_kv_b200.build import build
from oracle import kv8


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


@pytest.mark.gpu
def test_neighbours_are_not(cuda_device):
    """Every buffer cut from one allocation, side by side, and one tensor for both inputs: the map is right."""
    B, cap = 4, 64
    pool = torch.zeros(512, dtype=torch.int32, device=cuda_device)
    at = 0

    def cut(n):
        nonlocal at
        at += n
        return pool[at - n:at]
    slots, positions, lens, start, total, used, free = cut(cap), cut(cap), cut(B), cut(B + 1), cut(B), cut(1), cut(16)
    table = cut(B * 8).view(B, 8)
    lens.copy_(torch.tensor([3, 0, 5, 1]))
    free.copy_(torch.arange(16, 32))
    table[:, 0] = torch.tensor([7, 6, 5, 4])
    word = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    ak.page_map(lens, lens, table, free, 4, 40, start, slots, positions, total, used, status=word)
    want = kv8.page_map([3, 0, 5, 1], [3, 0, 5, 1], [[7] + [0] * 7, [6] + [0] * 7, [5] + [0] * 7, [4] + [0] * 7],
                        range(16, 32), 4, 40, cap)
    assert word.item() == want["status"]
    for got, name in ((start, "query_start"), (slots, "slot_map"), (positions, "positions"), (total, "total_lens"),
                      (used, "pages_used"), (table, "block_table")):
        assert got.tolist() == want[name].tolist(), name
