"""A NaN in a stored V row reaches the rows that see it, and no earlier one."""
import pytest
import torch

import asymmetric_head_kv_b200 as ak
from kv8_inputs import pools, queries, tables
from workloads import Shape

pytestmark = pytest.mark.gpu


def _run(p, q, start, table, lens, shape, dev):
    i32 = lambda x: torch.as_tensor(x, dtype=torch.int32).to(dev)  # noqa: E731
    return ak.prefill_paged_kv8(q.to(dev), i32(start), *[t.to(dev) for t in p], table.to(dev), i32(lens), scale=shape.scale)


@pytest.mark.parametrize("shape", [Shape(4, 2, 2, 64, 128), Shape(2, 1, 2, 128, 64), Shape(2, 2, 1, 64, 64)], ids=str)
@pytest.mark.parametrize("rows,lens", [([700], [700]), ([300, 150], [2000, 150]), ([5, 40], [9001, 4001]), ([256], [320])],
                         ids=str)
def test_a_nan_value_reaches_the_rows_that_see_it_alone(cuda_device, shape, rows, lens):
    """Whole and cut units, several NaNs a column, both signs of the code, in and out of the tiles on the diagonal."""
    dev = cuda_device
    num, table = tables(lens, 16, -(-max(lens) // 16), 1)
    p = pools(num, 16, 16, shape, 1)
    start = [sum(rows[:i]) for i in range(len(rows) + 1)]
    q = queries(start[-1], shape, 2)
    clean = _run(p, q, start, table, lens, shape, dev)
    per_v = shape.n_q // shape.n_v
    for b, (m, n) in enumerate(zip(rows, lens)):
        first = n - m
        spots = {first, n - 1, first + m // 2, max(0, first - 1), n - 2, (n - 1) // 64 * 64, first + m // 3}
        codes = p[1].view(torch.uint8).clone()
        want = clean.clone()
        for i, j in enumerate(sorted(spots)):
            vh, col = i % shape.n_v, (13 * i + 5) % shape.d_v if i != 2 else 5
            codes[int(table[b, j // 16]), j % 16, vh, col] = 0x7F if i % 2 else 0xFF
            lo = start[b] + max(0, j - first)
            want[lo:start[b + 1], vh * per_v:(vh + 1) * per_v, col] = float("nan")
        out = _run([p[0], codes.view(torch.float8_e4m3fn), *p[2:]], q, start, table, lens, shape, dev)
        assert torch.equal(torch.isnan(out), torch.isnan(want))
        ok = ~torch.isnan(want)
        assert torch.equal(out[ok], want[ok])
