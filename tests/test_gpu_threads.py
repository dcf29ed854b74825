"""Calls that are the first CUDA work of their host thread."""
import threading

import pytest
import torch

import asymmetric_head_kv_b200 as ak
import workloads as wl
from kv8_inputs import pools, queries, tables
from workloads import Shape

pytestmark = pytest.mark.gpu

SHAPE = Shape(4, 2, 4, 64, 128)


def _calls(dev):
    i32 = lambda x: torch.as_tensor(x, dtype=torch.int32).to(dev)  # noqa: E731
    lens = [90, 40]
    num, table = tables(lens, 16, 6, 1)
    p = [t.to(dev) for t in pools(num, 16, 16, SHAPE, 1)]
    td, ld, sd = table.to(dev), i32(lens), i32([0, 30, 60])
    dims = ak.make_dims(2, 4, 2, 4, 64, 128, SHAPE.scale)
    ws = torch.zeros(64 << 20, dtype=torch.uint8, device=dev)
    word = torch.zeros(1, dtype=torch.int32, device=dev)
    q, rows = queries(2, SHAPE, 1).to(dev), queries(60, SHAPE, 2).to(dev)
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device=dev)  # noqa: E731
    d = {k: v.to(dev) if isinstance(v, torch.Tensor) else v for k, v in
         wl.random_decode_inputs(2, 90, SHAPE, seed=3, seq_lens=lens).items()}
    kp, vp = bf(num, 16, 2, 64), bf(num, 16, 4, 128)
    tws = ak.decode_topv_workspace(dims, 90, 8, dev)
    out, idx, pre = bf(2, 4, 128), torch.zeros((2, 4, 8), dtype=torch.int32, device=dev), bf(1, 40, 4, 128)
    ro, maps = bf(60, 4, 128), [torch.zeros(n, dtype=torch.int32, device=dev) for n in (3, 8, 8, 2, 1)]
    x, wg, wd, h, qo = bf(8, 64), bf(128, 64), bf(64, 128), bf(8, 128), bf(8, 64)
    pq, pk, pv = bf(1, 40, 4, 64), bf(1, 40, 2, 64), bf(1, 40, 4, 128)
    new = (torch.ones(5, 2, 64, device=dev).bfloat16(), torch.ones(5, 4, 128, device=dev).bfloat16(), i32([0, 1, 2, 3, 4]))
    fresh = [t.clone() for t in p]
    ones, free = i32([1, 1]), i32([num, num + 1])
    return {
        "decode": lambda: ak.decode(d["q"], d["k_cache"], d["v_cache"], d["seq_lens"], scale=d["scale"], out=out, workspace=ws),
        "decode_paged": lambda: ak.decode_paged(q, kp, vp, td, ld, out=out, workspace=ws),
        "decode_noalloc": lambda: ak.decode_noalloc(d["q"], d["k_cache"], d["v_cache"], d["seq_lens"], scale=d["scale"],
                                                    out=out),
        "decode_topv": lambda: ak.decode_topv(d["q"], d["k_cache"], d["v_cache"], d["seq_lens"], 8, scale=d["scale"], out=out,
                                              idx_out=idx, workspace=tws)[0],
        "prefill_causal": lambda: ak.prefill_causal(pq, pk, pv, scale=0.125, out=pre),
        "augq_project": lambda: ak.augq_project(x, wg, wg, wd, h_out=h, q_out=qo),
        "decode_paged_kv8": lambda: ak.decode_paged_kv8(q, *p, td, ld, out=out, workspace=ws),
        "prefill_paged_kv8": lambda: ak.prefill_paged_kv8(rows, sd, *p, td, ld, out=ro, workspace=ws),
        "page_map": lambda: ak.page_map(ld, ones, td, free, 16, num + 4, *maps, status=word)[1],
        "kv8_store": lambda: (ak.kv8_store(*new, *fresh, status=word), fresh[0].view(torch.uint8))[1],
    }


NAMES = ("decode", "decode_paged", "decode_noalloc", "decode_topv", "prefill_causal", "augq_project", "decode_paged_kv8",
         "prefill_paged_kv8", "page_map", "kv8_store")


@pytest.mark.parametrize("name", NAMES)
def test_a_new_thread_may_begin_with_any_call(cuda_device, name):
    call = _calls(cuda_device)[name]
    torch.cuda.synchronize()
    got, failed = [], []

    def work():
        try:
            got.append(call())
        except Exception as e:  # noqa: BLE001  (reported by the test's thread)
            failed.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    assert not failed, failed
    torch.cuda.synchronize()
    first = [x.clone() for x in (got[0] if isinstance(got[0], tuple) else (got[0],))]
    again = call()
    torch.cuda.synchronize()
    for a, b in zip(first, again if isinstance(again, tuple) else (again,)):
        assert torch.equal(a, b)
