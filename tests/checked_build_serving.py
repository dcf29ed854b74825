"""The serving operators through the checked build (device-side index checks on): run as a script with
DIFFQKV_BOUNDS_CHECK=1 by tests/test_gpu_checked_serving.py.  Every result must match its definition and every status
word stay clear.  Prints "all cases ok" at the end."""
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

import torch  # noqa: E402

import asymmetric_head_kv_b200 as ak  # noqa: E402
from asymmetric_head_kv_b200 import _capi  # noqa: E402
from kv8_inputs import check_decode, check_prefill, queries  # noqa: E402
from oracle import kv8  # noqa: E402
from workloads import DIFFQKV, GQA_CONTROL, Shape  # noqa: E402


def main():
    assert _capi.CHECKED and _capi.LIB_PATH.endswith("libdiffqkv_checked.so"), "not the checked build"
    dev = torch.device("cuda", 0)
    for shape, page, sb in ((DIFFQKV, 16, 16), (GQA_CONTROL, 24, 8), (Shape(16, 1, 1, 64, 64), 64, 4),
                            (Shape(24, 12, 8, 128, 64), 8, 8)):
        lens, num, mb = [1, 129, 300, 0], 80, 60
        free = torch.randperm(num, generator=torch.Generator().manual_seed(1)).to(torch.int32)
        table = torch.full((4, mb), -1, dtype=torch.int32, device=dev)
        word = torch.zeros(1, dtype=torch.int32, device=dev)
        new = torch.tensor(lens, dtype=torch.int32, device=dev)
        start, slots, _, total, _ = ak.page_map(torch.zeros_like(new), new, table, free.to(dev), page, num,
                                                capacity=sum(lens) + 3, status=word)
        gpu = ak.kv8_pools(num, page, shape.n_k, shape.n_v, shape.d_k, shape.d_v, scale_block=sb, device=dev)
        pool = [t.cpu().clone() for t in gpu]
        g = torch.Generator().manual_seed(2)
        k = torch.randn((slots.numel(), shape.n_k, shape.d_k), generator=g).to(torch.bfloat16)
        v = torch.randn((slots.numel(), shape.n_v, shape.d_v), generator=g).to(torch.bfloat16)
        ak.kv8_store(k.to(dev), v.to(dev), slots, *gpu, status=word)
        torch.cuda.synchronize()
        assert word.item() == 0
        for x, codes, scales in ((k, pool[0], pool[2]), (v, pool[1], pool[3])):
            kv8.store(codes.view(torch.uint8).numpy(), scales.numpy(), x.double().numpy(), slots.cpu().tolist())
        for a, b in zip(gpu, pool):
            assert torch.equal(a.cpu().view(torch.uint8), b.view(torch.uint8))
        dims = ak.make_dims(4, shape.n_q, shape.n_k, shape.n_v, shape.d_k, shape.d_v, shape.scale)
        q = queries(4, shape, 3)
        ws = ak.decode_workspace(dims, device=dev)
        out = ak.decode_paged_kv8(q.to(dev), *gpu, table, total, scale=shape.scale, workspace=ws)
        assert ak.workspace_status(ws) == 0
        check_decode(out, q, pool, table.cpu(), lens, shape.scale, "checked decode")
        q = queries(sum(lens), shape, 4)
        ws = ak.prefill_paged_kv8_workspace(dims, dev)
        out = ak.prefill_paged_kv8(q.to(dev), start, *gpu, table, total, scale=shape.scale, workspace=ws)
        assert ak.workspace_status(ws) == 0
        check_prefill(out, q, start.cpu().tolist(), pool, table.cpu(), lens, shape.scale, "checked prefill")
        print(shape, "ok")
    print("all cases ok")


if __name__ == "__main__":
    main()
