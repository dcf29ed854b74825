"""The extension that marshals the serving operators, in processes of its own (what it is bound to is process-wide)."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _child(code):
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-2000:]
    return r.stdout


@pytest.fixture(scope="module", autouse=True)
def _built():
    from asymmetric_head_kv_b200.build import build
    build()


def test_calls_before_it_is_bound_are_refused():
    out = _child('''
import asymmetric_head_kv_b200
from asymmetric_head_kv_b200 import _serving as ext
for call, n in ((ext.page_map, 13), (ext.kv8_store, 9), (ext.decode_paged_kv8, 12), (ext.prefill_paged_kv8, 12)):
    try:
        call(*[None] * n)
    except RuntimeError as e:
        assert "bound" in str(e), e
        print("refused")
''')
    assert out.split() == ["refused"] * 4


@pytest.mark.gpu
def test_other_threads_run_while_a_call_waits(cuda_device):
    """An entry point that blocks (here libc's usleep, in the place of a launch that waits for a full queue) holds no
    interpreter lock."""
    out = _child('''
import ctypes, threading, time
import torch
from asymmetric_head_kv_b200 import _serving as ext
usleep = ctypes.cast(ctypes.CDLL(None).usleep, ctypes.c_void_p).value
ext.bind(usleep, usleep, usleep, usleep)
B = 400000  # usleep's argument, by page_map's first one
z = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")
lens, table, one, start, slots = z(B), z(B).view(B, 1), z(1), z(B + 1), z(4)
torch.cuda.synchronize()
ticks, stop = [], threading.Event()
def tick():
    while not stop.is_set():
        ticks.append(time.monotonic())
        time.sleep(0.001)
t = threading.Thread(target=tick)
t.start()
time.sleep(0.05)
t0 = time.monotonic()
assert ext.page_map(lens, lens, table, one, 16, 8, start, slots, None, lens, one, None, None) == 0
t1 = time.monotonic()
stop.set()
t.join()
print(t1 - t0, sum(t0 + 0.01 < x < t1 - 0.01 for x in ticks))
''')
    took, ticks = out.split()
    assert float(took) > 0.35 and int(ticks) >= 20, out
