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
