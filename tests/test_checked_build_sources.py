"""Every kernel file tests its global accesses in the checked build (its GPU tests run what they do not look into: code
whose checks were missing would pass them all the same)."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "asymmetric_head_kv_b200", "csrc")
KERNELS = sorted(f for f in glob.glob(os.path.join(CSRC, "*.cu"))
                 if "__global__" in open(f).read()
                 # the wait self-test touches nothing; the query fold has no status word to report into
                 and os.path.basename(f) not in ("api.cu", "fold.cu"))

# what each file's kernels index that a wrong size, length or table could lead astray
CHECKED = {
    "page_map.cu": ["a.num_free", "a.batch", "a.max_blocks"],
    "kv8_store.cu": ["a.slots / a.sb", "a.slots", "a.tokens"],
    "decode_kv8.cu": ["a.partial_slots", "kWsCounters", "a.scale_blocks", "(long long)a.batch * a.n_q"],
    "prefill_kv8.cu": ["kSlots", "a.scale_blocks", "a.tokens", "(long long)a.tokens * a.n_q"],
}


@pytest.mark.parametrize("path", KERNELS, ids=os.path.basename)
def test_kernels_check_their_indices(path):
    src = open(path).read()
    extents = re.findall(r"in_bounds\((?:[^;]*?), ([^,;]*(?:\([^;]*?\))?[^,;]*), a\.status\)", src)
    assert "in_bounds(" in src
    for want in CHECKED.get(os.path.basename(path), []):
        assert any(want in e for e in extents), f"no access is checked against {want}"
