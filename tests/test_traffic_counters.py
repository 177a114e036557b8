"""The committed DRAM counters belong to the committed kernel sources, so that bench.py's line carries them:
an entry whose sources have changed is retaken (or taken out) with the change."""
import json
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
with open(os.path.join(ROOT, "profiles", "traffic.json")) as f:
    ENTRIES = {k: v for k, v in json.load(f).items() if not k.startswith("_")}


@pytest.mark.parametrize("key", list(ENTRIES))
def test_the_bench_line_carries_its_dram_bytes(key):
    sys.path.insert(0, ROOT)
    import bench
    assert bench.traffic_for(key) == ENTRIES[key]["bytes"] > 0
