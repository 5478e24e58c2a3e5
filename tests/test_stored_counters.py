"""The traffic figures under profiles/ belong to the kernels in the tree: bench.py reports one only
while the digest of the kernel sources is the stored one."""
import glob
import json
import os

import pytest

from hierarchical_tiling_amd import counters

PROFILES = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "profiles")
FILES = sorted(glob.glob(os.path.join(PROFILES, "*_traffic.txt")))


@pytest.mark.parametrize("path", FILES, ids=[os.path.basename(f)[:-len("_traffic.txt")] for f in FILES])
def test_traffic_is_of_these_kernels(path):
    text = open(path).read()
    s = json.loads(text[text.index("{"):text.rindex("}") + 1])
    assert s["source_digest"] == counters.source_digest()
    got, source = counters.traffic_for(s["kernel"], s["workload"], PROFILES)
    assert got == s["traffic_bytes"], source
