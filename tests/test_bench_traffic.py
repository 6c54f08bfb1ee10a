"""The DRAM traffic that bench.py reports beside the decode was captured on the decode sources as they
are: a change of these goes with new captures, and what others need of shared code stays out of them."""

import json
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_every_capture_is_of_the_current_sources():
    sys.path.insert(0, ROOT)
    import bench
    rec = json.load(open(os.path.join(ROOT, "profiles", "traffic.json")))["decode_split_mma"]
    for name, e in rec.items():
        assert bench.profiled_traffic(name) == float(e["traffic_bytes_per_launch"]), name
