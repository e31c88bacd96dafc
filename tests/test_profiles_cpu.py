"""The DRAM traffic that bench.py reports is what the committed summary of the
captures says, row by row, all taken on one state of the kernel sources."""
import json
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_traffic_record_is_the_summary():
    with open(os.path.join(ROOT, "profiles", "traffic.json")) as f:
        record = json.load(f)
    with open(os.path.join(ROOT, "profiles", "dram_traffic_per_launch.md")) as f:
        text = f.read()
    rows = {m[0]: m for m in (
        [c.strip() for c in line.strip("|").split("|")] for line in text.splitlines() if line.startswith("| ")) if m[0] in record}
    assert set(rows) == set(record)
    (stated,) = re.findall(r"kernel\s+sources of these workloads: ([0-9a-f]{16}); all rows taken on these", text)
    for name, entry in record.items():
        moved, least = (int(rows[name][i].replace(",", "")) for i in (5, 6))
        assert entry["dram_bytes_per_launch"] == moved and entry["source_hash"] == stated, name
        assert rows[name][7] == f"{moved / least:.3f}", name
