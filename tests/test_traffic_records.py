"""The committed DRAM records belong to the present kernel sources: a change in a
header that they share would drop them from the benchmark's output."""
import glob
import json
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_every_record_is_of_a_present_source():
    sys.path.insert(0, ROOT)
    import bench

    present = {bench.source_hash(f) for f in glob.glob(os.path.join(ROOT, "attention_backward_gb300/csrc/*.cu"))}
    with open(os.path.join(ROOT, "profiles", "traffic.json")) as f:
        records = json.load(f)
    assert records
    assert [name for name, r in records.items() if r["source_sha256_16"] not in present] == []
