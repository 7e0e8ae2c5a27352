"""The benchmark's DRAM-traffic figure comes from a committed capture that is valid only for the sources it was taken
from: the pair attention kernel and the headers it includes."""
import json
import os

import bench


def test_traffic_record_belongs_to_the_present_sources():
    rec = json.load(open(os.path.join(bench.ROOT, "profiles", "traffic.json")))["gqa_attn_fwd_T32768"]
    assert rec["source_key"] == bench.source_key(bench.PAIR_SOURCES)
    assert bench.traffic_for("gqa_attn_fwd_T32768", bench.PAIR_SOURCES) == rec["bytes_per_launch"]
