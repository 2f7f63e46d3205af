"""The adapter kernels' recorded counters belong to the sources that are here: bench.py passes over a
record of other ones, and its line then has neither traffic nor matrix counters."""
import json
import os

import pytest

import bench

RECORDS = [(f, key) for f in (bench.TRAFFIC_FILE, bench.COUNTERS_FILE) for key in sorted(json.load(open(f)))]


@pytest.mark.parametrize("path,key", RECORDS, ids=[os.path.basename(f) + ":" + k for f, k in RECORDS])
def test_record_is_of_these_sources(path, key):
    with open(path) as f:
        record = json.load(f)[key]
    assert record["src_sha"] == bench.kernel_sources_sha(key.split("/")[0])


def test_default_line_has_its_records():
    assert bench.load_traffic("fused_stream_kernel", "oss20b_decode_w13_a6/with_align")[0] > 0
    assert bench.load_traffic("fused_mfma_kernel", "qwen3_prefill")[0] > 0
    assert bench.load_counters("fused_mfma_kernel", "qwen3_prefill")["mfma_util_pct"] > 0
