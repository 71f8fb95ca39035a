"""The committed counter records of the prefill GEMM belong to the present GEMM sources (bench.py leaves them out of its
line otherwise), without a GPU."""
import json
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
import bench  # noqa: E402


@pytest.mark.parametrize("record", [bench.TRAFFIC_RECORD, bench.MFMA_RECORD])
def test_records_are_of_the_present_sources(record):
    rec = json.load(open(record))
    assert rec["source_hash"] == bench.source_hash(bench.GEMM_SOURCES)
    assert rec["source_hash"] in open(os.path.splitext(record)[0] + ".md").read()


def test_the_bench_line_has_them():
    rec = bench.mfma_record()
    assert rec is not None and 0 < rec["mfma_busy_frac"] < 1
