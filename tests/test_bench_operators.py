"""CPU checks of the row-wise operators' table in bench.py."""

import pytest

import bench
from perf import operators as P


def test_limits():
    pk = {"hbm": 5000.0, "bf16": 1000.0}
    cases = {c["name"]: c for c in P.listed()}
    # 51200 x 2304 bf16: x, the stream and its sum, y; the weights
    c = cases["norm anchor"]
    assert bench.operator_limit(c, P.work(c), pk) == pytest.approx((4 * 51200 * 2304 * 2 + 4 * 2304) / 5e6)
    # 2 M K N at four times the bf16 rate; the bytes of a few rows
    c = cases["qkv anchor nvfp4"]
    assert bench.operator_limit(c, P.work(c), pk) == pytest.approx(2 * 51200 * 2304 * 6912 / 4e9)
    c = cases["modulation mxfp4"]
    assert bench.operator_limit(c, P.work(c), pk) == pytest.approx(P.work(c)["bytes"] / 5e6)
    assert bench.operator_limit(dict(c, fmt="mxfp8"), {"bytes": 1, "flops": 4e9}, pk) == pytest.approx(2.0)
    assert set(bench.MX_RATE) == set(P.BLOCK)
