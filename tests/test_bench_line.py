"""The benchmark's result line: one short line on standard output, the table of
the other workloads apart from it."""
import io
import json

import bench


def test_the_table_stays_out_of_the_result_line():
    configs = [{"workload": "w" * 100, "fused_us": 1.0, "n": i} for i in range(200)]
    line = {"metric": bench.METRIC, "value": 2.5, "configs": configs, "clocks": {"sm_mhz": 2070}}
    out, err = io.StringIO(), io.StringIO()
    bench.emit(line, out, err)
    (result,), (table,) = out.getvalue().splitlines(), err.getvalue().splitlines()
    assert json.loads(result) == {k: v for k, v in line.items() if k != "configs"}
    assert len(result) < 1000 and json.loads(table) == {"configs": configs}
    assert line["configs"] is configs                     # the caller's stays whole


def test_no_table_no_second_line():
    out, err = io.StringIO(), io.StringIO()
    bench.emit({"value": 1.0, "configs": None}, out, err)
    assert json.loads(out.getvalue()) == {"value": 1.0} and err.getvalue() == ""
