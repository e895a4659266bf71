"""bench.py prints one JSON line on standard output, short enough to be read back from the end of a log."""
import ast
import json
import os

import bench

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LONG = {"sweep", "routing_overhead", "configs"}


def test_details_do_not_share_the_line(capsys):
    bench.emit({"metric": bench.METRIC, "value": 1.0}, {k: list(range(10000)) for k in LONG})
    out, err = capsys.readouterr()
    assert json.loads(out)["value"] == 1.0 and out.count("\n") == 1
    assert set(json.loads(err)["details"]) == LONG


def test_the_result_line_holds_no_sweep():
    """The keys of the result that main() prints: none of the lists that grow with the configurations, and every one that a
    reader of the line relies on."""
    tree = ast.parse(open(os.path.join(ROOT, "bench.py")).read())
    main = next(n for n in tree.body if isinstance(n, ast.FunctionDef) and n.name == "main")
    line = next(n.value for n in ast.walk(main) if isinstance(n, ast.Assign) and getattr(n.targets[0], "id", "") == "line")
    keys = {k.value for k in line.keys}
    assert not keys & LONG
    assert {"metric", "value", "unit", "n_gpus", "steps", "warmup", "ms_per_step", "higher_is_better", "scaling", "vs_baseline",
            "dtype", "data", "config", "e2e", "gpu_launches", "clocks"} <= keys
