"""bench.py --operators: cases of perf/operators.py through the library."""
import json
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def run_bench(*args, timeout=110):
    return subprocess.run([sys.executable, os.path.join(ROOT, "bench.py"), *args], cwd=ROOT,
                          stdout=subprocess.PIPE, stderr=subprocess.PIPE, timeout=timeout)


@pytest.mark.gpu
def test_cases_are_timed():
    print("[bench] --operators norm_few,step_one", flush=True)
    res = run_bench("--operators", "norm_few,step_one", "--steps", "5")
    assert res.returncode == 0, res.stderr.decode()[-2000:]
    d = json.loads(res.stdout.decode())
    assert d["mode"] == "operators" and list(d["cases"]) == ["norm_few", "step_one"]
    for c in d["cases"].values():
        assert 0 < c["host_us"] <= c["us_per_pass"] and c["bytes"] > 0


@pytest.mark.gpu
def test_an_unknown_case_is_refused():
    res = run_bench("--operators", "no_such_case")
    assert res.returncode != 0 and b"unknown case no_such_case" in res.stderr
