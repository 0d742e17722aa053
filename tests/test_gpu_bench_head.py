"""bench.py with the head's losses: as cases of --operators, and where the pass
of --prefetch turns."""
import json
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def run_bench(*args, timeout=110):
    print("[bench]", *args, flush=True)
    res = subprocess.run([sys.executable, os.path.join(ROOT, "bench.py"), *args], cwd=ROOT,
                         stdout=subprocess.PIPE, stderr=subprocess.PIPE, timeout=timeout)
    assert res.returncode == 0, res.stderr.decode()[-2000:]
    return json.loads(res.stdout.decode())


@pytest.mark.gpu
def test_cases_are_timed():
    d = run_bench("--operators", "score_few,distill_frozen,norm_few", "--steps", "3")
    assert list(d["cases"]) == ["score_few", "distill_frozen", "norm_few"]
    assert d["cases"]["score_few"]["TFLOPs"] > 0 and "TFLOPs" not in d["cases"]["norm_few"]


@pytest.mark.gpu
@pytest.mark.parametrize("head", [False, True])
def test_prefetch_with_the_head(head):
    d = run_bench("--prefetch", "--layers", "2", "--steps", "1", "--warmup", "1", "--tokens", "256",
                  "--depths", "1", *(["--head-loss"] if head else []))
    assert d["head"] == ([32000, 4096] if head else None)
    assert d["positions"] == 4 + head
    run = d["runs"][0]
    assert run["tokens"] == 256 and run["compute_ms"] > 0 and run["depth"]["1"]["ms"] > 0
