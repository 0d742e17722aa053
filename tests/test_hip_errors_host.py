"""An error that a call has reported is not reported again by the next one
(tests/hip_errors.c, with a runtime of its own that fails on demand)."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
import __graft_entry__  # noqa: E402


def test_a_reported_error_is_cleared(tmp_path):
    __graft_entry__.ensure_built()
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    lib = os.path.join(ROOT, "zero_sharded_mixed_pad_amd")
    exe = str(tmp_path / "hip_errors")
    subprocess.run(["gcc", "-std=c99", "-O1", "-Wall", "-Wextra", "-Werror", "-rdynamic",
                    "-I", os.path.join(ROOT, "include"), "-I", os.path.join(rocm, "include"),
                    os.path.join(ROOT, "tests", "hip_errors.c"), "-o", exe,
                    "-L", lib, "-lzsp", "-L", os.path.join(rocm, "lib"), "-lamdhip64",
                    f"-Wl,-rpath,{lib}", "-Wl,-rpath," + os.path.join(rocm, "lib")], check=True)
    res = subprocess.run([exe], stdout=subprocess.PIPE, stderr=subprocess.STDOUT, timeout=60)
    out = res.stdout.decode(errors="replace")
    assert res.returncode == 0 and "hip errors ok" in out, out
