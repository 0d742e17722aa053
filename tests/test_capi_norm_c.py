"""Norm, clipping and clipped steps from plain C99 (tests/capi_norm.c, built
by __graft_entry__.build()): argument errors on the CPU; on the GPU the records
against 64-bit sums, and states and clipped tensors bit for bit against the
oracle."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
import __graft_entry__  # noqa: E402


def program():
    __graft_entry__.ensure_built()
    return __graft_entry__.CAPI_NORM


def test_argument_errors_from_c():
    res = subprocess.run([program(), "--host-only"], stdout=subprocess.PIPE,
                         stderr=subprocess.STDOUT, timeout=60)
    out = res.stdout.decode(errors="replace")
    assert res.returncode == 0 and "host checks ok" in out, out


@pytest.mark.gpu
def test_clipped_steps_from_c():
    print("[capi_norm] full run", flush=True)
    res = subprocess.run([program()], stdout=subprocess.PIPE, stderr=subprocess.STDOUT,
                         timeout=100)
    out = res.stdout.decode(errors="replace")
    assert res.returncode == 0 and "capi norm ok" in out, out
