"""The workspace sizes that zsp.h states, against what the library says (host
only: a plan that is not bound counts as bound for all ranks)."""
import os
import re

import pytest

import zero_sharded_mixed_pad_amd as zsp
from zero_sharded_mixed_pad_amd import binding

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include",
                      "zsp.h")


def stated():
    """(least, per 512 elements, per rank, constant), in bytes, from the text."""
    with open(HEADER) as f:
        text = re.sub(r"\n \* +", " ", f.read())
    m = re.search(r"the larger of ([\d,]+) bytes and (\d+) \* \(E / 512\) \+ (\d+) \* nd \+ (\d+)",
                  text)
    assert m, "zsp.h does not state the workspace's size"
    return [int(x.replace(",", "")) for x in m.groups()]


def test_lists():
    assert binding.zsp_norm_workspace() == stated()[0]


@pytest.mark.parametrize("numels,nd", [
    ([5], 2), ([0], 3), ([1000 * 1003], 4), ([1 << 20, 77], 8), ([1], 256), ([4096 * 4096] * 3, 1),
    ([4096 * 11008 + 1, 3], 64), ([70001, 9, 12345], 256), ([1 << 31], 17)])
def test_plans(numels, nd):
    least, per, rank, const = stated()
    plan = zsp.partition(numels, nd)
    want = max(least, per * (nd * plan.S // 512) + rank * nd + const)
    assert binding.zsp_norm_workspace(plan.handle) == want
