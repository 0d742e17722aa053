"""Every entry point that README.md names is in zsp.h and in the binding."""
import os
import re

from zero_sharded_mixed_pad_amd import binding

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def read(*path):
    with open(os.path.join(ROOT, *path)) as f:
        return f.read()


def promised():
    """Names in the first cells of the table of entry points; "(and `_params`)"
    promises the _params form of each name before it, back to a semicolon."""
    names = set()
    for line in read("README.md").splitlines():
        if not line.startswith("| `zsp_"):
            continue
        for group in line.split("|")[1].split(";"):
            for part in re.split(r"(\(and `_params`\))", group):
                if part.startswith("(and"):
                    names |= {n + "_params" for n in last}
                    continue
                last = re.findall(r"`(zsp_\w+)`", part)
                names |= set(last)
    return names


def test_entry_points_of_the_readme_exist():
    names = promised()
    assert {"zsp_partition", "zsp_grad_norm_params", "zsp_reduce_norm"} <= names
    header = read("include", "zsp.h")
    for n in sorted(names):
        assert re.search(rf"\b{n}\(", header), f"{n} is not in zsp.h"
        assert hasattr(binding.lib, n), f"libzsp has no {n}"
