"""bench.py's reading of profiler output: a name of its own for every op of
the shard kernel, as zsp_internal.hpp numbers them, and for the other kernels."""
import os
import re
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
import bench  # noqa: E402

CSRC = os.path.join(ROOT, "zero_sharded_mixed_pad_amd", "csrc")


def shard_ops():
    with open(os.path.join(CSRC, "zsp_internal.hpp"), encoding="utf-8") as f:
        body = re.search(r"enum ShardOp[^{]*\{(.*?)\};", f.read(), re.S).group(1)
    return {int(v): n for n, v in re.findall(r"(OP_\w+) = (\d+)", body)}


def demangled(op, t):
    return (f"void zsp::(anonymous namespace)::shard_kernel<{op}, {t}, 8, 2, false>"
            "(zsp::(anonymous namespace)::ShardArgs<8>)")


def mangled(op, t):
    return f"_ZN3zsp12_GLOBAL__N_112shard_kernelILi{op}E{t}Li8ELi2ELb0EEEvNS0_9ShardArgsIXT1_EEE"


def test_shard_ops_are_named():
    ops = shard_ops()
    assert len(ops) == 13 and ops[12] == "OP_ADAM_CLIP"
    names = {}
    for op in ops:
        for form, f32, bf16 in ((demangled, "float", "unsigned short"), (mangled, "f", "t")):
            for t, dt in ((f32, "f32"), (bf16, "bf16")):
                got = bench._short(form(op, t))
                assert got.endswith(f"[{dt}]"), (op, got)
                assert names.setdefault(got, op) == op, got
    assert len(names) == 2 * len(ops)
    assert bench._short(demangled(1, "float")) == "reduce_set[f32]"
    assert bench._short(mangled(4, "t")) == "fused_reduce_adam_cast_acc[bf16]"


def test_every_header_of_the_kernels_is_in_their_hash():
    """Stored counters count as current while the kernels' code is the same:
    all of it, the headers that zsp_kernels.hip includes among it."""
    with open(os.path.join(CSRC, "zsp_kernels.hip"), encoding="utf-8") as f:
        heads = re.findall(r'#include "(zsp_\w+\.hpp)"', f.read())
    assert "zsp_internal.hpp" in heads
    for h in heads:
        assert f"zero_sharded_mixed_pad_amd/csrc/{h}" in bench.KERNEL_SOURCES, h


@pytest.mark.parametrize("kernel", ["acc_norm", "list_norm", "list_clip", "finish", "fold",
                                    "combine"])
def test_norm_kernels_are_named(kernel):
    form = f"void zsp::(anonymous namespace)::{kernel}_kernel<0, false>(zsp::Args)"
    assert bench._short(form) == kernel
    assert bench._short(f"_ZN3zsp12_GLOBAL__N_1{len(kernel) + 7}{kernel}_kernelILi0EEEvv") == kernel
