"""bench.py's reading of profiler output: names for the kernels of the head's
losses, from mangled and demangled symbols."""
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
import bench  # noqa: E402


def demangled(kernel, args):
    inner = ", ".join({True: "true", False: "false"}.get(a, str(a)) if isinstance(a, bool)
                      else str(a) for a in args)
    return f"void zsp::(anonymous namespace)::{kernel}_kernel<{inner}>(zsp::(anonymous namespace)::Args)"


def mangled(kernel, args):
    inner = "".join(f"L{'b' if isinstance(a, bool) else 'i'}{int(a)}E" for a in args)
    return f"_ZN3zsp12_GLOBAL__N_1{len(kernel) + 7}{kernel}_kernelI{inner}EEvNS0_4ArgsE"


@pytest.mark.parametrize("kernel,args,name", [
    ("gemm", (256, 256, 4, 2, 2, False, False, False, False, 0), "head_logits_256x256[bf16]"),
    ("gemm", (128, 64, 2, 2, 6, True, False, False, True, 0), "head_logits_128x64[f32]"),
    ("gemm", (128, 128, 2, 2, 4, True, False, False, False, 1), "head_logit_parts_128x128[bf16]"),
    ("gemm", (256, 256, 4, 2, 2, False, True, False, False, 1), "head_grad_hidden_256x256[bf16]"),
    ("gemm", (256, 256, 4, 2, 2, False, True, True, True, 1), "head_grad_head_256x256[f32]"),
    ("thin", (2, False, 0), "head_logits_in_place_32[f32]"),
    ("thin", (4, True, 1), "head_grad_hidden_in_place_64[f32]"),
    ("outer", (3,), "head_grad_head_96_tokens[bf16]"),
    ("join", (False,), "head_join[bf16]"),
    ("raw_join", (True,), "head_raw_join[f32]"),
    ("split", (True,), "head_split[f32]"),
])
def test_head_kernels_are_named(kernel, args, name):
    assert bench._short(demangled(kernel, args)) == name
    assert bench._short(mangled(kernel, args)) == name


@pytest.mark.parametrize("kernel", ["setup", "scan", "flag"])
def test_kernels_without_sizes_are_named(kernel):
    assert bench._short(f"zsp::(anonymous namespace)::{kernel}_kernel(zsp::Args)") == f"head_{kernel}"


def test_other_libraries_keep_their_names():
    assert bench._short("void at::native::scan_kernel<int>(x)") == "at::native::scan_kernel<int>(x)"
