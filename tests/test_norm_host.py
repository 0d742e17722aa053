"""Gradient norm and clipping, host side: workspace sizes, and argument
errors that come back as the documented status codes before anything touches
a device (there is none here)."""
import ctypes

import pytest

import zero_sharded_mixed_pad_amd as zsp
from zero_sharded_mixed_pad_amd import binding

lib = binding.lib
INF = float("inf")
GOOD = 0x1000          # a 16-byte aligned address that no call may follow
WS = 1 << 30


def arrays(ptrs, numels, dtypes):
    n = max(len(ptrs), 1)
    return ((ctypes.c_void_p * n)(*ptrs), (ctypes.c_int64 * n)(*numels),
            (ctypes.c_int32 * n)(*dtypes), len(ptrs))


def norm_many(a, kind=0, max_norm=INF, ws=GOOD, ws_bytes=WS, out=GOOD):
    return lib.zsp_norm_many(*a, kind, max_norm, ws, ws_bytes, out, None)


def test_workspace_sizes():
    lists = binding.zsp_norm_workspace()
    assert lists > 0 and lists % 8 == 0
    small = zsp.partition([5], 2)
    assert binding.zsp_norm_workspace(small.handle) >= lists
    big = zsp.partition([1 << 28, 77], 8)
    # a 64-bit partial for every 256 elements
    assert binding.zsp_norm_workspace(big.handle) >= (1 << 28) // 256 * 8
    assert lib.zsp_norm_workspace(None, None) == zsp.binding.EINVAL


BAD_LISTS = [
    (arrays([None], [4], [0]), zsp.binding.EINVAL),            # NULL tensor with elements
    (arrays([GOOD + 2], [4], [0]), zsp.binding.EINVAL),        # fp32 at 2 bytes
    (arrays([GOOD + 1], [4], [1]), zsp.binding.EINVAL),        # bf16 at 1 byte
    (arrays([GOOD], [-1], [0]), zsp.binding.EINVAL),
    (arrays([GOOD], [4], [2]), zsp.binding.EINVAL),            # no such type
    (arrays([GOOD], [4], [-1]), zsp.binding.EINVAL),
    (arrays([GOOD], [1 << 62], [0]), zsp.binding.ERANGE),
    (arrays([GOOD] * 3, [(1 << 63) - 1] * 3, [1] * 3), zsp.binding.ERANGE),
    ((None, None, None, 1), zsp.binding.EINVAL),
    ((None, None, None, -1), zsp.binding.EINVAL),
]


@pytest.mark.parametrize("i", range(len(BAD_LISTS)))
def test_bad_lists_are_refused(i):
    a, want = BAD_LISTS[i]
    assert norm_many(a) == want
    assert lib.zsp_clip_many(*a, GOOD, None) == want
    h = ctypes.c_void_p(7)
    assert lib.zsp_tensor_list_create(*a, None, ctypes.byref(h)) == want
    assert h.value is None
    assert zsp.last_error()


def test_bad_norm_arguments_are_refused():
    a = arrays([GOOD], [4], [0])
    E, R = zsp.binding.EINVAL, zsp.binding.ERANGE
    assert norm_many(a, kind=2) == E
    assert norm_many(a, kind=-1) == E
    assert norm_many(a, max_norm=-0.5) == E
    assert norm_many(a, max_norm=float("nan")) == E
    assert norm_many(a, ws=None) == E
    assert norm_many(a, ws=GOOD + 8) == E
    assert norm_many(a, ws_bytes=binding.zsp_norm_workspace() - 1) == R
    assert norm_many(a, ws_bytes=-1) == R
    assert norm_many(a, out=None) == E
    assert norm_many(a, out=GOOD + 8) == E
    assert lib.zsp_clip_many(*a, None, None) == E
    assert lib.zsp_clip_many(*a, GOOD + 4, None) == E
    assert lib.zsp_clip_combine(GOOD, -1, 0, INF, GOOD, None) == E
    assert lib.zsp_clip_combine(None, 1, 0, INF, GOOD, None) == E
    assert lib.zsp_clip_combine(GOOD + 8, 1, 0, INF, GOOD, None) == E
    assert lib.zsp_clip_combine(GOOD, 1, 3, INF, GOOD, None) == E
    assert lib.zsp_clip_combine(GOOD, 1, 0, -1.0, GOOD, None) == E
    assert lib.zsp_clip_combine(GOOD, 1, 0, INF, None, None) == E
    assert lib.zsp_tensor_list_create(*a, None, None) == E
    assert lib.zsp_tensor_list_norm(None, 0, INF, GOOD, WS, GOOD, None) == E
    assert lib.zsp_tensor_list_clip(None, GOOD, None) == E
    lib.zsp_tensor_list_destroy(None)


@pytest.mark.parametrize("ptrs,numels,dtypes", [
    ([GOOD, GOOD], [4, 4], [0, 0]),                      # the same tensor twice
    ([GOOD, GOOD + 12], [4, 4], [0, 0]),                 # one element shared
    ([GOOD + 64, GOOD, GOOD + 30], [4, 16, 1], [0, 1, 1]),   # inside another, out of order
])
def test_clip_refuses_tensors_that_overlap(ptrs, numels, dtypes):
    got = lib.zsp_clip_many(*arrays(ptrs, numels, dtypes), GOOD, None)
    assert got == zsp.binding.EINVAL and "overlap" in zsp.last_error()


def test_plan_calls_need_a_binding():
    plan = zsp.partition([100, 7], 4)
    h = plan.handle
    E, S = zsp.binding.EINVAL, zsp.binding.ESTATE
    g = (ctypes.c_void_p * 4)(*[GOOD] * 4)
    n = (0, INF, GOOD, WS, GOOD, None)
    hp = (1e-3, 0.9, 0.999, 1e-8, 1, None)
    assert lib.zsp_grad_norm(None, -1, *n) == E
    assert lib.zsp_grad_norm(h, -1, *n) == S
    assert lib.zsp_grad_norm_params(h, -1, 0, 1, *n) == S
    assert lib.zsp_reduce_shard_norm(None, -1, g, 0, 0, 0, *n) == E
    assert lib.zsp_reduce_shard_norm(h, -1, g, 0, 0, 0, *n) == S
    assert lib.zsp_reduce_shard_norm_params(h, -1, 0, 1, g, 0, 0, 0, *n) == S
    assert lib.zsp_reduce_norm(None, -1, g, 0, 0, 0, *n) == E
    assert lib.zsp_reduce_norm(h, -1, g, 0, 0, 0, *n) == S
    assert lib.zsp_adam_step_clip(None, -1, GOOD, *hp) == E
    assert lib.zsp_adam_step_clip(h, -1, GOOD, *hp) == S
    assert lib.zsp_adam_step_clip(h, -1, None, *hp) == E
    assert lib.zsp_adam_step_clip_params(h, -1, 0, 1, GOOD, *hp) == S
    assert lib.zsp_adam_step_clip_params(h, -1, 0, 1, GOOD + 4, *hp) == E
    assert lib.zsp_reduce_adam_step_clip(None, -1, g, 0, 0, 0, GOOD, *hp) == E
    assert lib.zsp_reduce_adam_step_clip(h, -1, g, 0, 0, 0, GOOD, *hp) == S
    assert lib.zsp_reduce_adam_step_clip(h, -1, g, 0, 0, 0, None, *hp) == E
    assert lib.zsp_reduce_adam_step_clip_params(h, -1, 0, 1, g, 0, 0, 0, GOOD, *hp) == S
