"""The losses over the head: bounds of their arguments, and what a workspace
serves (host only)."""
import random
import time

import pytest
import torch

import zero_sharded_mixed_pad_amd as zsp
from zero_sharded_mixed_pad_amd import binding

BASE = 1 << 40                 # addresses that are only compared
EINVAL, ERANGE = binding.EINVAL, binding.ERANGE


def call(n, v, d, dtype, top=0, ws_bytes=None, grads=(True, True), temperature=1.0, bad=True):
    """The status of a call with good arguments but, where `bad`, the last that
    is looked at: a loss off its alignment, refused with EINVAL if all others
    (the workspace's size among them) are taken."""
    size = 2 if dtype == torch.bfloat16 else 4
    code = zsp.BF16 if size == 2 else zsp.F32
    if ws_bytes is None:
        ws_bytes = binding.zsp_head_workspace(n, v, d, dtype, top, *grads)
    at, step = {}, BASE
    for name, nbytes in (("hidden", n * d * size), ("head", v * d * size), ("index", n * max(top, 1) * 8),
                         ("logit", n * top * 4), ("loss", n * 4), ("grad_hidden", n * d * size),
                         ("grad_head", v * d * size), ("ws", ws_bytes)):
        at[name] = step
        step += (nbytes + 4096) // 4096 * 4096
    at["loss"] += 2 * bad
    head = [at["hidden"], at["head"], code, n, v, d]
    tail = [None, 1.0, at["loss"], None, at["grad_hidden"] if grads[0] else None,
            at["grad_head"] if grads[1] else None, at["ws"], ws_bytes, None]
    if top:
        return binding.lib.zsp_head_distill(*head, at["index"], at["logit"], top, temperature, *tail)
    return binding.lib.zsp_head_loss(*head, at["index"], *tail)


def test_temperature_whose_exponents_are_not_finite():
    """1 / 3.5e-39 is finite, log2(e) times that is not: every p would be NaN."""
    assert call(10, 100, 64, torch.bfloat16, 4, temperature=3.5e-39) == EINVAL
    assert "temperature" in zsp.last_error()
    assert call(10, 100, 64, torch.bfloat16, 4, temperature=4.3e-39) == EINVAL
    assert "loss is not aligned" in zsp.last_error()


def test_what_is_kept_of_the_largest_vocabulary():
    """The softmax takes 10 bytes a column in fp32, 2 in bf16, and partials an
    eighth of a byte a column: of up to 64 tokens 64 rows are kept, of more what
    4 GiB hold and 256 rows at least."""
    v, d = 1 << 22, 16
    planes, acc, small = v * 64 * 2 * 3, v * 64 * 4, 1 << 26
    size = lambda n, dt: binding.zsp_head_workspace(n, v, d, dt)  # noqa: E731
    for n in (1, 17, 64):
        assert size(n, torch.float32) < 64 * v * 10.125 + small
        assert size(n, torch.bfloat16) < 64 * v * 2.125 + small
    for n in (65, 256, 300, 5000):
        assert size(n, torch.float32) < 256 * v * 10.125 + planes + acc + small
        assert size(n, torch.bfloat16) < (1 << 32) * 2.125 / 2 + acc + small


@pytest.mark.parametrize("n,v,d,dtype", [(1 << 23, 64, 64, torch.bfloat16), (1 << 22, 256, 2048, torch.bfloat16),
                                         (1 << 23, 64, 1024, torch.float32)])
def test_a_call_of_many_tokens_plans_in_a_moment(n, v, d, dtype):
    """Parts of sums for every number of tokens that may count are bounded
    without trying each (which took 4 to 8 ms here)."""
    ws_bytes, least = binding.zsp_head_workspace(n, v, d, dtype), 1.0
    for _ in range(5):
        t0 = time.perf_counter()
        assert call(n, v, d, dtype, ws_bytes=ws_bytes) == EINVAL
        least = min(least, time.perf_counter() - t0)
    assert "loss is not aligned" in zsp.last_error()
    assert least < 1.5e-3, least


SERVED = [(300, 32000, 4096, torch.bfloat16, 0), (130, 32000, 4096, torch.bfloat16, 0),
          (8457, 50257, 2048, torch.float32, 0), (70000, 32000, 64, torch.bfloat16, 0),
          (200, 1000, 1003, torch.float32, 5), (400, 6000, 4096, torch.bfloat16, 0),
          (2000, 130, 512, torch.float32, 1), (64, 5000, 2048, torch.float32, 0),
          (3000, 1 << 20, 128, torch.bfloat16, 8), (90000, 256, 8192, torch.bfloat16, 0)]


@pytest.mark.parametrize("n,v,d,dtype,top", SERVED)
@pytest.mark.parametrize("grads", [(True, True), (True, False), (False, False)])
def test_a_workspace_serves_fewer_tokens(n, v, d, dtype, top, grads):
    """One sized for the largest batch takes every smaller one, also where its
    sums are cut into more parts or its chunks are larger."""
    ws_bytes = binding.zsp_head_workspace(n, v, d, dtype, top, *grads)
    near = [m + o for m in (64, 128, 192, 256, 512, n // 2, n // 3) for o in (-1, 0, 1)]
    for m in sorted({1, 16, 17, 32, 33, *near, *range(1, n, max(1, n // 400)), n}):
        if m <= n:
            assert call(m, v, d, dtype, top, ws_bytes, grads) == EINVAL
            assert "loss is not aligned" in zsp.last_error(), (m, zsp.last_error())
            assert binding.zsp_head_workspace(m, v, d, dtype, top, *grads) <= ws_bytes


def test_workspaces_serve_fewer_tokens_whatever_the_sizes():
    rng = random.Random(11)
    log = lambda lo, hi: int(2 ** rng.uniform(lo, hi))  # noqa: E731
    for _ in range(4000):
        n, v, d = log(0, 18), log(0, 20), log(0, 13)
        dtype = rng.choice([torch.bfloat16, torch.float32])
        top, grads = rng.choice([0, 0, 3]), (rng.random() < 0.7, rng.random() < 0.7)
        # of a head that may start anywhere: then too where it does not
        ws_bytes = binding.zsp_head_workspace(n, v, d, dtype, top, *grads, aligned=rng.random() < 0.7)
        for m in {rng.randint(1, n), log(0, n.bit_length()) % n + 1, n}:
            assert call(m, v, d, dtype, top, ws_bytes, grads) == EINVAL
            assert "loss is not aligned" in zsp.last_error(), (n, m, v, d, dtype, top, grads)


@pytest.mark.parametrize("n,v,d,dtype,top", [(773670, 897009, 68, torch.float32, 0), (3404901, 3013938, 4, torch.bfloat16, 0),
                                             (130039, 848989, 193, torch.float32, 3), (4096, 32000, 4096, torch.bfloat16, 64),
                                             (61, 1000, 1003, torch.float32, 1)])
def test_a_workspace_serves_fewer_gradients_and_entries(n, v, d, dtype, top):
    """A training step's serves an evaluation: losses alone may keep more tokens
    at a time."""
    ws_bytes = binding.zsp_head_workspace(n, v, d, dtype, top)
    for grads in ((True, True), (True, False), (False, True), (False, False)):
        for k in sorted({0, min(1, top), top // 2, top}):
            assert call(n, v, d, dtype, k, ws_bytes, grads) == EINVAL
            assert "loss is not aligned" in zsp.last_error(), (grads, k, zsp.last_error())
