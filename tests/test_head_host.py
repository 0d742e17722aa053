"""The losses over the head: what is refused before anything is launched, and
the workspace's size (host only)."""
import ctypes
import math

import pytest
import torch

import zero_sharded_mixed_pad_amd as zsp
from zero_sharded_mixed_pad_amd import binding

BASE = 1 << 40                 # addresses that are only compared
N, V, D, TOP = 10, 100, 64, 4
SIZE = {"hidden": N * D * 2, "head": V * D * 2, "target": N * 8, "index": N * TOP * 8,
        "logit": N * TOP * 4, "token_weight": N * 4, "loss": N * 4, "lse": N * 4,
        "grad_hidden": N * D * 2, "grad_head": V * D * 2}


def good(distill=False):
    a = {k: BASE + (i << 20) for i, k in enumerate(SIZE)}
    a.update(dtype=zsp.BF16, n=N, v=V, d=D, top=TOP, temperature=1.0, scale=1.0, ws=BASE + (64 << 20),
             ws_bytes=binding.zsp_head_workspace(N, V, D, torch.bfloat16, TOP if distill else 0))
    return a


def call(a, distill=False):
    head = [a["hidden"], a["head"], a["dtype"], a["n"], a["v"], a["d"]]
    tail = [a["token_weight"], a["scale"], a["loss"], a["lse"], a["grad_hidden"], a["grad_head"],
            a["ws"], a["ws_bytes"], None]
    if distill:
        return binding.lib.zsp_head_distill(*head, a["index"], a["logit"], a["top"],
                                            a["temperature"], *tail)
    return binding.lib.zsp_head_loss(*head, a["target"], *tail)


def refused(status, text, distill=False, **changes):
    a = good(distill)
    a.update(changes)
    assert call(a, distill) == status, zsp.last_error()
    assert text in zsp.last_error()


EINVAL, ERANGE = binding.EINVAL, binding.ERANGE


@pytest.mark.parametrize("distill", [False, True])
@pytest.mark.parametrize("status,text,changes", [
    (EINVAL, "bad dtype", dict(dtype=2)),
    (EINVAL, "n = -1", dict(n=-1)),
    (EINVAL, "v = 0", dict(v=0)),
    (EINVAL, "d = 0", dict(d=0)),
    (ERANGE, "too large", dict(n=(1 << 24) + 1)),
    (ERANGE, "too large", dict(n=(1 << 23) + 1)),
    (ERANGE, "n * d", dict(n=1 << 23, d=65536)),
    (ERANGE, "too large", dict(v=(1 << 22) + 1)),
    (ERANGE, "too large", dict(d=65537)),
    (EINVAL, "hidden is NULL", dict(hidden=None)),
    (EINVAL, "head is NULL", dict(head=None)),
    (EINVAL, "loss is NULL", dict(loss=None)),
    (EINVAL, "ws is NULL", dict(ws=None)),
    (EINVAL, "scale", dict(scale=math.inf)),
    (EINVAL, "scale", dict(scale=math.nan)),
    (EINVAL, "hidden is not aligned to 2", dict(hidden=BASE + 1)),
    (EINVAL, "head is not aligned to 2", dict(head=BASE + (1 << 20) + 3)),
    (EINVAL, "loss is not aligned to 4", dict(loss=BASE + (6 << 20) + 2)),
    (EINVAL, "ws is not aligned to 16", dict(ws=BASE + (64 << 20) + 8)),
    (ERANGE, "ws_bytes", dict(ws_bytes=100)),
    (EINVAL, "loss overlaps lse", dict(lse=BASE + (6 << 20) + 4 * (N - 1))),
    (EINVAL, "grad_hidden overlaps hidden", dict(grad_hidden=BASE)),
    (EINVAL, "grad_head overlaps head", dict(grad_head=BASE + (1 << 20) + 2 * (V * D - 1))),
    (EINVAL, "loss overlaps ws", dict(loss=BASE + (64 << 20))),
])
def test_refusals(distill, status, text, changes):
    if changes.get("head") and changes["head"] % 16:
        # a head off 16 bytes needs a larger workspace, which is checked first
        changes = dict(changes, ws_bytes=1 << 24)
    refused(status, text, distill, **changes)


@pytest.mark.parametrize("status,text,changes", [
    (EINVAL, "top = 0", dict(top=0)),
    (ERANGE, "too large", dict(top=1025)),
    (EINVAL, "index is NULL", dict(index=None)),
    (EINVAL, "logit is NULL", dict(logit=None)),
    (EINVAL, "temperature", dict(temperature=0.0)),
    (EINVAL, "temperature", dict(temperature=-1.0)),
    (EINVAL, "temperature", dict(temperature=math.nan)),
    (EINVAL, "temperature", dict(temperature=math.inf)),
    (EINVAL, "temperature", dict(temperature=1e-40)),
    (EINVAL, "scale", dict(scale=1e30, temperature=1e10)),
    (EINVAL, "index is not aligned to 8", dict(index=BASE + (3 << 20) + 4)),
])
def test_refusals_of_distillation(status, text, changes):
    refused(status, text, True, **changes)


def test_target_missing():
    refused(EINVAL, "target is NULL", target=None)


def test_a_head_off_alignment_needs_room_for_its_copy():
    ok = binding.zsp_head_workspace(N, V, D, torch.bfloat16)
    more = binding.zsp_head_workspace(N, V, D, torch.bfloat16, aligned=False)
    assert more >= ok + V * D * 2
    refused(ERANGE, "ws_bytes", head=BASE + (1 << 20) + 2, ws_bytes=ok)


def test_workspace_is_bounded():
    """The softmax kept at a time does not grow with the tokens."""
    size = lambda n: binding.zsp_head_workspace(n, 131072, 4096, torch.bfloat16)  # noqa: E731
    per_token = 4096 * 2 + 16                       # the copy of hidden, and a few words
    kept, acc, parts = (1 << 32) * 17 // 16, 131072 * 4096 * 4, 5 << 28
    assert size(1 << 20) < kept + acc + parts + (1 << 20) * (per_token + 8)
    assert size(1 << 20) - size(1 << 19) < (1 << 19) * (per_token + 8) + (1 << 29)
    none = binding.zsp_head_workspace(4096, 32000, 4096, torch.bfloat16, grad_hidden=False,
                                      grad_head=False)
    assert none < 4096 * 4096 * 2 + 4096 * 500 * 8 + (1 << 20)


@pytest.mark.parametrize("n,v,d,top,flags", [
    (-1, 1, 1, 0, 0), (1, 0, 1, 0, 0), (1, 1, 0, 0, 0), (1, 1, 1, -1, 0), (1, 1, 1, 0, 8),
    (1, 1, 1, 1025, 0)])
def test_workspace_refusals(n, v, d, top, flags):
    out = ctypes.c_int64()
    assert binding.lib.zsp_head_workspace(n, v, d, zsp.BF16, top, flags, ctypes.byref(out)) < 0
    assert binding.lib.zsp_head_workspace(1, 1, 1, zsp.BF16, 0, 0, None) == EINVAL


def test_binding_says_what_is_wrong():
    x, w = torch.zeros(3, 8), torch.zeros(5, 8)
    t, loss, ws = torch.zeros(3, dtype=torch.int64), torch.zeros(3), torch.zeros(4,
                                                                          dtype=torch.uint8)
    with pytest.raises(ValueError, match="hidden must be on the GPU"):
        zsp.head_loss(x, w, t, loss, ws)
    with pytest.raises(ValueError, match=r"hidden must be \[n, d\] and head \[v, d\]"):
        zsp.head_loss(x, w[:, :4], t, loss, ws)
    with pytest.raises(TypeError, match="loss must be a torch tensor"):
        zsp.head_loss(x, w, t, None, ws)
    with pytest.raises(TypeError, match="unsupported dtype"):
        zsp.head_loss(x.double(), w.double(), t, loss, ws)
    with pytest.raises(TypeError, match="unsupported dtype"):
        zsp.head_workspace(3, 5, 8, torch.float16, device="cpu")
