"""A whole step from the losses over the head, on the GPU: the head gathered
from its shards, every rank's loss writing its gradient where the reduce reads
it, the reduce with the norm, and the clipped update, against the same made in
64 bits from the definition's gradients.

eps is 1 and the clipped gradient small, so that the update lr g / (|g| + eps)
goes by the gradient's size. A rank's gradient of the head may be off by e |x|
summed over c (p + q), e = 2^-8 + 2^-10 + dl (bf16; dl, a logit's error, d u
sum|x w|), and one rounding 2^-8 of itself; the sum over ranks by u for each;
the coefficient by as much of itself as the gradient's norm; the update, whose
derivative by g is at most lr / eps, by 16 roundings to fp32 of itself and one
of the parameter.
"""
import pytest
import torch

import zero_sharded_mixed_pad_amd as zsp

pytestmark = pytest.mark.gpu

U, B = 2.0 ** -24, 2.0 ** -8
BF = torch.bfloat16
V, D, N = 211, 64, 75
LR, EPS, MAX_NORM = 1e3, 1.0, 1e-3


def parameters(device="cuda"):
    g = torch.Generator().manual_seed(3)
    return (torch.randn(37 + V * D + 5, generator=g) * 0.2).to(BF).to(device)


def batch(rank, head, device="cuda"):
    g = torch.Generator().manual_seed(100 + rank)
    t = torch.randint(0, V, (N,), generator=g)
    x = torch.randn(N, D, generator=g) + head.float().cpu()[t] * torch.rand(N, 1, generator=g) * 3.0
    t[rank::9] = -100
    return x.to(BF).to(device), t.to(device)


def gradient(x, head, target, scale):
    """Of the head, in 64 bits, and what the operator's may be off."""
    on = target >= 0
    X, W = x.double()[on], head.double()
    l = X @ W.t().contiguous()
    p = torch.softmax(l, 1)
    q = torch.zeros_like(p).scatter_(1, target[on][:, None], 1.0)
    dl = (D + 2) * U * (X.abs() @ W.abs().t().contiguous()).max()
    e = B + 2.0 ** -10 + dl
    want = scale * (p - q).t().contiguous() @ X
    return want, e * scale * (p + q).t().contiguous() @ X.abs() + B * want.abs()


def update(total, tol, master):
    """The clipped step's change of the head's parameters, and its tolerance."""
    norm = torch.linalg.norm(total)
    assert norm > 10 * MAX_NORM
    coef = MAX_NORM / norm
    off = torch.linalg.norm(tol) / norm
    g, dg = total * coef, tol * coef
    dg = (dg + g.abs() * off) * (1 + 2 * off)
    step = LR * g / (g.abs() + EPS)
    return step, LR / EPS * dg + 16 * U * step.abs() + U * master.abs()


def definition(nd, head, device="cuda"):
    total = torch.zeros(V, D, dtype=torch.float64, device=device)
    tol = torch.zeros_like(total)
    for r in range(nd):
        x, t = batch(r, head, device)
        want, off = gradient(x, head, t, 1.0 / (N * nd))
        total += want
        tol += off + nd * U * want.abs()
    return total, tol


@pytest.mark.parametrize("nd", [4, 3])
def test_clipped_step_from_the_losses(nd):
    numel = [37, V * D, 5]
    plan = zsp.partition(numel, nd)
    n = nd * plan.S
    master, m, v = (torch.empty(n, device="cuda") for _ in range(3))
    work, acc = torch.empty(n, dtype=BF, device="cuda"), torch.empty(n, device="cuda")
    plan.bind_state(zsp.ALL_RANKS, master, m, v, work, acc)
    plan.load_params(parameters())

    def full(t, source, dtype=torch.float32):
        out = torch.empty(numel[t], dtype=dtype, device="cuda")
        plan.gather(t, out, source)
        return out

    head = full(1, "work", BF).view(V, D)
    before = [full(t, "master") for t in range(3)]
    off = plan.tensor(1)["full_off"]
    grads = [torch.zeros(plan.total_padded, dtype=BF, device="cuda") for _ in range(nd)]
    ws = zsp.head_workspace(N, V, D, BF)
    for r in range(nd):
        x, t = batch(r, head)
        zsp.head_loss(x, head, t, torch.empty(N, device="cuda"), ws, scale=1.0 / (N * nd),
                      grad_head=grads[r][off:off + V * D].view(V, D))
    clip = zsp.clip_record()
    plan.reduce_shard_norm(zsp.ALL_RANKS, grads, clip, plan.norm_workspace(), max_norm=MAX_NORM)
    plan.adam_step_clip(zsp.ALL_RANKS, clip, lr=LR, beta1=0.9, beta2=0.999, eps=EPS, step=1)

    total, tol = definition(nd, head)
    norm = float(torch.linalg.norm(total))
    assert abs(float(zsp.clip_values(clip)[1]) - norm) <= float(torch.linalg.norm(tol)) + 4 * U * norm
    after = [full(t, "master") for t in range(3)]
    step, allowed = update(total, tol, before[1].double().view(V, D))
    moved = (before[1].double() - after[1].double()).view(V, D)
    assert bool(((moved - step).abs() <= allowed).all())
    assert float(torch.linalg.norm(allowed)) < 0.1 * float(torch.linalg.norm(step))
    for t in (0, 2):                       # their gradients are 0
        assert torch.equal(before[t], after[t])
    for t in range(3):
        assert after[t].isfinite().all()
        assert torch.equal(full(t, "work", BF), after[t].to(BF))
