"""The gradients of the losses over the head against differences of the loss,
in directions in which it changes, on the GPU.

 * Of the loss in 64 bits, from its definition alone: central differences at h
   and 2h, h = 2^-10, extrapolated: off by h^4 / 30 times a fifth derivative
   and 2^-52 / h of the sum, below 2^-20 of the derivative. The directions move
   every token away from its target (hidden along -w_target, head's row of the
   target along -x): a derivative of about (1 - p) |w|^2 a token.
   The gradient itself may be off as its G may, |dG| <= e c (p + q) with e =
   2^-8 + 2^-10 + dl for bf16 and 2^-16 + dl for fp32 (dl: a logit's error, d u
   sum|x w|, six times that and 4 u more for fp32), and rounds its result.
 * Of the operator's own losses (fp32): (f(h) - f(-h)) / 2h, h = 2^-3, is off
   by h^2 / 6 times the third derivative, the third central moment of z = dl/ds
   under p, taken at seven points of [-h, h] and twice over, and by the losses'
   rounding over h.
Each tolerance has to be below a tenth of the derivative, so that a gradient of
zeros and one of the wrong sign are told from the right one.
"""
import pytest
import torch

import zero_sharded_mixed_pad_amd as zsp

pytestmark = pytest.mark.gpu

U, B = 2.0 ** -24, 2.0 ** -8
BF, F32 = torch.bfloat16, torch.float32


def make(n, v, d, dtype, top, device="cuda"):
    """Inputs from the CPU's generator, so that what is said of their
    derivatives can be looked at there."""
    g = torch.Generator().manual_seed(n * 7919 + v * 31 + d + top)
    w = (torch.randn(v, d, generator=g) * 2.0 * d ** -0.5).to(dtype)
    first = torch.randint(0, v, (n,), generator=g)
    x = (torch.randn(n, d, generator=g) + w[first].float() * torch.rand(n, 1, generator=g) * 2.0).to(dtype)
    weight = torch.rand(n, generator=g) + 0.5
    if not top:
        return [t.to(device) for t in (x, w, first)] + [None, weight.to(device)]
    index = torch.randint(0, v, (n, top), generator=g)
    index[:, 0] = first
    logit = torch.randn(n, top, generator=g)
    logit[:, 0] += 3.0
    return [t.to(device) for t in (x, w, index, logit, weight)]


def losses(x, w, index, logit, T):
    """Of the definition, in 64 bits."""
    logp = torch.log_softmax(x.double() @ w.double().t().contiguous() / T, 1)
    if logit is None:
        return -logp.gather(1, index[:, None])[:, 0]
    logq = torch.log_softmax(logit.double() / T, 1)
    return T * T * (logq.exp() * (logq - logp.gather(1, index))).sum(1)


def gradients(x, w, index, logit, T, weight, scale):
    (n, d), v = x.shape, w.shape[0]
    loss, gx, gw = torch.empty(n, device="cuda"), torch.empty_like(x), torch.empty_like(w)
    ws = zsp.head_workspace(n, v, d, x.dtype, top=0 if logit is None else index.shape[1])
    more = dict(token_weight=weight, scale=scale, grad_hidden=gx, grad_head=gw)
    if logit is None:
        zsp.head_loss(x, w, index, loss, ws, **more)
    else:
        zsp.head_distill(x, w, index, logit, loss, ws, temperature=T, **more)
    return loss, gx, gw


def directions(x, w, index, logit):
    first = index if logit is None else index[:, 0]
    return -w.double()[first], torch.zeros_like(w, dtype=torch.float64).index_add_(0, first, -x.double())


def difference(x, w, index, logit, T, weight, scale, dx, dw):
    """The derivative of the sum of losses along (dx, dw)."""
    def f(s):
        moved = losses(x.double() + s * dx, w.double() + s * dw, index, logit, T)
        return float((weight.double() * moved).sum()) * scale
    h = 2.0 ** -10
    return (8 * (f(h) - f(-h)) - (f(2 * h) - f(-2 * h))) / (12 * h)


def tolerance(x, w, index, logit, T, weight, scale, dx, dw, want):
    X, W, f32 = x.double(), w.double(), x.dtype == F32
    d = x.shape[1]
    p = torch.softmax(X @ W.t().contiguous() / T, 1)
    if logit is None:
        p = p.scatter_add(1, index[:, None], torch.ones_like(p[:, :1]))
    else:
        p = p.scatter_add(1, index, torch.softmax(logit.double() / T, 1))
    dl = ((6 * d + 4 if f32 else d) + 2) * U * (X.abs() @ W.abs().t().contiguous()).max() / T
    e = (2.0 ** -16 if f32 else B + 2.0 ** -10) + dl
    E = e * scale * T * weight.double()[:, None] * p
    out = U if f32 else B
    gx, gw = E @ W.abs(), E.t().contiguous() @ X.abs()
    return float((gx * dx.abs()).sum() + (gw * dw.abs()).sum()) * (1 + out / e) + 2.0 ** -20 * abs(want)


CASES = [(12, 90, 64, F32, 0, 1.0), (70, 90, 64, F32, 3, 2.0), (64, 700, 1024, F32, 0, 1.0),
         (600, 3000, 129, F32, 4, 1.5), (30, 9000, 256, F32, 0, 1.0), (64, 700, 1024, BF, 0, 1.0),
         (5, 9001, 256, BF, 0, 1.0), (100, 9001, 256, BF, 4, 2.0), (200, 9100, 512, BF, 0, 1.0),
         (1500, 9100, 320, BF, 5, 1.5), (700, 130, 256, BF, 0, 1.0)]


@pytest.mark.parametrize("n,v,d,dtype,top,T", CASES)
def test_gradients_along_the_loss(n, v, d, dtype, top, T):
    x, w, index, logit, weight = make(n, v, d, dtype, top)
    scale = 0.25
    _, gx, gw = gradients(x, w, index, logit, T, weight, scale)
    for what, grad, keep in (("hidden", gx, (1, 0)), ("head", gw, (0, 1))):
        dx, dw = (k * t for k, t in zip(keep, directions(x, w, index, logit)))
        want = difference(x, w, index, logit, T, weight, scale, dx, dw)
        tol = tolerance(x, w, index, logit, T, weight, scale, dx, dw, want)
        got = float((grad.double() * (dx if what == "hidden" else dw)).sum())
        assert tol < 0.1 * want, (what, want, tol)
        assert abs(got - want) <= tol, (what, got, want, tol)


@pytest.mark.parametrize("n,v,d,top,T", [(12, 90, 16, 0, 1.0), (70, 90, 16, 0, 1.0), (12, 9000, 16, 5, 2.0),
                                         (70, 9000, 17, 4, 1.0)])
def test_gradients_along_the_operators_own_losses(n, v, d, top, T):
    x, w, index, logit, weight = make(n, v, d, F32, top)
    scale, h = 0.25, 2.0 ** -3
    _, gx, gw = gradients(x, w, index, logit, T, weight, scale)
    for what, grad, keep in (("hidden", gx, (1, 0)), ("head", gw, (0, 1))):
        dx, dw = (k * t for k, t in zip(keep, directions(x, w, index, logit)))
        dx, dw = dx / w.double().norm(dim=1).mean(), dw / x.double().norm(dim=1).mean()
        side = [gradients((x + s * dx).float(), (w + s * dw).float(), index, logit, T, weight, scale)[0]
                for s in (h, -h)]
        got = float((weight.double() * (side[0].double() - side[1].double())).sum()) * scale / (2 * h)
        z = (dx @ w.double().t().contiguous() + x.double() @ dw.t().contiguous()) / T
        third = torch.zeros(n, device="cuda", dtype=torch.float64)
        for s in torch.linspace(-h, h, 7).tolist():
            p = torch.softmax((x + s * dx) @ (w + s * dw).t().contiguous() / T, 1)
            mean = (p * z).sum(1, keepdim=True)
            third = torch.maximum(third, 2 * T * T * (p * (z - mean) ** 3).sum(1).abs())
        # the losses' rounding: two logits and lse, and what moving x and w in fp32 leaves
        moved = (x.double().abs() + h * dx.abs()) @ (w.double().abs() + h * dw.abs()).t().contiguous()
        dl = (6 * d + 12) * U * moved.max(1).values / T
        one = T * T * (2 * dl + 2.0 ** -18) + 4 * U * side[0].double().abs()
        tol = float((weight.double() * (third * h * h / 6 + one / h)).sum()) * scale
        want = float((grad.double() * (dx if what == "hidden" else dw)).sum())
        assert tol < 0.1 * got, (what, got, want, tol)
        assert abs(got - want) <= tol, (what, got, want, tol)
