"""How often the gradients of the losses over the head round, element by
element, on the GPU.

hidden holds rows of the identity and head the logits: l_iv = head[v, i]
exactly, and column i of grad_head is G_i = c_i (p_i - q_i) itself, through no
other sum. u = 2^-24 (fp32), b = 2^-8 (bf16): half a step relative to the value.

 * bf16: p comes to G with a relative error of at most e = 2^-11: it is held
   as (m - l) log2(e) in steps of 64 / 65535 (half a step: 3.4e-4), and 1e-6
   for exponentials and their arguments; below 2^-63.9 of its block's largest
   as 0. G is rounded once:
   |dG| <= b |g| + (1 + b) (e c p + 2^-63.9 c).
 * fp32: logits l - m are exact where they have a common size, |l - m| <= 24;
   exponentials are off by |x| log2(e) u + 2^-22 <= 2^-18 relative, their sum
   as much at most: |dG| <= 2^-17 c p + 2 u |g|.
"""
import zlib

import pytest
import torch

import zero_sharded_mixed_pad_amd as zsp

pytestmark = pytest.mark.gpu

U, B = 2.0 ** -24, 2.0 ** -8
BF, F32 = torch.bfloat16, torch.float32


def gen(*key):
    g = torch.Generator(device="cuda")
    g.manual_seed(zlib.crc32(repr(key).encode()))
    return g


def columns_of_g(head, index, logit, T, weight, n, want="both"):
    """G of `n` tokens over head [v, d], whose rows of hidden are e_0, e_1, ..."""
    v, d = head.shape
    x = torch.eye(d, device="cuda", dtype=head.dtype)[:n].contiguous()
    loss, lse = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    gx = torch.empty_like(x) if want == "both" else None
    gw = torch.full((v, d), float("nan"), dtype=head.dtype, device="cuda")
    ws = zsp.head_workspace(n, v, d, head.dtype, top=0 if logit is None else index.shape[1],
                            grad_hidden=gx is not None)
    ws.fill_(255)
    more = dict(token_weight=weight, scale=1.0 / T, lse=lse, grad_hidden=gx, grad_head=gw)
    if logit is None:
        zsp.head_loss(x, head, index, loss, ws, **more)
    else:
        zsp.head_distill(x, head, index, logit, loss, ws, temperature=T, **more)
    assert not gw[:, n:].any()              # no token's
    return gw[:, :n].t().double(), lse.double()


def definition(head, index, logit, T, weight, n):
    l = head.double().t()[:n] / T
    lse = torch.logsumexp(l, 1)
    p = torch.exp(l - lse[:, None])
    c = torch.ones(n, device="cuda", dtype=torch.float64) if weight is None else weight.double()
    q = torch.zeros_like(p)
    if logit is None:
        q[torch.arange(n, device="cuda"), index] = 1.0
    else:
        q.scatter_add_(1, index, torch.softmax(logit.double() / T, 1))
    return c[:, None] * (p - q), c[:, None].abs() * p, lse


def within(got, want, tol, what):
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()}, first "
                           f"{bad.nonzero()[0].tolist()}: {got[bad][0].item()} for "
                           f"{want[bad][0].item()}, tolerance {tol[bad][0].item()}")


@pytest.mark.parametrize("top,T", [(0, 1.0), (6, 2.0)])
@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("n,v,d", [(5, 9001, 64), (64, 9001, 64), (100, 9001, 128), (200, 9100, 256),
                                   (320, 9100, 320), (300, 40000, 320), (64, 1000, 64),
                                   (64, 1000, 1024)])
def test_bf16_gradient_is_rounded_once(n, v, d, weighted, top, T):
    g = gen(n, v, d, top)
    head = (torch.randn(v, d, device="cuda", generator=g) * 2.0).to(BF)
    weight = torch.rand(n, device="cuda", generator=g) + 0.3 if weighted else None
    index = torch.randint(0, v, (n,) if not top else (n, top), device="cuda", generator=g)
    logit = torch.randn(n, top, device="cuda", generator=g) if top else None
    got, _ = columns_of_g(head, index, logit, T, weight, n)
    want, cp, _ = definition(head, index, logit, T, weight, n)
    c = 1.0 if weight is None else weight.double()[:, None]
    tol = B * want.abs() + (1 + B) * (2.0 ** -11 * cp + 2.0 ** -63.9 * c)
    within(got, want, tol, "G")


@pytest.mark.parametrize("v,d", [(9001, 64), (700, 64), (700, 1024)])
def test_bf16_gradient_of_logits_far_apart(v, d):
    """Logits from 0 to 120 below a block's largest: what lies past the steps
    is 0, not something small."""
    n = 64
    g = gen(v, d)
    head = (-120.0 * torch.rand(v, d, device="cuda", generator=g)).to(BF)
    index = torch.randint(0, v, (n,), device="cuda", generator=g)
    got, _ = columns_of_g(head, index, None, 1.0, None, n)
    want, cp, _ = definition(head, index, None, 1.0, None, n)
    within(got, want, B * want.abs() + (1 + B) * (2.0 ** -11 * cp + 2.0 ** -63.9), "G")


@pytest.mark.parametrize("top", [0, 5])
@pytest.mark.parametrize("n,v,d", [(16, 9000, 64), (64, 9001, 64), (67, 9001, 67), (300, 9001, 320),
                                   (64, 700, 1024), (40, 5000, 1001)])
def test_fp32_gradient_of_large_logits(n, v, d, top):
    """An lse of about 3000 costs p nothing: it depends on l - lse."""
    g = gen(n, v, d, top, "large")
    head = 3000.0 + 2.0 * torch.randn(v, d, device="cuda", generator=g)
    index = torch.randint(0, v, (n,) if not top else (n, top), device="cuda", generator=g)
    logit = torch.randn(n, top, device="cuda", generator=g) if top else None
    got, lse = columns_of_g(head, index, logit, 1.0, None, n)
    want, cp, ref = definition(head, index, logit, 1.0, None, n)
    within(got, want, 2.0 ** -17 * cp + 2 * U * want.abs(), "G")
    within(lse, ref, 2.0 ** -18 + U * ref, "lse")


def test_bf16_gradient_is_rounded_once_over_chunks():
    """2^22 columns: 512 tokens at a time, the head's gradient summed over two
    chunks in fp32. A few tokens of either."""
    n = d = 600
    v = 1 << 22
    g = gen("chunks")
    head = torch.empty(v, d, device="cuda", dtype=BF).normal_(0.0, 2.0, generator=g)
    index = torch.randint(0, v, (n,), device="cuda", generator=g)
    x = torch.eye(d, device="cuda", dtype=BF)
    loss, gw = torch.empty(n, device="cuda"), torch.full_like(head, float("nan"))
    zsp.head_loss(x, head, index, loss, zsp.head_workspace(n, v, d, BF, grad_hidden=False), grad_head=gw)
    for i in (0, 300, 511, 512, 599):
        l = head[:, i].double()
        p = torch.softmax(l, 0)
        want = p.clone()
        want[index[i]] -= 1.0
        tol = B * want.abs() + (1 + B) * (2.0 ** -11 * p + 2.0 ** -63.9)
        within(gw[:, i].double(), want, tol, f"G of token {i}")


@pytest.mark.parametrize("T", [0.7, 3.0])
@pytest.mark.parametrize("n,v,d", [(16, 9000, 64), (67, 9001, 67), (300, 9001, 320), (64, 700, 1024)])
def test_fp32_gradient_of_large_logits_at_a_temperature(n, v, d, T):
    """l / T is not rounded to fp32 before its difference from lse is taken:
    |l - m| / T log2(e) <= 40 leaves 40 u + 2^-22 of p."""
    g = gen(n, v, d, "T")
    head = 3000.0 + 2.0 * torch.randn(v, d, device="cuda", generator=g)
    index = torch.randint(0, v, (n, 5), device="cuda", generator=g)
    logit = torch.randn(n, 5, device="cuda", generator=g)
    T32 = float(torch.tensor(T))
    got, lse = columns_of_g(head, index, logit, T32, None, n)
    want, cp, ref = definition(head, index, logit, T32, None, n)
    # scale * T: 1 / T and its product with T round once each
    within(got, want, 2.0 ** -17 * cp + 5 * U * want.abs(), "G")
    within(lse, ref, 2.0 ** -18 + U * ref, "lse")
