"""The losses over the head and their gradients against the definition in 64
bits, on the GPU.

Tolerances, derived before the first run. u = 2^-24 (fp32), b = 2^-8 (bf16):
half a step relative to the value.

 * A logit: a sum of d products in fp32, in any order: error at most
   d u sum|x w|; for fp32 operands the three planes add what is left out,
   below 2^-22 sum|x w|, and six sums instead of one: (6 d + 4) u sum|x w|.
   Multiplying by 1/T (rounded) adds 2 u |l|. Call it dl (largest of a row).
 * lse: dl, plus the relative error of a sum of exponentials: 2^-21 for each
   (hardware exp2 and the rounding of its argument, |x| log2(e) u <= 2^-19 for
   |x| <= 20, weighted by exp(x): below 2^-21 on the whole), 24 additions in
   fp32, plus one rounding of lse. So dl + 2^-19 + u |lse|.
 * loss: twice that (lse and the entry's logit), times T^2, and one rounding;
   the teacher's part is taken in 64 bits.
 * G (bf16): P is rounded once (b), G once more (b), the entries' own G once;
   p's relative error before that is dl + 2^-19 + 2^-21. |dG| <= (2 b + b^2 +
   dl + 2^-18) |G| + entry terms: an entry's G = c (p - q) has the error
   c p (dl + 2^-19) and one rounding. With e_G = 2 b + 2^-15 + dl:
   |dG| <= e_G |c| (p + q) elementwise, written E.
   fp32: e_G = 2^-17 + dl in place of it.
 * A gradient: |d(G W)| <= E |W| elementwise plus the sum's own error
   k u |G| |W| (6 k for planes) plus one rounding b |result| (u for fp32).
   In norms: ||E||_F ||W||_2 + ... : the second, sharper check.
"""
import math
import zlib

import pytest
import torch

import zero_sharded_mixed_pad_amd as zsp

pytestmark = pytest.mark.gpu

U, B = 2.0 ** -24, 2.0 ** -8
BF, F32 = torch.bfloat16, torch.float32


def dev():
    return torch.device("cuda:0")


def gen(*key):
    g = torch.Generator(device="cuda")
    g.manual_seed(zlib.crc32(repr(key).encode()))
    return g


def make(n, v, d, dtype, top=0, seed=0):
    """Inputs whose logits spread by about 2 and lean to their target."""
    g = gen(n, v, d, top, seed, dtype == BF)
    w = (torch.randn(v, d, device=dev(), generator=g) * (2.0 / math.sqrt(d))).to(dtype)
    t = torch.randint(0, v, (n,), device=dev(), generator=g)
    x = torch.randn(n, d, device=dev(), generator=g)
    if n:
        x = x + w[t].float() * torch.rand(n, 1, device=dev(), generator=g) * 3.0
    x = x.to(dtype)
    if not top:
        return x, w, t, None
    idx = torch.randint(0, v, (n, top), device=dev(), generator=g)
    if n:
        idx[:, 0] = t
    return x, w, idx, torch.randn(n, top, device=dev(), generator=g) * 3.0


class Ref:
    """Everything in 64 bits, and the tolerances of the docstring."""

    def __init__(self, x, w, index, logit=None, T=1.0, weight=None, scale=1.0):
        n, v = x.shape[0], w.shape[0]
        f32 = x.dtype == F32
        d = x.shape[1]
        idx = index if logit is not None else index[:, None]
        ok = (idx >= 0) & (idx < v)
        if logit is not None:
            ok &= logit != -math.inf
        on = ok.any(1)
        if weight is not None:
            on &= weight != 0
        self.on = on
        T = float(torch.tensor(T, dtype=F32))
        scale = float(torch.tensor(scale, dtype=F32))
        X = torch.where(on[:, None], x.double(), 0.0)
        W = w.double()
        ok &= on[:, None]
        at = torch.where(ok, idx, 0)
        l = (X @ W.t()) / T
        absl = (X.abs() @ W.abs().t()) / T
        dl = (6 * d + 4 if f32 else d) * U * absl + 2 * U * l.abs()
        dl = dl.max(1).values
        lse = torch.logsumexp(l, 1)
        if logit is None:
            q = ok.double()
            logq = torch.zeros_like(q)
        else:
            t = torch.where(ok, logit.double() / T, -math.inf)
            logq = torch.where(on[:, None], torch.log_softmax(torch.where(on[:, None], t, 0.0), 1), -math.inf)
            q = torch.where(ok, logq.exp(), 0.0)
        term = torch.where(ok & (q > 0), q * (logq - (l.gather(1, at) - lse[:, None])), 0.0)
        z = torch.zeros_like(lse)
        self.lse = torch.where(on, lse, z)
        self.loss = torch.where(on, T * T * term.sum(1), z)
        self.tol_lse = torch.where(on, dl + 2.0 ** -19 + U * lse.abs(), z)
        self.tol_loss = torch.where(on, T * T * (2 * dl + 2.0 ** -18) + 2 * U * self.loss.abs()
                                    + 2.0 ** -40, z)
        p = torch.exp(l - lse[:, None])
        c = torch.where(on, scale * T, z)
        if weight is not None:
            c = torch.where(on, c * weight.double(), z)
        Q = torch.zeros_like(p).scatter_add_(1, at, q)
        G = c[:, None] * (p - Q)
        eG = (2.0 ** -17 if f32 else 2 * B + 2.0 ** -15) + dl
        E = (eG * c.abs())[:, None] * (p + Q)
        out = U if f32 else B
        six = 6 if f32 else 1

        def grad(g, e, m):
            ref = g @ m
            tol = (e + six * g.shape[1] * U * g.abs()) @ m.abs() + out * ref.abs() + 2.0 ** -60
            small = m if m.shape[0] < m.shape[1] else m.t()
            two = (torch.linalg.eigvalsh((small @ small.t()).cpu()).max().clamp_min(0).sqrt().to(dev())
                   if min(m.shape) else 0.0)
            norm = (float(torch.linalg.norm(e + six * math.sqrt(g.shape[1]) * U * g.abs()) * two)
                    + out * float(torch.linalg.norm(ref)) + 2.0 ** -60)
            return ref, tol, norm

        self.gx = grad(G, E, W)
        self.gw = grad(G.t().contiguous(), E.t().contiguous(), X)
        self.gx = (torch.where(on[:, None], self.gx[0], 0.0),) + self.gx[1:]


def call(x, w, index, logit=None, T=1.0, weight=None, scale=1.0, want="both", lse=True, ws=None,
         stream=None, fill=float("nan")):
    """Runs the operator into outputs that hold `fill`; the workspace holds NaN."""
    n, v, d = x.shape[0], w.shape[0], x.shape[1]
    new = lambda *s, t=F32: torch.full(s, fill, dtype=t, device=dev())  # noqa: E731
    loss, ls = new(n), new(n) if lse else None
    gx = new(n, d, t=x.dtype) if want in ("both", "hidden") else None
    gw = new(v, d, t=x.dtype) if want in ("both", "head") else None
    if ws is None:
        ws = zsp.head_workspace(n, v, d, x.dtype, top=0 if logit is None else index.shape[1],
                                grad_hidden=gx is not None, grad_head=gw is not None,
                                aligned=w.data_ptr() % 16 == 0)
        ws.fill_(255)
    more = dict(token_weight=weight, scale=scale, lse=ls, grad_hidden=gx, grad_head=gw,
                stream=stream)
    if logit is None:
        zsp.head_loss(x, w, index, loss, ws, **more)
    else:
        zsp.head_distill(x, w, index, logit, loss, ws, temperature=T, **more)
    return loss, ls, gx, gw


def check(out, r):
    loss, lse, gx, gw = out

    def near(got, want, tol, what):
        err = (got.double() - want).abs()
        bad = ~(err <= tol)
        assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, first "
                               f"{bad.nonzero()[0].tolist()}: {got[bad][0].item()} for "
                               f"{want[bad][0].item()}, tolerance {tol[bad][0].item()}")

    near(loss, r.loss, r.tol_loss, "loss")
    if lse is not None:
        near(lse, r.lse, r.tol_lse, "lse")
    for got, (want, tol, norm), what in ((gx, r.gx, "grad_hidden"), (gw, r.gw, "grad_head")):
        if got is not None:
            near(got, want, tol, what)
            far = float(torch.linalg.norm(got.double() - want))
            assert far <= norm, f"{what}: {far} from the definition, {norm} allowed"
    if gx is not None:
        assert not gx[~r.on].any()          # exactly 0
    assert not loss[~r.on].any()


SHAPES = [(1, 1, 1), (1, 7, 3), (3, 64, 64), (5, 65, 40), (16, 256, 64), (31, 257, 128),
          (64, 1000, 72), (129, 1000, 1003), (200, 511, 192), (300, 4099, 320), (1, 5000, 512),
          (700, 130, 256), (2, 3, 1000), (1025, 777, 64), (2500, 130, 72), (40, 9000, 256),
          (20000, 70, 24), (64, 8192, 1000), (65, 8193, 1000), (1500, 93, 4416)]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("n,v,d", SHAPES)
def test_loss(n, v, d, dtype):
    x, w, t, _ = make(n, v, d, dtype)
    check(call(x, w, t, scale=0.37), Ref(x, w, t, scale=0.37))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("top,T", [(1, 1.0), (3, 2.0), (8, 0.5), (64, 1.5), (130, 4.0), (1024, 2.0)])
@pytest.mark.parametrize("n,v,d", [(1, 1, 1), (7, 300, 64), (70, 1029, 200), (260, 2000, 128)])
def test_distill(n, v, d, top, T, dtype):
    x, w, idx, lg = make(n, v, d, dtype, top)      # indices may occur twice
    check(call(x, w, idx, lg, T, scale=0.37), Ref(x, w, idx, lg, T, scale=0.37))


@pytest.mark.parametrize("top", [0, 40])
@pytest.mark.parametrize("want", ["hidden", "both"])
@pytest.mark.parametrize("n,v,d", [(40, 9001, 512), (100, 9001, 512), (129, 9001, 1024),
                                   (200, 9100, 1000), (256, 8321, 640), (200, 4000, 328)])
def test_few_tokens(n, v, d, want, top):
    """Forms that read the head once, kept in the caches (its gradient not
    asked for) or not, some of whose tokens do not count."""
    x, w, t, lg = make(n, v, d, BF, top)
    t[5::9] = -1
    x[5::9] = float("nan")
    check(call(x, w, t, lg, 2.0 if top else 1.0, want=want), Ref(x, w, t, lg, 2.0 if top else 1.0))


@pytest.mark.parametrize("want", ["none", "hidden", "head"])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("top", [0, 5])
def test_what_is_not_asked_for(top, dtype, want):
    x, w, t, lg = make(100, 700, 128, dtype, top)
    out = call(x, w, t, lg, want=want, lse=want == "head")
    check(out, Ref(x, w, t, lg))
    full = call(x, w, t, lg)
    for a, b in zip(out, full):
        assert a is None or torch.equal(a, b)


def masks(n, kind, g):
    on = torch.ones(n, dtype=torch.bool, device=dev())
    if kind == "none":
        on[:] = False
    elif kind == "last":
        on[:-1] = False
    elif kind == "first":
        on[1:] = False
    elif kind == "half":
        on = torch.rand(n, device=dev(), generator=g) < 0.5
    elif kind == "prompt":
        on[: n // 3] = False
    return on


@pytest.mark.parametrize("kind", ["none", "first", "last", "half", "prompt"])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), torch.finfo(F32).min])
def test_tokens_that_do_not_count(kind, dtype, bad):
    """Their rows of hidden may hold anything."""
    n, v, d = 333, 900, 128
    x, w, t, _ = make(n, v, d, dtype)
    on = masks(n, kind, gen(kind))
    t = torch.where(on, t, torch.tensor([-100, -1, v, v + 5, 1 << 40], device=dev())[
        torch.arange(n, device=dev()) % 5])
    x[~on] = bad
    check(call(x, w, t), Ref(x, w, t))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("top", [0, 6])
def test_weights(top, dtype):
    """Of either sign, and 0: such a token does not count."""
    n, v, d = 500, 640, 192
    x, w, t, lg = make(n, v, d, dtype, top)
    tw = torch.randn(n, device=dev(), generator=gen("w"))
    tw[::7] = 0.0
    x[::7] = float("nan")
    check(call(x, w, t, lg, 2.0 if top else 1.0, tw, 0.01),
          Ref(x, w, t, lg, 2.0 if top else 1.0, tw, 0.01))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_teacher_entries(dtype):
    """Entries left out (whatever their logits), -infinity, the same index
    several times, tokens with one entry and with none."""
    n, v, d, k = 64, 300, 64, 12
    x, w, idx, lg = make(n, v, d, dtype, k)
    idx[0:8, 3:] = -1
    lg[0:8, 3:] = float("nan")
    idx[8:16, 5] = v
    lg[8:16, 5] = float("inf")
    idx[16:24] = idx[16:24, :1]                 # all the same
    lg[24:32, 1:] = -math.inf                   # one left
    lg[32:36] = -math.inf                       # none left
    idx[36:40] = -7
    lg[40:44] = torch.finfo(F32).min            # all equal, at the lowest value
    idx[44:48, 1::2] = idx[44:48, 0::2]         # each twice
    check(call(x, w, idx, lg, 1.5), Ref(x, w, idx, lg, 1.5))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_sure_of_the_target(dtype):
    """Where p of the target is nearly 1, its own gradient keeps 1 - p."""
    n, v, d = 40, 500, 256
    x, w, t, _ = make(n, v, d, dtype)
    x = (w[t].float() * torch.linspace(2, 8, n, device=dev())[:, None]).to(dtype)
    r = Ref(x, w, t)
    out = call(x, w, t)
    check(out, r)
    assert float(r.loss.min()) < 1e-6 < float(r.loss.max())


@pytest.mark.parametrize("big", [50.0, 2000.0])
def test_wide_logits(big):
    """Logits thousands apart: no overflow, zeros where p is nothing."""
    n, v, d = 30, 400, 64
    x, w, t, _ = make(n, v, d, F32)
    x = x * big
    check(call(x, w, t), Ref(x, w, t))


def test_not_finite():
    """NaN and infinity in a token's own row stay in that row of grad_hidden."""
    n, v, d = 20, 300, 64
    x, w, t, _ = make(n, v, d, BF)
    x[3, 5] = float("nan")
    loss, lse, gx, gw = call(x, w, t)
    assert loss[3].isnan() and lse[3].isnan() and gx[3].isnan().all()
    keep = [i for i in range(n) if i != 3]
    r = Ref(x[keep], w, t[keep])
    check((loss[keep], lse[keep], gx[keep], None), r)
    assert gw.isnan().any()


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("off", [1, 3, 4])
def test_views_off_alignment(dtype, off):
    """Head and gradients as views that start on any element; what lies
    around them stays."""
    n, v, d = 90, 333, 128
    x, w, t, _ = make(n, v, d, dtype)

    def view(rows):
        buf = torch.full((rows * d + 16,), 7.0, dtype=dtype, device=dev())
        return buf, buf[off:off + rows * d].view(rows, d)

    _, wv = view(v)
    wv.copy_(w)
    _, xv = view(n)
    xv.copy_(x)
    bx, gx = view(n)
    bw, gw = view(v)
    loss = torch.empty(n, device=dev())
    ws = zsp.head_workspace(n, v, d, dtype, aligned=False)
    zsp.head_loss(xv, wv, t, loss, ws, grad_hidden=gx, grad_head=gw)
    check((loss, None, gx, gw), Ref(x, w, t))
    for b, rows in ((bx, n), (bw, v)):
        assert (b[:off] == 7).all() and (b[off + rows * d:] == 7).all()


def test_no_tokens():
    w = torch.randn(70, 64, device=dev(), dtype=BF)
    x, t = torch.empty(0, 64, device=dev(), dtype=BF), torch.empty(0, device=dev(),
                                                                    dtype=torch.int64)
    _, _, gx, gw = call(x, w, t)
    assert gx.shape == (0, 64) and not gw.any()


def test_equal_inputs_give_equal_bits():
    x, w, t, _ = make(700, 3001, 320, BF)
    a, b = call(x, w, t), call(x, w, t, fill=3.0)
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_differences():
    """The gradients against central differences of the loss itself (fp32)."""
    n, v, d = 12, 90, 64
    x, w, t, _ = make(n, v, d, F32)
    tw = torch.rand(n, device=dev(), generator=gen("d")) + 0.5
    _, _, gx, gw = call(x, w, t, weight=tw, scale=0.5)
    g = gen("dir")
    for what, grad in (("hidden", gx), ("head", gw)):
        v_ = torch.randn(grad.shape, device=dev(), generator=g)
        h = 2.0 ** -6

        def at(s):
            xs, ws_ = (x + s * v_, w) if what == "hidden" else (x, w + s * v_)
            loss = call(xs, ws_, t, want="none")[0]
            return float((loss.double() * tw.double()).sum() * 0.5)

        # the difference's error: the third derivative times h^2 / 6 and the
        # losses' rounding over 2 h. Third derivatives of a log-sum-exp along v
        # are at most max|v . w|^3 a token, taken here from 64 bits.
        z = (v_.double() @ w.double().t() if what == "hidden" else x.double() @ v_.double().t())
        third = 2 * (z.abs().max(1).values + z.abs().max()) ** 3
        tol = (float((third * tw.double()).sum()) * 0.5 * h * h / 6
               + float(Ref(x, w, t).tol_loss.sum()) / h)
        got = (at(h) - at(-h)) / (2 * h)
        want = float((grad.double() * v_.double()).sum())
        assert abs(got - want) <= tol, (what, got, want, tol)


@pytest.mark.parametrize("n,v,d,dtype,top", [
    (5, 9000, 256, BF, 0),        # few tokens
    (100, 9000, 256, BF, 6),
    (180, 9000, 1024, BF, 3),
    (9, 9000, 256, F32, 0),       # an fp32 head read in place
    (50, 700, 1000, F32, 4),      # the same, logits in parts
    (40, 500, 333, BF, 0),        # the head copied, logits in parts
    (600, 3000, 128, F32, 0),
])
def test_forms_replayed(n, v, d, dtype, top):
    """Each form captured on a side stream and replayed over other inputs, a
    workspace full of NaN each time, eager work of its own between."""
    sets = [make(n, v, d, dtype, top, seed) for seed in range(2)]
    T = 1.5 if top else 1.0
    live = [None if s is None else s.clone() for s in sets[0]]
    want = [[o.clone() for o in call(*s, T)] for s in sets]
    out = [torch.zeros_like(o) for o in want[0]]
    ws = zsp.head_workspace(n, v, d, dtype, top=top)
    st = torch.cuda.Stream()

    def run():
        more = dict(lse=out[1], grad_hidden=out[2], grad_head=out[3], stream=st)
        if top:
            zsp.head_distill(*live, out[0], ws, temperature=T, **more)
        else:
            zsp.head_loss(*live[:3], out[0], ws, **more)

    torch.cuda.synchronize()
    run()
    st.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        run()
    for k in (1, 0, 1):
        for a, b in zip(live, sets[k]):
            if a is not None:
                a.copy_(b)
        for o in out:
            o.fill_(float("nan"))
        ws.fill_(255)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want[k]):
            assert torch.equal(a, b)
        call(*sets[0], T)


def test_two_streams_at_once():
    """Two calls in flight together, each with a workspace of its own."""
    sets = [make(700, 5000, 256, BF, 0, s) for s in range(2)]
    want = [call(*s) for s in sets]
    ws = [zsp.head_workspace(700, 5000, 256, BF) for _ in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(4):
        for i, s in enumerate(sets):
            with torch.cuda.stream(streams[i]):
                got[i].append(call(*s, ws=ws[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for out in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(out, want[i]))


def test_binding_refuses():
    x, w, t, _ = make(10, 70, 64, BF)
    loss, ws = torch.empty(10, device=dev()), zsp.head_workspace(10, 70, 64, BF)
    ok = lambda **k: zsp.head_loss(**{**dict(hidden=x, head=w, target=t, loss=loss, ws=ws), **k})  # noqa: E731
    ok()
    wide = torch.empty(10, 128, device=dev(), dtype=BF)
    for bad, error, text in (
            (dict(hidden=wide[:, ::2]), ValueError, "hidden must be contiguous"),
            (dict(target=t.int()), TypeError, "target must be torch.int64"),
            (dict(target=t[:9]), ValueError, "target must have shape"),
            (dict(loss=loss.double()), TypeError, "loss must be torch.float32"),
            (dict(lse=loss[:9]), ValueError, "lse must have shape"),
            (dict(head=w.float()), TypeError, "head must be torch.bfloat16"),
            (dict(grad_hidden=x.float()), TypeError, "grad_hidden must be torch.bfloat16"),
            (dict(grad_head=w[:69].clone()), ValueError, "grad_head must have shape"),
            (dict(token_weight=loss.to(BF)), TypeError, "token_weight must be torch.float32"),
            (dict(ws=ws.float()), TypeError, "ws must be torch.uint8")):
        with pytest.raises(error, match=text):
            ok(**bad)
    for bad in (dict(ws=ws[:256]), dict(lse=loss), dict(grad_hidden=x), dict(scale=float("nan"))):
        with pytest.raises(zsp.ZspError):
            ok(**bad)


def test_on_another_stream_and_replayed():
    """A captured call, replayed over new inputs with eager work between."""
    n, v, d = 260, 1100, 192
    sets = [make(n, v, d, BF, 4, seed) for seed in range(3)]
    x, w, idx, lg = (s.clone() for s in sets[0])
    want = [[o.clone() for o in call(*s, 2.0)] for s in sets]
    loss, lse = torch.zeros(n, device=dev()), torch.zeros(n, device=dev())
    gx, gw = torch.zeros_like(x), torch.zeros_like(w)
    ws = zsp.head_workspace(n, v, d, BF, top=4)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()

    def run():
        zsp.head_distill(x, w, idx, lg, loss, ws, temperature=2.0, lse=lse, grad_hidden=gx,
                         grad_head=gw, stream=st)

    run()
    st.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        run()
    for k in (1, 2, 0, 1):
        for a, b in zip((x, w, idx, lg), sets[k]):
            a.copy_(b)
        for o in (loss, lse, gx, gw):
            o.fill_(float("nan"))
        ws.fill_(255)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((loss, lse, gx, gw), want[k]):
            assert torch.equal(a, b)
        call(*sets[0], 2.0)


@pytest.mark.parametrize("n,dtype,top", [(2200, BF, 0), (2200, BF, 3), (900, F32, 0)])
def test_more_tokens_than_are_kept_at_a_time(n, dtype, top):
    """2^20 columns by so many tokens are more than 4 GiB of P: chunks, the
    head's gradient summed over them in fp32."""
    v, d = 1 << 20, 64
    x, w, t, lg = make(n, v, d, dtype, top)
    t[::5] = -100
    loss, lse, gx, gw = call(x, w, t, lg)
    idx = t if top else t[:, None]
    ok = idx >= 0
    on = ok.any(1)
    l = x.double() @ w.double().t()
    ref = torch.logsumexp(l, 1)
    assert float(((lse.double() - ref) * on).abs().max()) < 2.0 ** -16
    at = idx.clamp_min(0)
    q = torch.softmax(torch.where(ok & on[:, None], lg.double(), -1e300), 1) if top else ok.double()
    q = torch.where(ok, q, 0.0)
    terms = torch.where(q > 0, q * (q.clamp_min(1e-300).log() - l.gather(1, at) + ref[:, None]), 0)
    assert float((loss.double() - terms.sum(1) * on).abs().max()) < 2.0 ** -15
    l.sub_(ref[:, None]).exp_()
    l.scatter_add_(1, at, -q)
    l[~on] = 0
    far = 3 * B if dtype == BF else 2.0 ** -15
    for got, want in ((gx, l @ w.double()), (gw, l.t() @ x.double())):
        e = torch.linalg.norm(got.double() - want) / torch.linalg.norm(want)
        assert float(e) < far, float(e)


def test_rows_of_the_softmax_past_31_bits():
    """A tile's last row of P starts more than 2^31 bytes behind its first."""
    n, v, d = 300, (1 << 22), 16
    x, w, t, _ = make(n, v, d, BF)
    t[7] = v - 1
    loss, lse, gx, gw = call(x, w, t)
    l = x.double() @ w.double().t()
    ref = torch.logsumexp(l, 1)
    assert float((lse.double() - ref).abs().max()) < 2.0 ** -16
    assert float((loss.double() - ref + l.gather(1, t[:, None])[:, 0]).abs().max()) < 2.0 ** -15
    l.sub_(ref[:, None]).exp_()
    l[torch.arange(n), t] -= 1
    for got, want in ((gx, l @ w.double()), (gw, l.t() @ x.double())):
        e = torch.linalg.norm(got.double() - want) / torch.linalg.norm(want)
        assert float(e) < 3 * B, float(e)


def test_offsets_past_32_bits():
    """A head and its gradient of more than 2^32 elements."""
    n, v, d = 5, (1 << 20) + 77, 4160
    w = torch.empty(v, d, device=dev(), dtype=BF).normal_(0, 0.02, generator=gen("big"))
    x = torch.randn(n, d, device=dev(), generator=gen("x")).to(BF)
    t = torch.tensor([0, v - 1, v - 2, 5, v // 2], device=dev())
    loss, lse, gx, gw = call(x, w, t)
    l = torch.cat([x.double() @ p.double().t() for p in w.split(1 << 16)], 1)
    ref = torch.logsumexp(l, 1)
    assert float((lse.double() - ref).abs().max()) < 2.0 ** -15
    G = torch.exp(l - ref[:, None])
    G[torch.arange(n), t] -= 1
    for a in (0, (1 << 20) - 100):
        want = G[:, a:a + 177].t() @ x.double()
        far = torch.linalg.norm(gw[a:a + 177].double() - want) / torch.linalg.norm(want)
        assert float(far) < 3 * B
    want = sum(G[:, i:i + (1 << 16)] @ w[i:i + (1 << 16)].double() for i in range(0, v, 1 << 16))
    assert float(torch.linalg.norm(gx.double() - want) / torch.linalg.norm(want)) < 3 * B


@pytest.mark.parametrize("nd", [4, 3])
def test_in_a_step(nd):
    """The head gathered from its shards, every rank's loss writing its
    gradient of the head where the reduce reads it (off alignment), then the
    reduce with the norm and the clipped update, against the same made of the
    definition's gradients."""
    v, d, n = 211, 64, 75
    numel = [37, v * d, 5]
    plan = zsp.partition(numel, nd)
    N = nd * plan.S
    master, m, vv = (torch.empty(N, device=dev()) for _ in range(3))
    work, acc = torch.empty(N, dtype=BF, device=dev()), torch.empty(N, device=dev())
    plan.bind_state(zsp.ALL_RANKS, master, m, vv, work, acc)
    flat = (torch.randn(sum(numel), device=dev(), generator=gen("p")) * 0.2).to(BF)
    plan.load_params(flat)
    head = torch.empty(v * d, dtype=BF, device=dev())
    plan.gather(1, head)
    head = head.view(v, d)
    off = plan.tensor(1)["full_off"]
    grads = [torch.zeros(plan.total_padded, dtype=BF, device=dev()) for _ in range(nd)]
    ws = zsp.head_workspace(n, v, d, BF)
    total = torch.zeros(v, d, dtype=torch.float64, device=dev())
    tol = torch.zeros(v, d, dtype=torch.float64, device=dev())
    for r in range(nd):
        x, _, t, _ = make(n, v, d, BF, seed=r)
        loss = torch.empty(n, device=dev())
        gw = grads[r][off:off + v * d].view(v, d)
        zsp.head_loss(x, head, t, loss, ws, scale=1.0 / (n * nd), grad_head=gw)
        ref = Ref(x, head, t, scale=1.0 / (n * nd))
        check((loss, None, None, gw), ref)
        total += ref.gw[0]
        tol += ref.gw[1]
    clip, nws = zsp.clip_record(), plan.norm_workspace()
    plan.reduce_shard_norm(zsp.ALL_RANKS, grads, clip, nws, max_norm=1e-3)
    got = torch.empty(v * d, device=dev())
    plan.gather(1, got, "acc")
    err = (got.view(v, d).double() - total).abs()
    assert bool((err <= tol + nd * U * total.abs()).all())
    before = master.clone()
    plan.adam_step_clip(zsp.ALL_RANKS, clip, lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, step=1)
    norm = float(zsp.clip_values(clip)[1])
    assert abs(norm - float(torch.linalg.norm(got.double()))) <= 4 * U * norm
    assert not torch.equal(before, master)
