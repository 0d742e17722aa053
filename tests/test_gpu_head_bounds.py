"""The losses over the head keep to their workspace and outputs, on the GPU."""
import zlib

import pytest
import torch

import zero_sharded_mixed_pad_amd as zsp
from zero_sharded_mixed_pad_amd import binding

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
GUARD = 1 << 16


def gen(*key):
    g = torch.Generator(device="cuda")
    g.manual_seed(zlib.crc32(repr(key).encode()))
    return g


def inputs(n, v, d, dtype, top):
    g = gen(n, v, d, top)
    x = torch.randn(n, d, device="cuda", generator=g).to(dtype)
    w = (torch.randn(v, d, device="cuda", generator=g) * d ** -0.5).to(dtype)
    index = torch.randint(0, v, (n, top) if top else (n,), device="cuda", generator=g)
    return x, w, index, torch.randn(n, top, device="cuda", generator=g) if top else None


def run(x, w, index, logit, ws, out, **more):
    more.update(lse=out[1], grad_hidden=out[2], grad_head=out[3])
    if logit is None:
        zsp.head_loss(x, w, index, out[0], ws, **more)
    else:
        zsp.head_distill(x, w, index, logit, out[0], ws, temperature=1.5, **more)


def outputs(x, w, fill=float("nan")):
    n = len(x)
    return [torch.full((n,), fill, device="cuda"), torch.full((n,), fill, device="cuda"),
            torch.full_like(x, fill), torch.full_like(w, fill)]


@pytest.mark.parametrize("top", [0, 3])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("n,v,d", [(1, 9001, 64), (16, 9001, 200), (33, 9100, 77), (64, 9001, 512),
                                   (64, 700, 1024), (50, 300, 130), (65, 9001, 64), (300, 700, 96)])
def test_nothing_behind_the_workspace_is_touched(n, v, d, dtype, top):
    """Bytes behind it stay, and what they hold reaches no output."""
    x, w, index, logit = inputs(n, v, d, dtype, top)
    need = binding.zsp_head_workspace(n, v, d, dtype, top)
    outs = []
    for fill in (255, 0):
        buf = torch.full((need + GUARD,), fill, dtype=torch.uint8, device="cuda")
        outs.append(outputs(x, w))
        run(x, w, index, logit, buf[:need], outs[-1])
        assert (buf[need:] == fill).all()
    for a, b in zip(*outs):
        assert torch.equal(a, b) and not a.isnan().any()


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("count", [0, 1, 50])
def test_chunks_without_a_token_that_counts(count, dtype):
    """2^20 columns: chunks of at most 2048 (fp32 256) tokens, the tokens that
    count fewer than the first holds. Against their rows alone, whose gradients
    are rounded in the same places (twice 2^-8 of each; fp32: sums of planes,
    2^-17)."""
    n, v, d = 9000 if dtype == BF else 1500, 1 << 20, 64
    x, w, index, _ = inputs(n, v, d, dtype, 0)
    on = torch.randperm(n, device="cuda", generator=gen("on", n))[:count].sort().values
    masked = torch.full_like(index, -100)
    masked[on] = index[on]
    out = outputs(x, w)
    run(x, w, masked, None, zsp.head_workspace(n, v, d, dtype), out)
    few = outputs(x[on], w)
    run(x[on], w, index[on], None, zsp.head_workspace(count, v, d, dtype), few)
    off = torch.ones(n, dtype=torch.bool, device="cuda")
    off[on] = False
    assert not any(o[off].any() for o in out[:3])
    far = 2.0 ** -7 if dtype == BF else 2.0 ** -17
    for got, want in zip([o[on] for o in out[:3]] + out[3:], few):
        assert torch.linalg.norm(got.double() - want.double()) <= far * torch.linalg.norm(want.double())
        assert not got.isnan().any()


def test_chunks_without_a_token_that_counts_cost_next_to_nothing():
    """The sum of the head's gradient is not read and written for them: 2 GiB
    here, 335 us at 6.4 TB/s; what is left are launches that end at once."""
    v, d = 1 << 20, 256
    least = []
    for chunks in (2, 12):
        n = 2048 * chunks
        x, w, index, _ = inputs(n, v, d, BF, 0)
        index[40:] = -100
        ws, out = zsp.head_workspace(n, v, d, BF), outputs(x, w)
        times = []
        for _ in range(6):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            run(x, w, index, None, ws, out)
            b.record()
            b.synchronize()
            times.append(a.elapsed_time(b))
        least.append(min(times[1:]))
    print("ms of 2 and 12 chunks", least)
    assert (least[1] - least[0]) / 10 < 0.15, least


@pytest.mark.parametrize("n,m,v,d,dtype,top", [(130, 127, 9000, 4096, BF, 0), (300, 33, 9000, 512, F32, 0),
                                               (900, 257, 700, 2048, BF, 4), (2500, 2000, 1 << 20, 64, BF, 0)])
def test_a_smaller_last_batch(n, m, v, d, dtype, top):
    """With the workspace of the others, whose parts it cuts otherwise."""
    x, w, index, logit = inputs(n, v, d, dtype, top)
    ws = zsp.head_workspace(n, v, d, dtype, top=top)
    for k in (n, m, n, m):
        out, own = outputs(x[:k], w), outputs(x[:k], w)
        few = (x[:k], w, index[:k], logit if logit is None else logit[:k])
        run(*few, ws, out)
        run(*few, zsp.head_workspace(k, v, d, dtype, top=top), own)
        for a, b in zip(out, own):
            assert torch.equal(a, b) and not a.isnan().any()


def near_the_definition(out, x, w, index, on, dl, run_of_tokens):
    """Against 64 bits, in norm. dl: a logit's error; G: e c (p + q) with e = 2^-8
    + 2^-10 + dl (bf16) or 2^-16 + dl (fp32); a gradient: that times the other
    operand's largest singular value, k u |G| |the other| for a sum of k at a
    time and one rounding."""
    f32, u = x.dtype == F32, 2.0 ** -24
    X, W = x.double() * on[:, None], w.double()
    l = X @ W.t().contiguous()
    lse = torch.logsumexp(l, 1)
    at = torch.where(on, index, 0)[:, None]
    loss = (lse - l.gather(1, at)[:, 0]) * on
    lse *= on
    for got, ref in zip(out[:2], (loss, lse)):
        assert float((got.double() - ref).abs().max()) <= 2 * dl + 2.0 ** -18 + 2 * u * float(ref.abs().max())
    p = torch.softmax(l, 1) * on[:, None]
    q = torch.zeros_like(p).scatter_(1, at, 1.0) * on[:, None]
    e = float(torch.linalg.norm(p + q)) * ((2.0 ** -16 if f32 else 2.0 ** -8 + 2.0 ** -10) + dl)
    G = p - q
    last = u if f32 else 2.0 ** -8
    for got, g, m, k in ((out[2], G, W, len(W)), (out[3], G.t().contiguous(), X, run_of_tokens)):
        ref, small = g @ m, m if m.shape[0] < m.shape[1] else m.t()
        two = float(torch.linalg.eigvalsh((small @ small.t().contiguous()).cpu()).max()) ** 0.5
        tol = (e * two + (6 if f32 else 1) * k * u * float(torch.linalg.norm(g.abs() @ m.abs()))
               + last * float(torch.linalg.norm(ref)))
        far, size = float(torch.linalg.norm(got.double() - ref)), float(torch.linalg.norm(ref))
        assert far <= tol and tol < 0.1 * size, (far, tol, size)


@pytest.mark.parametrize("half", [False, True])
def test_the_most_tokens(half):
    """2^23, of which all or about half count; the head's gradient is summed over
    2^17 of them at a time, and then over 64 parts."""
    n, v, d = 1 << 23, 70, 8
    x, w, index, _ = inputs(n, v, d, BF, 0)
    on = torch.ones(n, dtype=torch.bool, device="cuda")
    if half:
        on = torch.rand(n, device="cuda", generator=gen("half")) < 0.5
        on[-1] = True
        index[~on] = -1
    out = outputs(x, w)
    run(x, w, index, None, zsp.head_workspace(n, v, d, BF), out)
    sum_xw = float((x[:1 << 16].double().abs() @ w.double().abs().t().contiguous()).max()) * 2
    near_the_definition(out, x, w, index, on, d * 2.0 ** -24 * sum_xw, (1 << 17) + 64)
    assert not half or not any(o[~on].any() for o in out[:3])


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("n", [3, 70, 300])
def test_the_longest_rows(n, dtype):
    """d = 65536. Products of -1, 0 and 1 by 2^-7 of them: sums of any order are
    exact, and logits spread by 1.3."""
    v, d = 200, 65536
    g = gen(n, "rows")
    x = torch.randint(-1, 2, (n, d), device="cuda", generator=g).to(dtype)
    w = (torch.randint(-1, 2, (v, d), device="cuda", generator=g) * 2.0 ** -7).to(dtype)
    index = torch.randint(0, v, (n,), device="cuda", generator=g)
    out = outputs(x, w)
    run(x, w, index, None, zsp.head_workspace(n, v, d, dtype), out)
    assert not any(o.isnan().any() for o in out)
    near_the_definition(out, x, w, index, torch.ones(n, dtype=torch.bool, device="cuda"), 0.0, n)


@pytest.mark.parametrize("n,v,d,dtype", [(300, 9000, 512, BF), (64, 700, 1024, F32)])
def test_an_evaluation_in_a_training_steps_workspace(n, v, d, dtype):
    """With fewer gradients, tokens and entries than it was sized for."""
    x, w, index, logit = inputs(n, v, d, dtype, 4)
    ws = zsp.head_workspace(n, v, d, dtype, top=4)
    for m, top in ((n, 4), (n // 3, 2), (n // 3, 0)):
        few = (x[:m], w, index[:m, :top].contiguous() if top else index[:m, 0].contiguous(),
               logit[:m, :top].contiguous() if top else None)
        whole, alone = outputs(x[:m], w), outputs(x[:m], w)
        run(*few, ws, whole)
        run(*few, ws, alone[:2] + [None, None])
        for a, b in zip(whole[:2], alone[:2]):
            assert torch.equal(a, b) and not a.isnan().any()
