"""The global gradient norm, gradient clipping and the clipped optimizer step.

What a training step does between the reduce of its gradients and the update,
in plain torch (`own` false) and through zero_sharded_mixed_pad_amd (`own`
true):

  norm         global norm of a list of tensors, and the clipping coefficient
  clip         the list scaled in place by a coefficient in device memory
  acc_norm     global norm of the sharded gradient accumulator
  reduce_norm  the reduce of N_d ranks' gradients into the accumulator, with
               the norm of what it wrote
  layers       the same layer by layer, the layers' norms joined at the end
  step         norm of the reduced gradient, then the clipped fused step, with
               no accumulator
  window       the end of an accumulation window: the accumulator's norm,
               then the clipped step from it

State arrays are indexed [rank, slot] as zsp.h describes; shard-layout
gradients likewise, full-layout ones hold each padded parameter in turn.
"""
import math
import os
import sys

import numpy as np
import torch

own = False

DEV = "cuda"
HP = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8)
STEP = 7

_D, _F = 4096, 11008
_LAYER = [_D * _D] * 4 + [_D * _F] * 3 + [_D] * 2


# ---- parameter sizes by name ---------------------------------------------------

def _sizes(case):
    """Element counts of the case's parameters or tensors."""
    kind = case["sizes"]
    if kind == "layer":            # one decoder layer: 202 M elements, no pad
        return list(_LAYER)
    if kind == "ragged_layer":     # the same with odd sizes, each padded
        return [n + d for n, d in zip(_LAYER, (1, -3, 5, 0, 7, -1, 2, 3, -5))]
    if kind == "stack":            # 32 layers, embedding and head (6.7 G elements)
        return _LAYER * 32 + [32000 * _D] * 2
    if kind == "one":
        return [1000 * 1003]
    # "many": count sizes, log-uniform in [lo, hi]
    rng = np.random.default_rng(case["sizes_seed"])
    x = rng.uniform(math.log(case["lo"]), math.log(case["hi"]), size=case["count"])
    return [int(round(math.exp(v))) for v in x]


def listed():
    many = dict(sizes="many", count=10_000, lo=64, hi=65536, sizes_seed=1)
    return [
        # a handful of small gradients in one call: latency
        dict(name="norm_few", op="norm", sizes="many", count=9, lo=5, hi=4100, sizes_seed=3,
             dtype="mixed", kind="l2", clip=0.5, once=True),
        # 10,000 gradients of both types, the list prepared once
        dict(name="norm_10k", op="norm", dtype="mixed", kind="l2", clip=0.5, once=False, **many),
        # one decoder layer's bf16 gradients
        dict(name="norm_layer", op="norm", sizes="layer", dtype="bf16", kind="l2", clip=2.0,
             once=False),
        # clipping the 10,000 gradients in place
        dict(name="clip_10k", op="clip", dtype="mixed", coef=0.96875, once=False, **many),
        # clipping a layer's fp32 gradients in place
        dict(name="clip_layer", op="clip", sizes="layer", dtype="fp32", coef=0.96875, once=False),
        # norm of one weight's reduced gradient, a few MB over 4 ranks
        dict(name="acc_norm_one", op="acc_norm", sizes="one", nd=4, rank=-1, kind="l2", clip=0.5),
        # norm of a layer's accumulator with odd sizes: pad slots at every shard end
        dict(name="acc_norm_ragged", op="acc_norm", sizes="ragged_layer", nd=8, rank=-1, kind="max",
             clip=0.5),
        # the last micro-batch's reduce of a layer, with the norm
        dict(name="reduce_layer", op="reduce_norm", sizes="layer", nd=8, rank=-1, dtype="bf16",
             layout="full", acc=True, kind="l2", clip=0.5),
        # backward over 10,000 small parameters in four buckets, one norm each
        dict(name="layers_10k", op="layers", nd=8, rank=-1, dtype="bf16", layout="shard", groups=4,
             acc=False, kind="l2", clip=0.5, **many),
        # the whole step of one fp32 weight: latency
        dict(name="step_one", op="step", sizes="one", nd=4, rank=-1, dtype="fp32", layout="full",
             kind="l2", clip=0.5),
        # one rank's step of a 7B-shaped model over 64 ranks
        dict(name="step_rank_nd64", op="step", sizes="stack", nd=64, rank=0, dtype="bf16",
             layout="shard", kind="l2", clip=0.5),
        # the end of an accumulation window for one layer over 8 ranks
        dict(name="window_layer", op="window", sizes="layer", nd=8, rank=-1, kind="l2", clip=0.5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "clip", "acc_norm", "reduce_norm", "layers", "step", "window"])
    nd = rng.choice([1, 2, 3, 5, 8, 8, 13, 16, 24, 64])
    grads = op in ("reduce_norm", "layers", "step")
    # elements, about; gradients of all ranks together at most 1.2 G elements
    total = _log(rng, 300, min(60_000_000, 1_200_000_000 // nd) if grads else 60_000_000)
    count = min(_log(rng, 1, 3000), max(1, total // 40))
    mean = max(1, total // count)
    wide = count >= 8
    c = dict(op=op, sizes="many", count=count, lo=max(1, mean // (4 if wide else 2)),
             hi=max(2, mean * 5 // (2 if wide else 4)), sizes_seed=rng.randrange(1 << 30))
    if op in ("norm", "clip"):
        c.update(dtype=rng.choice(["bf16", "fp32", "mixed"]), once=count <= 200 and rng.random() < 0.5)
        if op == "clip":
            c.update(coef=rng.uniform(0.9, 0.97))
            return c
    else:
        c.update(nd=nd, rank=rng.randrange(nd) if rng.random() < 0.4 else -1)
        if grads:
            c.update(dtype=rng.choice(["bf16", "fp32"]), layout=rng.choice(["full", "shard"]))
        if op in ("reduce_norm", "layers"):
            c.update(acc=rng.random() < 0.5)
        if op == "layers":
            c.update(groups=min(count, rng.choice([1, 2, 3, 5])))
    c.update(kind=rng.choice(["l2", "l2", "max"]), clip=rng.choice([0.25, 0.7, 3.0]))
    return c


# ---- inputs ------------------------------------------------------------------------

class _Layout:
    """Offsets of parameters padded to N_d and cut into N_d slices each."""

    def __init__(self, numel, nd, rank):
        n = np.array(numel, dtype=np.int64)
        self.numel, self.nd, self.rank = n, nd, rank
        self.shard = -(-n // nd)                      # shard_len
        self.padded = self.shard * nd
        self.shard_off = np.concatenate([[0], np.cumsum(self.shard)])
        self.full_off = np.concatenate([[0], np.cumsum(self.padded)])
        self.S = int(self.shard_off[-1])
        self.total_padded = int(self.full_off[-1])
        self.ranks = nd if rank < 0 else 1            # rows of the bound state

    def owned(self):
        """Elements of the bound ranks, pads left out."""
        lo = (0 if self.rank < 0 else self.rank) * self.shard
        hi = (self.nd if self.rank < 0 else self.rank + 1) * self.shard
        return int(np.clip(np.minimum(hi, self.numel) - lo, 0, None).sum())

    def real(self):
        """[ranks, S] truth values: not a pad slot. None where nothing is padded."""
        if not (self.padded - self.numel).any():
            return None
        s = torch.from_numpy(self.shard).to(DEV)
        t = torch.repeat_interleave(torch.arange(len(s), device=DEV), s, output_size=self.S)
        slot = torch.arange(self.S, device=DEV) - torch.from_numpy(self.shard_off).to(DEV)[t]
        left = torch.from_numpy(self.numel).to(DEV)[t] - slot      # real iff r * s_t < left
        s = s[t]
        rows = range(self.nd) if self.rank < 0 else [self.rank]
        return torch.stack([r * s < left for r in rows])


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 1_000_003 + 17)
    return g


_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _zsp():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    if root not in sys.path:
        sys.path.insert(0, root)
    import zero_sharded_mixed_pad_amd as zsp
    return zsp


def _prepare_list(case, seed):
    """The tensors as views of one arena per type, each starting on 16 bytes
    (every seventh one element further on, as views into a flat buffer may)."""
    g = _gen(seed)
    numel = _sizes(case)
    types = [case["dtype"] if case["dtype"] != "mixed" else "fp32" if i % 4 == 3 else "bf16"
             for i in range(len(numel))]
    off, end = [], {"bf16": 0, "fp32": 0}
    for i, (n, t) in enumerate(zip(numel, types)):
        at = end[t] + (1 if i % 7 == 6 else 0)
        off.append(at)
        end[t] = -(-(at + n) // 8) * 8
    arena = {}
    for t, e in end.items():
        if e:                          # 0 in the gaps between tensors
            inside = np.zeros(e + 1, dtype=np.int8)
            for n, o, u in zip(numel, off, types):
                if u == t:
                    inside[o] += 1
                    inside[o + n] -= 1
            arena[t] = torch.empty(e, dtype=_TYPES[t], device=DEV).normal_(0.0, 1e-2, generator=g)
            arena[t].mul_(torch.from_numpy(np.cumsum(inside[:-1], dtype=np.int8)).to(DEV))
    st = dict(op=case["op"], arena=arena,
              xs=[arena[t][o:o + n] for n, t, o in zip(numel, types, off)])
    if case["op"] == "norm":
        st.update(kind=case["kind"], max_norm=case["clip"] * _size_of_norm(case, sum(numel), 1e-2))
    else:
        # the record that a norm call left: sum of squares, norm and coefficient
        norm = torch.tensor([3.5, case["coef"]], dtype=torch.float32, device=DEV)
        st["record"] = torch.stack([torch.tensor(12.25, dtype=torch.float64, device=DEV),
                                    norm.view(torch.float64)[0]])[None]
    if own:
        zsp = _zsp()
        st["zsp"] = zsp
        st["ws"], st["out"] = zsp.norm_workspace(), zsp.clip_record()
        st["list"] = None if case["once"] else zsp.TensorList(st["xs"])
    return st


def _size_of_norm(case, n, sigma):
    """About the norm of n values of N(0, sigma^2): what max_norm is set by."""
    return sigma * (math.sqrt(n) if case["kind"] == "l2" else math.sqrt(2 * math.log(n + 2)))


def _prepare_plan(case, seed):
    g = _gen(seed)
    nd, op = case["nd"], case["op"]
    numel = _sizes(case)
    lay = _Layout(numel, nd, case["rank"])
    n = lay.ranks * lay.S
    st = dict(op=op, lay=lay, real=lay.real(), kind=case["kind"], acc=None,
              layout=case.get("layout"), accumulate=bool(case.get("acc")),
              max_norm=case["clip"] * _size_of_norm(case, lay.owned(), 1e-3 * math.sqrt(nd)))

    def values(sigma):
        x = torch.empty(lay.ranks, lay.S, device=DEV).normal_(0.0, sigma, generator=g)
        return x if st["real"] is None else x.mul_(st["real"])

    if op != "step":
        st["acc"] = values(1e-3 * math.sqrt(nd))
    if op in ("step", "window"):       # the state some steps into training
        st["master"], st["m"] = values(0.02), values(1e-3)
        st["v"] = values(2e-3).square_()
        st["work"] = st["master"].to(torch.bfloat16)
    if "dtype" in case:
        k = lay.total_padded if case["layout"] == "full" else n
        buf = torch.empty(nd, -(-k // 8) * 8, dtype=_TYPES[case["dtype"]], device=DEV)
        st["grads"] = buf.normal_(0.0, 1e-3, generator=g)[:, :k]
    if op == "layers":
        cut = np.linspace(0, len(numel), case["groups"] + 1).astype(int)
        st["groups"] = [(int(a), int(b - a)) for a, b in zip(cut[:-1], cut[1:])]
    if own:
        zsp = _zsp()
        flat = lambda k, t=torch.float32: (  # noqa: E731
            st[k].view(-1) if st.get(k) is not None else torch.zeros(n, dtype=t, device=DEV))
        st["zsp"], st["rank"] = zsp, case["rank"]
        st["plan"] = zsp.partition(numel, nd)
        st["plan"].bind_state(case["rank"], flat("master"), flat("m"), flat("v"),
                              flat("work", torch.bfloat16), None if op == "step" else flat("acc"))
        st["ws"], st["out"] = st["plan"].norm_workspace(), zsp.clip_record()
        st["parts"] = zsp.clip_record(case.get("groups", 1))
        st["rows"] = list(st["grads"].unbind(0)) if "grads" in st else None
    return st


def prepare(case, seed):
    return _prepare_list(case, seed) if case["op"] in ("norm", "clip") else _prepare_plan(case, seed)


# ---- one pass -----------------------------------------------------------------------

def run(st):
    return _run_own(st) if own else _run_plain(st)


def _record(op, total, norm, coef):
    """What a norm call says. The 64-bit total is among it where the values
    under it are inputs; a sum over ranks has rounded them to 32 bits, and
    the norm then says all there is to compare."""
    rec = {"norm": norm.reshape(()), "coef": coef.reshape(())}
    return {"total": total.reshape(()), **rec} if op in ("norm", "acc_norm", "window") else rec


def _state(st):
    return {k: st[k] for k in ("master", "m", "v", "work")}


def _run_own(st):
    op, zsp, out, ws = st["op"], st["zsp"], st["out"], st["ws"]
    if op == "clip":
        if st["list"] is None:
            zsp.clip_many(st["xs"], st["record"])
        else:
            st["list"].clip(st["record"])
        return dict(st["arena"])
    lim = dict(max_norm=st["max_norm"], kind=st["kind"])
    if op == "norm":
        if st["list"] is None:
            zsp.norm_many(st["xs"], out, ws, **lim)
        else:
            st["list"].norm(out, ws, **lim)
        return _record(op, *zsp.clip_values(out))
    plan, rank = st["plan"], st["rank"]
    if op == "acc_norm":
        plan.grad_norm(rank, out, ws, **lim)
        return _record(op, *zsp.clip_values(out))
    if op == "reduce_norm":
        plan.reduce_shard_norm(rank, st["rows"], out, ws, layout=st["layout"],
                               accumulate=st["accumulate"], **lim)
        return {"acc": st["acc"], **_record(op, *zsp.clip_values(out))}
    if op == "layers":
        for i, (first, n) in enumerate(st["groups"]):
            plan.reduce_shard_norm_params(rank, first, n, st["rows"], st["parts"][i:i + 1], ws,
                                          layout=st["layout"], accumulate=st["accumulate"],
                                          kind=st["kind"])
        zsp.clip_combine(st["parts"], out, **lim)
        return {"acc": st["acc"], **_record(op, *zsp.clip_values(out))}
    if op == "step":
        plan.reduce_norm(rank, st["rows"], out, ws, layout=st["layout"], **lim)
        plan.reduce_adam_step_clip(rank, st["rows"], out, step=STEP, layout=st["layout"], **HP)
    else:
        plan.grad_norm(rank, out, ws, **lim)
        plan.adam_step_clip(rank, out, step=STEP, **HP)
    return {**_state(st), **_record(op, *zsp.clip_values(out))}


def _coef(total, norm, max_norm):
    """The clipping coefficient (64-bit norm): NaN where the norm is not finite."""
    c = torch.where(norm > max_norm, max_norm / norm, torch.ones_like(norm))
    return torch.where(torch.isfinite(norm), c, torch.full_like(norm, math.nan))


def _norm_of(parts, kind, max_norm):
    """The record of the values in `parts` (64-bit sums)."""
    if kind == "l2":
        total = torch.stack([torch.sum(p.double().square()) for p in parts]).sum()
        norm = total.sqrt()
    else:
        total = torch.stack([p.abs().max() for p in parts]).double().max()
        norm = total
    return total, norm.float(), _coef(total, norm, max_norm).float()


def _reduced(st):
    """The sum over ranks in 32 bits, [ranks, S], 0 in pad slots."""
    lay, g = st["lay"], st["grads"]
    red = torch.sum(g, 0, dtype=torch.float32)
    if st["layout"] == "full":
        rows = slice(None) if lay.rank < 0 else slice(lay.rank, lay.rank + 1)
        red = torch.cat([p.view(lay.nd, -1)[rows]
                         for p in torch.split(red, lay.padded.tolist())], 1)
    red = red.view(lay.ranks, lay.S)
    return red if st["real"] is None else torch.where(st["real"], red, 0.0)


def _scalars():
    f = np.float32
    b1, b2 = f(HP["beta1"]), f(HP["beta2"])
    return (float(f(HP["lr"])), float(b1), float(b2), float(f(HP["eps"])), float(f(1) - b1),
            float(f(1) - b2), float(f(1.0 - float(b1) ** STEP)), float(f(1.0 - float(b2) ** STEP)))


def _adam_plain(st, g, norm, coef):
    """The clipped update in 32 bits, in place; nothing changes where the norm is not finite."""
    lr, b1, b2, eps, o1, o2, c1, c2 = _scalars()
    ok = torch.isfinite(coef)
    g = torch.where(ok, g * coef, 0.0)
    keep = lambda a, b: torch.where(ok, a, b)  # noqa: E731
    m = st["m"].mul_(keep(b1, 1.0)).add_(g * o1)
    v = st["v"].mul_(keep(b2, 1.0)).add_(g.square_().mul_(o2))
    den = (v / c2).sqrt_().add_(eps)
    st["master"].sub_((m / c1).mul_(keep(lr, 0.0)).div_(den))
    st["work"].copy_(st["master"])


def _run_plain(st):
    op = st["op"]
    if op == "clip":
        coef = st["record"].view(torch.float32)[0, 3]
        ok = torch.isfinite(coef)
        c = torch.where(ok, coef, 1.0)
        for x in st["arena"].values():      # the gaps between the tensors hold zeros
            x.copy_(x * c if x.dtype == torch.float32 else x.float() * c)
        return dict(st["arena"])
    kind, max_norm = st["kind"], st["max_norm"]
    if op == "norm":
        flat = [torch.cat([x for x in st["xs"] if x.dtype == t]) for t in _TYPES.values()
                if any(x.dtype == t for x in st["xs"])]
        return _record(op, *_norm_of(flat, kind, max_norm))
    if op == "acc_norm":
        return _record(op, *_norm_of([st["acc"]], kind, max_norm))
    if op in ("reduce_norm", "layers"):
        red = _reduced(st)
        st["acc"].copy_(st["acc"] + red if st["accumulate"] else red)
        return {"acc": st["acc"], **_record(op, *_norm_of([st["acc"]], kind, max_norm))}
    g = _reduced(st) if op == "step" else st["acc"]
    rec = _norm_of([g], kind, max_norm)
    _adam_plain(st, g, rec[1], rec[2])
    return {**_state(st), **_record(op, *rec)}


# ---- what a pass cannot do without -------------------------------------------------

def work(case):
    op = case["op"]
    numel = _sizes(case)
    if op in ("norm", "clip"):
        size = {"bf16": 2, "fp32": 4}
        b = sum(n * (size[case["dtype"]] if case["dtype"] != "mixed" else 4 if i % 4 == 3 else 2)
                for i, n in enumerate(numel))
        return {"bytes": b * (1 if op == "norm" else 2) + 16,
                "flops": sum(numel) * (2 if op == "norm" else 1)}
    n = _Layout(numel, case["nd"], case["rank"]).owned()
    g = case["nd"] * {"bf16": 2, "fp32": 4, None: 0}[case.get("dtype")]
    per = {"acc_norm": 4, "reduce_norm": g + 4, "layers": g + 4, "step": g + 26, "window": 30}[op]
    per += 4 if case.get("acc") else 0
    ops = (case["nd"] if g else 0) + 2 + (20 if op in ("step", "window") else 0)
    return {"bytes": n * per + 16, "flops": n * ops}


# ---- the definition in 64 bits -----------------------------------------------------

def _exact_record(op, chunks, kind, max_norm):
    s = mx = 0.0
    for x in chunks:
        x = x.double().abs()
        s += float(torch.dot(x, x))
        mx = max(mx, float(x.max()) if x.numel() else 0.0)
    norm = math.sqrt(s) if kind == "l2" else mx
    coef = 1.0 if norm <= max_norm else max_norm / norm
    f = lambda v: torch.tensor(v, dtype=torch.float64)  # noqa: E731
    return _record(op, f(s if kind == "l2" else mx), f(norm), f(coef))


def _exact_reduced(st):
    """The 64-bit sum over ranks in [ranks, S], parameter by parameter."""
    lay, real = st["lay"], st["real"]
    g = sum(st["grads"][r].double() for r in range(lay.nd))
    if st["layout"] == "shard":
        out = g.view(lay.ranks, lay.S)
    else:
        out = torch.zeros(lay.ranks, lay.S, dtype=torch.float64, device=DEV)
        for t, (o, s, so) in enumerate(zip(lay.full_off, lay.shard, lay.shard_off)):
            for i, r in enumerate(range(lay.nd) if lay.rank < 0 else [lay.rank]):
                a = int(o + r * s)
                out[i, int(so):int(so + s)] = g[a:a + int(s)]
    return out if real is None else out.masked_fill_(~real, 0.0)


def exact(case, seed):
    op = case["op"]
    st = prepare(case, seed)
    if op == "clip":
        c = float(st["record"].view(torch.float32)[0, 3])
        return {t: x.double() * c for t, x in st["arena"].items()}
    kind, max_norm = st["kind"], st["max_norm"]
    if op == "norm":
        return _exact_record(op, st["xs"], kind, max_norm)
    if op == "acc_norm":
        return _exact_record(op, [st["acc"].view(-1)], kind, max_norm)
    if op in ("reduce_norm", "layers"):
        g = _exact_reduced(st)
        if st["accumulate"]:
            g += st["acc"].double()
        return {"acc": g, **_exact_record(op, [g.view(-1)], kind, max_norm)}
    g = _exact_reduced(st) if op == "step" else st["acc"].double()
    rec = _exact_record(op, [g.view(-1)], kind, max_norm)
    lr, b1, b2, eps, o1, o2, c1, c2 = _scalars()
    g = g * float(rec["coef"])
    m = b1 * st["m"].double() + o1 * g
    v = b2 * st["v"].double() + o2 * g * g
    p = st["master"].double() - lr * (m / c1) / ((v / c2).sqrt() + eps)
    return {"master": p, "m": m, "v": v, "work": p, **rec}
