"""The losses over a model's output matrix, with their gradients.

What a training step does between its forward and its backward pass, in plain
torch (`own` false) and through zero_sharded_mixed_pad_amd (`own` true). The
head is the [v, d] output matrix, a parameter gathered from its shards;
hidden is [n, d]; logits l_iv = (hidden_i . head_v) / T.

  loss     softmax cross entropy with a target per token (T = 1):
           loss_i = lse_i - l_iy, lse_i = log sum_v exp l_iv
  distill  distillation from a teacher's top logits t_ik at the indices
           idx_ik, q_i = softmax_k(t_ik / T):
           loss_i = T^2 sum_k q_ik (log q_ik - log p_i,idx_ik), p = softmax(l)

Both give loss and lse per token and, where asked for, the gradients of
scale * sum_i weight_i * loss_i with regard to hidden and head, in the inputs'
type (the head's is what a rank hands to the reduce of gradients). A target
outside [0, v) or a row without a teacher's index in that range does not
count: loss, lse and gradient are 0.
"""
import math
import os
import sys

import torch

own = False

DEV = "cuda"
_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
_ROWS = 4096            # tokens at a time in the plain form and in 64 bits


def _case(name, op, n, v, d, dtype, grads, **more):
    """prompt: the share of each of `seqs` sequences whose tokens do not
    count; weights: a weight per token; top, temp, ragged: the teacher's
    entries per token, the temperature, and whether rows hold fewer."""
    c = dict(name=name, op=op, n=n, v=v, d=d, dtype=dtype, grads=grads, prompt=0.0, seqs=1,
             weights=False, top=0, temp=1.0, ragged=False)
    c.update(more)
    return c


def listed():
    return [
        # scoring a handful of tokens with a 7B head: one read of the head
        _case("score_few", "loss", 5, 32000, 4096, "bf16", "none"),
        # a small fp32 weight with odd rows as the head: latency
        _case("loss_one_fp32", "loss", 61, 1000, 1003, "fp32", "both"),
        # one short sequence: the head read twice, its gradient written once
        _case("loss_short", "loss", 96, 32000, 4096, "bf16", "both"),
        # a micro-batch of 4096 tokens through a 7B head
        _case("loss_micro", "loss", 4096, 32000, 4096, "bf16", "both"),
        # fine-tuning on answers: 60% of a ragged batch is prompt
        _case("loss_prompt", "loss", 6001, 32000, 4096, "bf16", "both", prompt=0.6, seqs=7,
              weights=True),
        # an evaluation batch: losses alone
        _case("score_long", "loss", 16384, 32000, 4096, "bf16", "none"),
        # a large vocabulary and a long batch
        _case("loss_wide", "loss", 10000, 131072, 4096, "bf16", "both"),
        # odd sizes in every direction
        _case("loss_odd", "loss", 1777, 50021, 1283, "bf16", "both", weights=True),
        # fp32 parameters and gradients
        _case("loss_fp32", "loss", 2048, 32000, 2048, "fp32", "both"),
        # distillation of a few tokens
        _case("distill_few", "distill", 17, 32000, 4096, "bf16", "both", top=8, temp=2.0),
        # distillation of a micro-batch
        _case("distill_micro", "distill", 4096, 32000, 4096, "bf16", "both", top=64, temp=2.0,
              prompt=0.25, seqs=4),
        # a frozen fp32 head, rows with fewer entries than others
        _case("distill_frozen", "distill", 333, 10007, 768, "fp32", "hidden", top=100, temp=1.5,
              ragged=True, weights=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    grads = rng.choice(["both", "both", "hidden", "head", "none"])
    v, d = _log(rng, 60, 131072), _log(rng, 16, 5120)
    if rng.random() < 0.6:                # widths are mostly round
        d = max(64, d // 64 * 64)
    # at most a sixth of the largest listed case's products, fp32 a sixth of that
    most = 2 * 10000 * 131072 * 4096 / (6 if dtype == "bf16" else 36)
    n = _log(rng, 1, max(2, min(16384, most / (2 * v * d))))
    c = _case("", rng.choice(["loss", "loss", "distill"]), n, v, d, dtype, grads,
              weights=rng.random() < 0.5)
    del c["name"]
    if rng.random() < 0.4:
        c.update(prompt=rng.uniform(0.1, 0.8), seqs=rng.randint(1, 9))
    if c["op"] == "distill":
        c.update(top=min(v // 2, _log(rng, 1, 256)), temp=rng.choice([1.0, 1.5, 2.0, 4.0]),
                 ragged=rng.random() < 0.5)
    return c


def _counts(case):
    """Which tokens count: those past the prompt of their sequence."""
    length = -(-case["n"] // case["seqs"])
    return torch.arange(case["n"]) % length >= int(case["prompt"] * length)


# ---- inputs ------------------------------------------------------------------------

def _zsp():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    if root not in sys.path:
        sys.path.insert(0, root)
    import zero_sharded_mixed_pad_amd as zsp
    return zsp


def prepare(case, seed):
    """Normalised hidden states over a head whose logits spread by about 1.5,
    drawn towards their target (or the teacher's first index) so that the
    model's probability of it runs from next to nothing to nearly 1."""
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 1_000_003 + 29)
    n, v, d, k = case["n"], case["v"], case["d"], case["top"]
    dt = _TYPES[case["dtype"]]
    rand = lambda *s: torch.rand(*s, device=DEV, generator=g)  # noqa: E731
    head = torch.empty(v, d, device=DEV).normal_(0.0, 1.5 / math.sqrt(d), generator=g).to(dt)
    target = torch.randint(0, v, (n,), device=DEV, generator=g)
    hidden = torch.empty(n, d, device=DEV).normal_(0.0, 1.0, generator=g)
    hidden += head[target].float() * (rand(n, 1) * (math.log(v) + 6.0) / 2.25)
    hidden = hidden.to(dt)
    counts = _counts(case).to(DEV)
    st = dict(op=case["op"], hidden=hidden, head=head, grads=case["grads"], temp=case["temp"],
              scale=1.0 / max(1, int(_counts(case).sum())),
              weight=0.25 + 1.5 * rand(n) if case["weights"] else None)
    if case["op"] == "loss":
        st["target"] = torch.where(counts, target, -100)
    else:                       # distinct indices in a row, the logits in falling order
        step = v // k
        st["index"] = (target[:, None] + step * torch.arange(k, device=DEV)) % v
        fall = torch.empty(n, k, device=DEV).exponential_(1.0, generator=g)
        st["logit"] = 14.0 * rand(n, 1) + 4.0 - torch.cumsum(fall, 1) * (8.0 / (k + 8))
        keep = counts[:, None].expand(n, k)
        if case["ragged"]:
            keep = keep & (torch.arange(k, device=DEV) <= rand(n, 1) * k)
        st["index"] = torch.where(keep, st["index"], -1)
    if own:
        zsp = _zsp()
        st["zsp"] = zsp
        st["loss"], st["lse"] = torch.empty(n, device=DEV), torch.empty(n, device=DEV)
        st["grad_hidden"] = torch.empty_like(hidden) if case["grads"] in ("both", "hidden") else None
        st["grad_head"] = torch.empty_like(head) if case["grads"] in ("both", "head") else None
        st["ws"] = zsp.head_workspace(n, v, d, dt, top=k,
                                      grad_hidden=st["grad_hidden"] is not None,
                                      grad_head=st["grad_head"] is not None)
    return st


# ---- one pass -----------------------------------------------------------------------

def run(st):
    return _run_own(st) if own else _run_plain(st)


def _run_own(st):
    more = dict(token_weight=st["weight"], scale=st["scale"], lse=st["lse"],
                grad_hidden=st["grad_hidden"], grad_head=st["grad_head"])
    if st["op"] == "loss":
        st["zsp"].head_loss(st["hidden"], st["head"], st["target"], st["loss"], st["ws"], **more)
    else:
        st["zsp"].head_distill(st["hidden"], st["head"], st["index"], st["logit"], st["loss"],
                               st["ws"], temperature=st["temp"], **more)
    out = {"loss": st["loss"], "lse": st["lse"]}
    out.update({k: st[k] for k in ("grad_hidden", "grad_head") if st[k] is not None})
    return out


def _run_plain(st):
    hidden, temp = st["hidden"], st["temp"]
    n, v = len(hidden), len(st["head"])
    dt = hidden.dtype
    w = st["head"].float()
    want_h, want_w = st["grads"] in ("both", "hidden"), st["grads"] in ("both", "head")
    losses, lses, gh = [], [], []
    gw = torch.zeros_like(w) if want_w else None
    for a in range(0, n, _ROWS):
        rows = slice(a, a + _ROWS)
        x = hidden[rows].float()
        if st["op"] == "loss":
            idx = st["target"][rows, None]
            ok = (idx >= 0) & (idx < v)
            q = ok.float()
        else:
            idx = st["index"][rows]
            ok = (idx >= 0) & (idx < v)
            t = torch.where(ok, st["logit"][rows] / temp, -math.inf)
            top = t.max(1, keepdim=True).values
            e = torch.where(ok, torch.exp(t - top), 0.0)
            q = e / e.sum(1, keepdim=True).clamp_min(1e-30)
        counts = ok.any(1)
        idx = torch.where(ok, idx, 0)
        p = x @ w.t()
        if temp != 1.0:
            p /= temp
        own_logit = p.gather(1, idx)
        top = p.max(1, keepdim=True).values
        p.sub_(top).exp_()
        total = p.sum(1, keepdim=True)
        lse = (top + total.log())[:, 0]
        # a sum over the row's entries of q (log q - log p)
        ratio = torch.where(q > 0, q.clamp_min(1e-38).log(), 0.0) - (own_logit - lse[:, None])
        loss = (temp * temp) * torch.where(ok, q * ratio, 0.0).sum(1)
        losses.append(torch.where(counts, loss, 0.0))
        lses.append(torch.where(counts, lse, 0.0))
        if not (want_h or want_w):
            continue
        c = torch.where(counts, st["scale"] * temp, 0.0)
        if st["weight"] is not None:
            c = c * st["weight"][rows]
        p.mul_(c[:, None] / total)
        p.scatter_add_(1, idx, -(c[:, None] * q))
        if want_h:
            gh.append((p @ w).to(dt))
        if want_w:
            gw += p.t() @ x
    out = {"loss": torch.cat(losses), "lse": torch.cat(lses)}
    if want_h:
        out["grad_hidden"] = torch.cat(gh)
    if want_w:
        out["grad_head"] = gw.to(dt)
    return out


# ---- what a pass cannot do without -------------------------------------------------

def work(case):
    n, v, d = case["n"], case["v"], case["d"]
    size = 2 if case["dtype"] == "bf16" else 4
    h, w = case["grads"] in ("both", "hidden"), case["grads"] in ("both", "head")
    b = size * ((n * d) * (2 if h else 1) + (v * d) * (2 if w else 1)) + 8 * n
    b += 8 * n if case["op"] == "loss" else 12 * n * case["top"]
    b += 4 * n if case["weights"] else 0
    active = int(_counts(case).sum())
    return {"bytes": b, "flops": 2 * active * v * d * (1 + h + w)}


# ---- the definition in 64 bits -----------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    n, v, temp = case["n"], case["v"], case["temp"]
    w = st["head"].double()
    h_on, w_on = case["grads"] in ("both", "hidden"), case["grads"] in ("both", "head")
    out = {"loss": torch.zeros(n, dtype=torch.float64, device=DEV),
           "lse": torch.zeros(n, dtype=torch.float64, device=DEV)}
    if h_on:
        out["grad_hidden"] = torch.zeros(n, case["d"], dtype=torch.float64, device=DEV)
    if w_on:
        out["grad_head"] = torch.zeros_like(w)
    index = st["target"][:, None] if case["op"] == "loss" else st["index"]
    good = ((index >= 0) & (index < v)).any(1).nonzero()[:, 0]     # the tokens that count
    for part in good.split(_ROWS):
        if not len(part):
            continue
        x = st["hidden"][part].double()
        idx = index[part]
        ok = (idx >= 0) & (idx < v)
        if case["op"] == "loss":
            logq = torch.zeros(idx.shape, dtype=torch.float64, device=DEV)
        else:
            t = (st["logit"][part].double() / temp).masked_fill(~ok, -math.inf)
            logq = torch.log_softmax(t, 1)
        q = logq.exp().masked_fill(~ok, 0.0)
        logp = torch.matmul(x, w.T) / temp
        lse = torch.logsumexp(logp, 1)
        logp -= lse[:, None]
        at = idx.clamp(0, v - 1)
        terms = (q * (logq - torch.gather(logp, 1, at))).masked_fill(~ok | (q == 0), 0.0)
        out["lse"][part] = lse
        out["loss"][part] = temp ** 2 * terms.sum(1)
        if h_on or w_on:
            grad = torch.exp(logp)
            grad.scatter_add_(1, at, -q)
            c = torch.full((len(part), 1), st["scale"] * temp, dtype=torch.float64, device=DEV)
            if st["weight"] is not None:
                c = c * st["weight"][part].double()[:, None]
            grad *= c
            if h_on:
                out["grad_hidden"][part] = torch.matmul(grad, w)
            if w_on:
                out["grad_head"] += torch.matmul(grad.T, x)
    return out
