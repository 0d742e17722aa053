"""Norms of parameter ranges of all ranks whose partials are too many for one
workgroup to join: several spans in one launch, each with its own run of
partials, in a workspace of exactly the documented size with guards behind it.

References and tolerances as in test_gpu_norm_clip.py: the accumulator bit for
bit that of the plain reduce, the norm within (N + 2) * 2^-53 of the 64-bit
sum (one rounding per square and per addition).
"""
import pytest
import torch

import zero_sharded_mixed_pad_amd as zsp
from zero_sharded_mixed_pad_amd import binding, synth

from test_gpu_norm_clip import BF, FP, check_record, grads_of, real_mask
from test_gpu_parity import Mirror, assert_bits, np_of

pytestmark = pytest.mark.gpu

TILE = 512          # elements a wave (long pieces: two waves) takes
ONE_JOIN = 8192     # partials that one workgroup joins
GUARD = 4096

# parameters 1 .. of a model whose parameter 0 has one element, so that no
# rank's span starts with a tile. By ranks and elements per rank:
LONG = [
    (8, [600 * TILE + 2]),         # spans of 602 tiles where a multiple of 512 needs 600:
    (16, [300 * TILE + 2]),        # the workspace is full to a few partials
    (8, [290_001, 40_961, 1]),
    (3, [900_011, 7]),             # some spans meet one tile less than others
]
SHORT = [(8, 1500), (16, 1500)]    # ranks, parameters


def layout(case):
    if case < len(LONG):
        nd, shards = LONG[case]
        return [1] + [nd * s for s in shards], nd
    nd, count = SHORT[case - len(LONG)]
    return [1] + synth.small_tensor_sizes(count=count, lo=900, hi=9000, seed=case), nd


@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("case", range(len(LONG) + len(SHORT)))
def test_many_partials_in_a_range_of_all_ranks(case, dt):
    numels, nd = layout(case)
    A, B = Mirror(numels, nd), Mirror(numels, nd)
    S = A.L.S
    per_wave = TILE // 2 if case < len(LONG) else TILE
    assert nd * ((S - 1) // per_wave) > ONE_JOIN
    need = binding.zsp_norm_workspace(A.plan.handle)
    buf = torch.full((need + GUARD,), 0xA5, dtype=torch.uint8, device="cuda")
    ws, guard = buf[:need], buf[need:]
    layout_of = "full" if dt == BF else "shard"
    grads = grads_of(A, dt, ("ranges", case), layout_of)
    first, n = 1, len(numels) - 1
    at = real_mask(A.L, A.ranks, first, n)
    start = synth.normal(A.g_acc.numel(), 1e-2, FP, 13).to("cuda")
    rec = zsp.clip_record()
    for accumulate, kind in ((False, "l2"), (True, "max"), (True, "l2")):
        A.g_acc.copy_(start)
        B.g_acc.copy_(start)
        A.plan.reduce_shard_norm_params(zsp.ALL_RANKS, first, n, grads, rec, ws,
                                        layout=layout_of, accumulate=accumulate, max_norm=0.5,
                                        kind=kind)
        B.plan.reduce_shard_params(zsp.ALL_RANKS, first, n, grads, layout=layout_of,
                                   accumulate=accumulate)
        assert_bits(np_of(A.g_acc), np_of(B.g_acc), "accumulator")   # outside the range too
        vals = np_of(B.g_acc)[at]
        check_record(rec, vals, kind, 0.5)
        assert (guard == 0xA5).all()
        A.plan.grad_norm_params(zsp.ALL_RANKS, first, n, rec, ws, max_norm=0.5, kind=kind)
        check_record(rec, vals, kind, 0.5)
        assert (guard == 0xA5).all()
    # the whole model through the same workspace
    A.plan.reduce_norm(zsp.ALL_RANKS, grads, rec, ws, layout=layout_of, max_norm=0.5)
    B.plan.reduce_shard(zsp.ALL_RANKS, grads, layout=layout_of)
    check_record(rec, np_of(B.g_acc)[real_mask(A.L, A.ranks)], "l2", 0.5)
    assert (guard == 0xA5).all()


def test_every_span_counts_once():
    """One element larger than the rest in each rank's span in turn, at the
    range's two ends and in the span's last tile."""
    numels, nd = layout(3)
    M = Mirror(numels, nd)
    S = M.L.S
    rec, ws = zsp.clip_record(), M.plan.norm_workspace()
    zero = [torch.zeros(nd * S, dtype=BF, device="cuda") for _ in range(nd)]
    at = real_mask(M.L, M.ranks, 1, len(numels) - 1)
    for r in range(nd):
        own = at[(at >= r * S) & (at < (r + 1) * S)]
        for i, p in enumerate((own[0], own[-1], own[-1] // TILE * TILE, own[len(own) // 2])):
            g = zero[r].clone()
            g[int(p)] = -3.0 - i
            grads = zero[:r] + [g] + zero[r + 1:]
            for kind, want in (("l2", (3.0 + i) ** 2), ("max", 3.0 + i)):
                M.plan.reduce_shard_norm_params(zsp.ALL_RANKS, 1, len(numels) - 1, grads, rec, ws,
                                                layout="shard", kind=kind)
                assert float(zsp.clip_values(rec)[0]) == want, (r, i, kind)
