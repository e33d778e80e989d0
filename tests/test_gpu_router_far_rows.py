"""Router balance loss on rows whose scores are all small: sigmoid shares are
s(z) / sum s(z) at every distance from 0, not a softmax's, on both sides of
the sum at which the kernel changes to shares around the maximum.

Tolerances: bounds() of test_gpu_router.py.  Its sigmoid share is off by 2 e
+ 34 u for exponentials and sums and e + 6 u for 1 - s; around the maximum a
share takes one exponential (e), 1 - s once (u, as s <= 2^-10 there) and two
products, which that covers.
"""
import numpy as np
import pytest
import torch

import sharded_state_raggedshard_amd as rs
from gpu_harness import log
from oracle import objectives as ob
from test_gpu_objectives import HALF, SENT, TORCH, close, np64
from test_gpu_router import SCORES, bounds, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [rs.RS_F32, rs.RS_BF16])
@pytest.mark.parametrize("experts", [1, 2, 8, 32, 256, 600])
@pytest.mark.parametrize("centre", [-6.5, -7.5, -9.5, -12.0, -20.0])
def test_rows_far_below_zero(centre, experts, dtype, score):
    log(f"router far rows centre={centre} experts={experts} dtype={dtype} {score}")
    rows, k = 70, min(experts, 2)
    rng = np.random.default_rng(61)
    # rows on either side of the centre: neighbours in a wave differ in kind
    x = rng.normal(centre, 1.0, (rows, experts)) + rng.uniform(-2, 2, (rows, 1))
    x[5] = rng.normal(0, 1, experts)
    z = torch.from_numpy(x).to(TORCH[dtype]).cuda()
    z64 = np64(z)
    topk = np.argsort(-z64, axis=1, kind="stable")[:, :k].copy()
    mask = np.ones(rows, dtype=bool)
    mask[11] = False
    exp = ob.router_balance(z64, topk, mask, [0, rows], balance_coef=0.3, score=SCORES[score][1])
    d = torch.full((rows, experts), SENT, dtype=TORCH[dtype], device="cuda")
    counts, mean, stats = run(z, dtype, experts, torch.from_numpy(topk).cuda(),
                              torch.from_numpy(mask).cuda(), None, d, experts, score=SCORES[score][0],
                              balance_coef=0.3)
    assert np.array_equal(counts.cpu().numpy(), exp["counts"])
    tol_d, tol_m, tol_s = bounds(exp, z64, mask, [0, rows], k, 0.3, 0.0, SCORES[score][1])
    close(np64(mean).ravel(), exp["mean_prob"].ravel(), tol_m.ravel(), "mean_prob")
    close(np64(stats), exp["stats"], tol_s, "stats")
    close(np64(d).ravel(), exp["dlogits"].ravel(),
          (tol_d + HALF[dtype] * np.abs(exp["dlogits"]) + 1e-37).ravel(), "dlogits")


@pytest.mark.parametrize("dtype", [rs.RS_F32, rs.RS_BF16])
@pytest.mark.parametrize("masked", [False, True])
def test_infinite_sigmoid_scores(dtype, masked):
    """s(+inf) = 1, as s(80) is to 115 bits: same shares, no gradient at the
    expert itself; with a masked row in the wave too (its other way of
    taking rows)."""
    log(f"router infinite scores dtype={dtype} masked={masked}")
    rows, experts, k = 40, 48, 2
    g = torch.Generator(device="cuda").manual_seed(62)
    z = torch.randn(rows, experts, device="cuda", generator=g).to(TORCH[dtype])
    topk = torch.randint(0, experts, (rows, k), device="cuda", generator=g)
    mask = np.ones(rows, dtype=bool)
    mask[3::8] = not masked
    z[1, 5] = z[2, 7] = z[2, 9] = z[30, 0] = 80.0
    z64 = np64(z)
    z[z == 80] = float("inf")
    exp = ob.router_balance(z64, topk.cpu().numpy(), mask, [0, rows], balance_coef=0.3, score=ob.NORMALISED_SIGMOID)
    d = torch.full((rows, experts), SENT, dtype=TORCH[dtype], device="cuda")
    counts, mean, stats = run(z, dtype, experts, topk, torch.from_numpy(mask).cuda(), None, d, experts,
                              score=rs.RS_SCORE_SIGMOID, balance_coef=0.3)
    tol_d, tol_m, tol_s = bounds(exp, z64, mask, [0, rows], k, 0.3, 0.0, ob.NORMALISED_SIGMOID)
    close(np64(mean).ravel(), exp["mean_prob"].ravel(), tol_m.ravel(), "mean_prob")
    close(np64(stats), exp["stats"], tol_s, "stats")
    close(np64(d).ravel(), exp["dlogits"].ravel(),
          (tol_d + HALF[dtype] * np.abs(exp["dlogits"]) + 1e-37).ravel(), "dlogits")
    assert not d[torch.isinf(z)].any()
