"""Mean probabilities of the router balance loss over so many rows that a
lane's share of a chunk is hundreds of rows: sums over rows keep their
digits whatever their number.

Tolerance of a mean, with u = 2^-24: a share's own (2 e + 34 u, with e = (3 X +
7) u as in test_gpu_router.py, and e + 6 u more for sigmoid scores), at most
64 rows in one binary32 chain, 10 additions that join lanes, and one
rounding each of the chunk's sum and of the output: 76 u.
"""
import numpy as np
import pytest
import torch

import sharded_state_raggedshard_amd as rs
from gpu_harness import log
from test_gpu_objectives import HALF, SENT, TORCH, U, close, np64
from test_gpu_router import SCORES, run

pytestmark = pytest.mark.gpu


def scores_of(z, score):
    if score == "softmax":
        return torch.softmax(z, dim=-1)
    p = torch.sigmoid(z)
    return p / p.sum(-1, keepdim=True)


def share_bound(x, score):
    e = (3 * x + 7) * U
    return 2 * e + 34 * U + (e + 6 * U if score == "sigmoid" else 0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [rs.RS_F32, rs.RS_BF16])
def test_equal_rows(dtype, score):
    """2^26 rows of the same two logits: a chain's error does not average out."""
    log(f"router equal rows dtype={dtype} {score}")
    rows = 1 << 26
    row = torch.tensor([0.125, 0.0], dtype=TORCH[dtype])
    z = row.cuda().expand(rows, 2).contiguous()
    topk = torch.zeros(rows, 1, dtype=torch.int64, device="cuda")
    counts, mean, stats = run(z, dtype, 2, topk, None, None, None, 2, score=SCORES[score][0],
                              balance_coef=1.0)
    p = np64(scores_of(row.double(), score))
    tol = share_bound(0.125, score) + 76 * U
    assert counts.tolist() == [[rows, 0]]
    close(np64(mean)[0], p, 1.01 * tol * p, "mean_prob")
    close(np64(stats), [2 * p[0], 0.0], 1.01 * 2 * p[0] * (tol + 44 * U), "stats")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("rows,experts,dtype", [(4300007, 16, rs.RS_BF16), (270001, 600, rs.RS_F32)])
def test_ragged_chunks_of_many_rows(rows, experts, dtype, score):
    """Shares that are no whole number of chains, over several sequences."""
    log(f"router many rows {rows} x {experts} dtype={dtype} {score}")
    g = torch.Generator(device="cuda").manual_seed(71)
    z = torch.randn(rows, experts, device="cuda", generator=g).to(TORCH[dtype])
    topk = torch.randint(0, experts, (rows, 2), device="cuda", generator=g)
    starts = [3, 1000, rows // 2 + 1, rows - 5]
    d = torch.full((rows, experts), SENT, dtype=TORCH[dtype], device="cuda")
    counts, mean, stats = run(z, dtype, experts, topk, None, torch.tensor(starts, device="cuda"), d,
                              experts, score=SCORES[score][0], balance_coef=0.5)
    assert (d[:3] == SENT).all() and (d[-5:] == SENT).all()
    X = z.abs().max().item()
    balance = 0.0
    for s, (a, b) in enumerate(zip(starts[:-1], starts[1:])):
        p = scores_of(z[a:b].double(), score)
        n = b - a
        c = torch.bincount(topk[a:b].reshape(-1), minlength=experts)
        assert torch.equal(counts[s].long(), c)
        f = c.double() * (experts / (2 * n))
        exp = np64(p.mean(0))
        close(np64(mean[s]), exp, 1.01 * (share_bound(2 * X, score) + 76 * U) * exp, "mean_prob")
        dot = (p @ f)[:, None]
        balance += 0.5 * dot.mean().item()
        slope = p if score == "softmax" else p * torch.sigmoid(-z[a:b].double())
        want = 0.5 / n * slope * (f - dot)
        dp = share_bound(2 * X, score)
        tol = 0.5 / n * slope * ((dp + 4 * U) * (f - dot).abs() + 2 * U * f + (dp + 44 * U) * dot)
        off = (d[a:b].double() - want).abs()
        bad = ~(off <= 1.01 * tol + HALF[dtype] * want.abs() + 1e-37)
        assert not bad.any(), (s, int(bad.sum()), bad.nonzero()[:3].tolist())
    close([stats[0].item()], [balance], 1.01 * (share_bound(2 * X, score) + 45 * U) * balance, "balance")
