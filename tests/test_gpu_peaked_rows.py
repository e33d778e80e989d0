"""Rows in which the token holds nearly all the probability: its 1 - p, and
with it its log-probability and its own gradient, keep their digits wherever
the runner-up lies, also in the 16 bytes that hold the token itself.

Tolerances, with u = 2^-24 and R the runner-up's distance over the
temperature: 1 - p is a sum over the other values only, so it is off by an
exponential (3 R + 3) u, at most 10 binary32 additions and 8 rescalings of
(3 R + 3) u, all relative to 1 - p itself: d = (9 (3 R + 3) + 10) u.
log p = -log(1 + rest) is off by d and u of itself for the output; the
token's gradient c (1 - p) by d, the coefficient's error, u for its binary32
form and half a step of the type; another value's -c p_i by (3 R_i + 3 + 4) u,
with its own distance R_i, and half a step.
"""
import numpy as np
import pytest
import torch

import sharded_state_raggedshard_amd as rs
from gpu_harness import log
from test_gpu_objectives import HALF, SENT, TORCH, U, close, np64, work_for

pytestmark = pytest.mark.gpu

TOP = 30.0


def peaked(rows, vocab, dtype, temp, shift, seed):
    """(z on the device, z in binary64, targets): a token of TOP in every row,
    runner-ups 13 to 17 temperatures below it next to the token or anywhere,
    the rest far below or masked."""
    rng = np.random.default_rng(seed)
    x = np.full((rows, vocab), TOP - 80.0 * temp)
    x[1::2] = -np.inf
    y = rng.integers(0, vocab, rows)
    y[0], y[-1] = vocab - 1, 0
    for t in range(rows):
        x[t, y[t]] = TOP
        near = [y[t] + 1, y[t] - 1, y[t] ^ 1, int(rng.integers(0, vocab))][t % 4]
        if near == y[t] or not 0 <= near < vocab:
            near = y[t] - 1 if y[t] else 1
        x[t, near] = TOP - temp * [13.0, 16.0, 17.0][t % 3]
    store = torch.full((shift + rows * vocab + 8,), SENT, dtype=TORCH[dtype])
    store[shift:shift + rows * vocab] = torch.from_numpy(x).to(TORCH[dtype]).reshape(-1)
    z = store.cuda()[shift:shift + rows * vocab].view(rows, vocab)
    return z, np64(z), y


def truth(z64, y, temp):
    """(rest, 1 - p, p, distances): rest = sum of exp((z_i - z_y) / T), i != y."""
    at = np.arange(len(y))
    away = (z64[at, y][:, None] - z64) / temp
    e = np.exp(-away)
    e[at, y] = 0
    rest = e.sum(1)
    return rest, rest / (1 + rest), e / (1 + rest)[:, None], away


def bound(z64, y, temp):
    away = truth(z64, y, temp)[3].copy()
    away[np.arange(len(y)), y] = np.inf
    return (9 * (3 * away.min(1) + 3) + 10) * U


def check(got, z64, y, temp, c, dc, dtype, what):
    """got against c ([i = y] - p) / T; dc: the coefficients' relative error."""
    rest, miss, p, away = truth(z64, y, temp)
    d = bound(z64, y, temp)
    at = np.arange(len(y))
    own = got[at, y]
    close(own, c * miss / temp, (1.01 * (d + dc + U) + HALF[dtype]) * np.abs(c) * miss / temp, what + " of the token")
    others = got.copy()
    others[at, y] = 0
    R = np.minimum(np.where(np.isfinite(away), away, 0), 90)
    tol = (1.01 * ((3 * R + 8) * U + d[:, None] * miss[:, None] + dc) + HALF[dtype]) * np.abs(c)[:, None] * p / temp
    close(others.ravel(), (-c[:, None] * p / temp).ravel(), (tol + 1e-37).ravel(), what)


# rows split over workgroups and not; every workgroup size of the row kernel,
# with the token among the values that stay in registers and behind them
SHAPES = [
    (1, 2, rs.RS_F32, 1.0, 0), (5, 9, rs.RS_BF16, 1.0, 1), (40, 1000, rs.RS_BF16, 1.0, 0),
    (40, 1003, rs.RS_F32, 0.5, 1), (12, 33001, rs.RS_BF16, 1.0, 3), (12, 33000, rs.RS_F32, 1.0, 0),
    (70, 2047, rs.RS_BF16, 1.0, 1), (66, 70001, rs.RS_BF16, 2.0, 0), (66, 120000, rs.RS_F32, 1.0, 0),
    (300, 40003, rs.RS_BF16, 1.0, 0), (300, 9001, rs.RS_F32, 1.0, 1), (2100, 1031, rs.RS_BF16, 1.0, 0),
    (2100, 8111, rs.RS_BF16, 1.0, 1), (2060, 3500, rs.RS_F32, 1.0, 0),
]
IDS = [f"{r}x{v}@{s}-{'f32' if d == rs.RS_F32 else 'bf16'}-T{t}" for r, v, d, t, s in SHAPES]


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_logp_of_a_nearly_certain_token(shape):
    rows, vocab, dtype, temp, shift = shape
    log(f"peaked token_logp {shape}")
    z, z64, y = peaked(rows, vocab, dtype, temp, shift, 81)
    logp, lse = torch.zeros(rows, device="cuda"), torch.zeros(rows, device="cuda")
    work, n = work_for(rows, vocab)
    rs.rs_token_logp(z, dtype, rows, vocab, vocab, torch.from_numpy(y).cuda(), logp, work, n, lse=lse,
                     temperature=temp)
    want = -np.log1p(truth(z64, y, temp)[0])
    close(np64(logp), want, 1.01 * (bound(z64, y, temp) + U) * np.abs(want), "logp")
    close(np64(lse), TOP / temp - want, 1.01 * U * TOP / temp + 1e-9, "lse")


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_policy_gradient_of_a_nearly_certain_token(shape):
    rows, vocab, dtype, temp, shift = shape
    log(f"peaked policy {shape}")
    z, z64, y = peaked(rows, vocab, dtype, temp, shift, 82)
    adv = np.random.default_rng(83).uniform(0.5, 2, rows).astype(np.float32)
    zero, one = torch.zeros(rows, device="cuda"), torch.ones(rows, device="cuda")
    d = torch.full((rows, vocab), SENT, dtype=TORCH[dtype], device="cuda")
    logp, stats = torch.zeros(rows, device="cuda"), torch.zeros(4, device="cuda")
    work, n = work_for(rows, vocab)
    rs.rs_policy_loss(z, dtype, rows, vocab, vocab, torch.from_numpy(y).cuda(), zero, None,
                      torch.from_numpy(adv).cuda(), one, d, vocab, logp, stats, work, n, temperature=temp)
    l = -np.log1p(truth(z64, y, temp)[0])
    close(np64(logp), l, 1.01 * (bound(z64, y, temp) + U) * np.abs(l), "logp")
    # r = exp(l), inside the clipping range: the coefficient's error is l's
    check(np64(d), z64, y, temp, -adv.astype(np.float64) * np.exp(l), bound(z64, y, temp).max() * np.abs(l).max() + 2.0 ** -50,
          dtype, "dlogits")


@pytest.mark.parametrize("shape", [s for s in SHAPES if s[0] >= 4],
                         ids=[i for i, s in zip(IDS, SHAPES) if s[0] >= 4])
def test_preference_gradient_of_nearly_certain_tokens(shape):
    rows, vocab, dtype, temp, shift = shape
    log(f"peaked preference {shape}")
    z, z64, y = peaked(rows, vocab, dtype, temp, shift, 84)
    start = np.array([0, rows // 3, rows // 2, rows // 2 + 1, rows])
    d = torch.full((rows, vocab), SENT, dtype=TORCH[dtype], device="cuda")
    seq, stats = torch.zeros(4, device="cuda"), torch.zeros(3, device="cuda")
    work, n = work_for(rows, vocab, 4)
    rs.rs_preference_loss(z, dtype, rows, vocab, vocab, torch.from_numpy(y).cuda(), torch.from_numpy(start).cuda(),
                          2, None, None, d, vocab, seq, stats, work, n, temperature=temp, beta=0.25)
    l = -np.log1p(truth(z64, y, temp)[0])
    total = np.array([l[a:b].sum() for a, b in zip(start[:-1], start[1:])])
    tol = bound(z64, y, temp).max()
    close(np64(seq), total, 1.01 * (tol + U) * np.abs(total) + 1e-300, "seq_logp")
    h = 0.25 * (total[:2] - total[2:])
    g = 0.5 * 0.25 * -1.0 / (1.0 + np.exp(h))
    c = np.repeat(np.concatenate([g, -g]), np.diff(start))
    dc = 0.25 * tol * np.abs(total).max() * 2 + 2.0 ** -48
    check(np64(d), z64, y, temp, c, dc, dtype, "dlogits")


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("rows,vocab,dtype", [(6, 1, rs.RS_F32), (6, 9, rs.RS_BF16), (6, 40000, rs.RS_F32),
                                              (70, 1003, rs.RS_BF16), (300, 40003, rs.RS_BF16)])
def test_a_token_that_is_not_finite(rows, vocab, dtype, bad):
    """NaN or +inf at the token itself, among finite and among masked values,
    makes its row NaN and no other."""
    log(f"token of {bad} in {rows} x {vocab} dtype={dtype}")
    z, _, y = peaked(rows, max(vocab, 2), dtype, 1.0, 0, 85)
    if vocab == 1:
        z, y = z[:, :1].contiguous(), np.zeros(rows, dtype=y.dtype)
        z[:] = 1.0
    yt = torch.from_numpy(y).cuda()
    zero, one = torch.zeros(rows, device="cuda"), torch.ones(rows, device="cuda")
    work, n = work_for(rows, vocab)

    def call():
        d = torch.full((rows, vocab), SENT, dtype=TORCH[dtype], device="cuda")
        logp, lse, stats = torch.zeros(rows, device="cuda"), torch.zeros(rows, device="cuda"), torch.zeros(4, device="cuda")
        rs.rs_token_logp(z, dtype, rows, vocab, vocab, yt, logp, work, n, lse=lse)
        first = logp.clone()
        rs.rs_policy_loss(z, dtype, rows, vocab, vocab, yt, zero, None, one, one, d, vocab, logp, stats, work, n)
        return d, first, lse, logp, stats

    good = call()
    for t in (2, 3):
        z[t, int(y[t])] = bad
    got = call()
    keep = [t for t in range(rows) if t not in (2, 3)]
    for g, h in zip(got[:4], good):
        assert torch.equal(g[keep], h[keep])
        assert torch.isnan(g[[2, 3]]).all()
    assert torch.isnan(got[4][:2]).all() and not torch.isnan(good[4]).any()
