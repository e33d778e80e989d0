"""Token statistics: log-probabilities to half a step of binary32 where the
sums leave no doubt.

Rows have one value `a` temperatures below the largest, a = 20 and more, and
the rest far below both: ln S = ln(1 + rest), rest < 2^-25, is known to its
last digits, so log p = -a - ln S of the value is off by its own rounding, U =
2^-24 of itself, whatever the temperature (a factor log2(e) / T rounded to
binary32 would take up to U |log p| more), and by 64 U of the rest."""
import math

import numpy as np
import pytest
import torch

import sharded_state_raggedshard_amd as rs
from gpu_harness import log

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPE = {rs.RS_F32: torch.float32, rs.RS_BF16: torch.bfloat16}


def temperatures():
    """1, and those of [0.3, 1.5] whose factor is rounded most, up and down."""
    t = np.linspace(0.3, 1.5, 5001)
    k = 1 / (math.log(2) * t)
    off = k.astype(np.float32).astype(np.float64) / k - 1
    order = np.argsort(off)
    assert off[order[0]] < -0.9 * U and off[order[-1]] > 0.9 * U
    return [1.0, *(float(t[i]) for i in (order[0], order[1], order[-2], order[-1]))]


def run(z, dtype, target, top, temperature):
    rows, vocab = z.shape
    nb = rs.rs_token_stats_bytes(rows, vocab, top)
    work = torch.zeros(nb, dtype=torch.uint8, device="cuda")
    logp = None if target is None else torch.zeros(rows, device="cuda")
    entropy, top_logp = torch.zeros(rows, device="cuda"), torch.zeros(rows, top, device="cuda")
    top_id = torch.zeros(rows, top, dtype=torch.int64, device="cuda")
    rs.rs_token_stats(z, dtype, rows, vocab, vocab, target, logp, entropy, top, top_id if top else None,
                      top_logp if top else None, None, work, nb, temperature=temperature)
    return logp, entropy, top_id, top_logp


SHAPES = [(3, 40), (200, 500), (600, 9000), (8, 40_000), (600, 20_003), (4, 128_256)]


@pytest.mark.parametrize("rows,vocab", SHAPES)
@pytest.mark.parametrize("dtype", [rs.RS_F32, rs.RS_BF16])
def test_any_temperature_keeps_the_last_digit(rows, vocab, dtype):
    log(f"token stats digits {rows} x {vocab} {dtype}")
    g = torch.Generator(device="cuda").manual_seed(vocab)
    for temperature in temperatures():
        a = 22 + 60 * torch.rand(rows, device="cuda", generator=g)
        base = 20 * torch.randn(rows, 1, device="cuda", generator=g)
        z = (base - 150 * temperature).expand(rows, vocab).to(TYPE[dtype]).contiguous()
        at = torch.argsort(torch.rand(rows, vocab, device="cuda", generator=g), dim=1)[:, :2]
        z.scatter_(1, at, torch.cat([base, base - a[:, None] * temperature], 1).to(z.dtype))
        target = at[:, 1].contiguous()
        x = (z.double() - z.double().gather(1, at[:, :1])) / temperature
        rest = torch.exp(x).scatter(1, at[:, :1], 0.0).sum(1)
        assert (rest < 2.0 ** -25).all()
        want = x.gather(1, at[:, 1:])[:, 0] - torch.log1p(rest)
        tol = U * want.abs() + 64 * U * rest
        logp, _, top_id, top_logp = run(z, dtype, target, 2, temperature)
        assert torch.equal(top_id, at)
        assert ((logp.double() - want).abs() <= tol).all(), temperature
        assert ((top_logp[:, 1].double() - want).abs() <= tol).all(), temperature
        # as the log-probability of the training objectives, to a step
        other = torch.zeros(rows, device="cuda")
        nb = rs.rs_objective_bytes(rows, vocab, 0)
        rs.rs_token_logp(z, dtype, rows, vocab, vocab, target, other, torch.zeros(nb, dtype=torch.uint8, device="cuda"), nb,
                         temperature=temperature)
        assert ((other - logp).abs() <= torch.nextafter(logp.abs(), torch.tensor(math.inf, device="cuda")) - logp.abs()).all(), temperature


@pytest.mark.parametrize("rows,vocab", SHAPES)
@pytest.mark.parametrize("dtype", [rs.RS_F32, rs.RS_BF16])
@pytest.mark.parametrize("token", ["none", "another"])
def test_nearly_certain_rows_keep_their_digits_whatever_their_token(rows, vocab, dtype, token):
    """A value 9 to 24 above the rest that is not the row's token: what the
    others weigh, most of it in its neighbours (a thread's same 32 values), is
    known to (3 |x| + 20) U of itself and 2^-51 of 1 + rest, a sum in binary64;
    so are -log p of the value and the entropy, which is rest (1 + mean |x|)."""
    log(f"token stats certain rows {rows} x {vocab} {dtype} token {token}")
    g = torch.Generator(device="cuda").manual_seed(vocab + 1)
    for shift in (0.0, -90.0, 33.0):
        a = 9 + 15 * torch.rand(rows, 3, device="cuda", generator=g)
        z = torch.full((rows, vocab), shift - 70, device="cuda") + torch.randn(rows, vocab, device="cuda", generator=g)
        at = (torch.rand(rows, 1, device="cuda", generator=g) * (vocab // 4 - 1)).long() * 4 + 1
        z.scatter_(1, at, shift + 10.0)
        for i, near in enumerate((-1, 1, 2)):
            z.scatter_(1, at + near, shift + 10.0 - a[:, i:i + 1])
        z = z.to(TYPE[dtype])
        target = None if token == "none" else (at[:, 0] + vocab // 2) % vocab
        x = z.double() - z.double().gather(1, at)
        others = torch.exp(x).scatter(1, at, 0.0)
        rest = others.sum(1)
        assert (rest < 1e-3).all() and (rest > 0).all()
        want, h = -torch.log1p(rest), torch.log1p(rest) - (others * x).sum(1) / (1 + rest)
        rel = (3 * 90 + 20) * U
        logp, entropy, top_id, top_logp = run(z, dtype, target, 2, 1.0)
        assert torch.equal(top_id[:, 0], at[:, 0])
        assert (top_logp <= 0).all() and (entropy >= 0).all()
        assert ((top_logp[:, 0].double() - want).abs() <= rel * rest + 2.0 ** -51).all()
        assert ((entropy.double() - h).abs() <= 2 * rel * h + 2.0 ** -51).all()
        if target is not None:
            own = x.gather(1, target[:, None])[:, 0] + want
            assert ((logp.double() - own).abs() <= U * own.abs() + rel * rest).all()
        # without alternatives the same sums
        assert ((run(z, dtype, target, 0, 1.0)[1].double() - h).abs() <= 2 * rel * h + 2.0 ** -51).all()
