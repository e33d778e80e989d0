"""Scratch sizes of the objectives: a workspace sized for a call serves every
smaller one (fewer rows, a shorter vocabulary or fewer experts, fewer
sequences), so a training program keeps the one of its largest micro-batch."""
import random

import pytest

import sharded_state_raggedshard_amd as rs

VOCABS = (1, 1000, 4096, 8191, 8192, 16384, 50000, 65536, 128256, 131072, 201088, 1 << 24)


@pytest.mark.parametrize("vocab", VOCABS)
@pytest.mark.parametrize("n_seq", [0, 2, 64])
def test_objective_bytes_do_not_fall_as_rows_grow(vocab, n_seq):
    last = 0
    for rows in list(range(1, 1400)) + [1 << k for k in range(11, 24)]:
        n = rs.rs_objective_bytes(rows, vocab, n_seq)
        assert n >= last, (rows, vocab, n_seq)
        last = n


@pytest.mark.parametrize("n_seq", [1, 2, 7, 61, 1000])
def test_balance_bytes_do_not_fall_as_rows_grow(n_seq):
    for experts in (1, 32, 256, 1000):
        last = 0
        for rows in list(range(0, 3000)) + list(range(32000, 36000, 7)) + [1 << k for k in range(16, 31)]:
            n = rs.rs_router_balance_bytes(rows, experts, n_seq)
            assert n >= last, (rows, experts, n_seq)
            last = n


def test_smaller_calls_fit_in_any_direction():
    rng = random.Random(5)
    for _ in range(20000):
        rows, vocab, seqs = rng.randrange(1, 3000), rng.choice(VOCABS), 2 * rng.randrange(0, 40)
        most = rs.rs_objective_bytes(rows, vocab, seqs)
        less = (rng.randrange(0, rows + 1), rng.choice([v for v in VOCABS if v <= vocab]), 2 * rng.randrange(0, seqs // 2 + 1))
        assert rs.rs_objective_bytes(*less) <= most, (rows, vocab, seqs, less)
        rows, experts, seqs = rng.randrange(1, 70000), rng.randrange(1, 1025), rng.randrange(1, 400)
        most = rs.rs_router_balance_bytes(rows, experts, seqs)
        less = (rng.randrange(0, rows + 1), rng.randrange(1, experts + 1), rng.randrange(1, seqs + 1))
        assert rs.rs_router_balance_bytes(*less) <= most, (rows, experts, seqs, less)


def test_scratch_stays_small():
    """A few statistics a row, whatever the split."""
    for rows in (1, 64, 512, 5000, 100000):
        assert rs.rs_objective_bytes(rows, 201088, 16) <= 80 * rows + (64 << 10)
        assert rs.rs_router_balance_bytes(rows, 256, 61) <= (1024 + 61) * 256 * 4 + (32 << 10)
