"""Alternatives of rows whose best values are crowded or tie: more of them than
are held reach the bound that the gathering starts from, or few lie above it.
Indexes exactly, values with the tolerances of test_gpu_token_stats."""
import pytest
import torch

import sharded_state_raggedshard_amd as rs
from gpu_harness import log
from test_gpu_token_stats import DTYPES, TYPE, check, run

pytestmark = pytest.mark.gpu

# one wave a row, one workgroup, rows in parts (held and not), odd lengths
SHAPES = [(6, 700), (520, 1500), (300, 5217), (4, 9001), (300, 20_003), (8, 128_256), (2, 201_088), (300, 40_000)]


@pytest.mark.parametrize("rows,vocab", SHAPES)
@pytest.mark.parametrize("dtype", DTYPES)
def test_few_values_above_the_types_lowest(rows, vocab, dtype):
    log(f"few values {rows} x {vocab} {dtype}")
    g = torch.Generator(device="cuda").manual_seed(vocab)
    low = torch.finfo(TYPE[dtype]).min
    for top in (1, 8, 32):
        z = torch.full((rows, vocab), low, device="cuda", dtype=TYPE[dtype])
        for r in range(rows):
            keep = (0, 1, top - 1, top, top + 1, 3 * top, 255, 256, 257, 300)[r % 10]
            at = torch.randperm(vocab, device="cuda", generator=g)[:keep]
            z[r, at] = (torch.randn(keep, device="cuda", generator=g) * 3).to(z.dtype)
        target = torch.randint(0, vocab, (rows,), device="cuda", generator=g)
        target[::3] = -1
        z[torch.arange(rows, device="cuda"), target.clamp(min=0)] = 2.0
        check(z, dtype, target, run(z, dtype, target, top), 1.0, top)
        check(z, dtype, None, run(z, dtype, None, top), 1.0, top)


@pytest.mark.parametrize("rows,vocab", SHAPES)
@pytest.mark.parametrize("dtype", DTYPES)
def test_crowds(rows, vocab, dtype):
    """Values in order, upward and downward, over all of a row or over one half
    of every stretch of 64, 512 or 4096 values, in few steps or many."""
    log(f"crowds {rows} x {vocab} {dtype}")
    g = torch.Generator(device="cuda").manual_seed(vocab + 1)
    i = torch.arange(vocab, device="cuda", dtype=torch.float64)
    z = torch.empty(rows, vocab, device="cuda", dtype=TYPE[dtype])
    for r in range(rows):
        up = (i if r % 2 else vocab - 1 - i) * (8.0 / vocab)
        steps = (1e9, 40.0, 300.0)[r // 2 % 3]
        up = torch.round(up * steps) / steps
        half = (0, 64, 512, 4096)[r // 6 % 4]
        if half:
            up = torch.where(i % half < half // 2, up, -5.0 + 0.1 * torch.randn(vocab, device="cuda", generator=g, dtype=torch.float64))
        z[r] = up.to(z.dtype)
    target = torch.randint(0, vocab, (rows,), device="cuda", generator=g)
    for top in (2, 20, 32):
        check(z, dtype, target, run(z, dtype, target, top), 1.0, top)
