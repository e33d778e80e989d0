"""AdamW with an eps out of the ordinary.  Tolerance: 1e-8 + 1e-6 |theta|, what
the step may differ by from correctly rounded operations, and the roundings of
the moments: m and v carry at most 5 and 8 u (u = 2^-24) of their terms, a
subnormal v half of 2^-149 a product, three of them."""
import math

import pytest
import torch

import sharded_state_raggedshard_amd as rs
from gpu_harness import log
from synth import ROWS, TensorSpec

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.mark.parametrize("eps,top_v,top_m", [
    (1e-30, 1e-38, 1e-30), (1e-26, 1e-38, 1e-26), (1e-22, 1e-38, 1e-22), (1e-20, 1e-38, 1e-20), (0.0, 1e-38, 1e-20),
    (1e-16, 1e-38, 1e-16), (1e-12, 1e-36, 1e-12), (1e-8, 1e-36, 1e-8), (3e38, 1e30, 1e38)])
@pytest.mark.parametrize("state", [rs.RS_STATE_F32, rs.RS_STATE_INT8])
def test_against_binary64(eps, top_v, top_m, state):
    """Second moments on both sides of 2^-126 = 1.2e-38."""
    log(f"adamw eps {eps} state {state}")
    n, block = 4096 + 77, 64
    g = torch.Generator(device="cuda").manual_seed(5)
    rand = lambda: torch.rand(n, device="cuda", generator=g, dtype=torch.float64)  # noqa: E731
    v0 = top_v * 10.0 ** (-5 * rand())
    m0 = top_m * (rand() - 0.5)
    params = torch.zeros(n, device="cuda")
    grads = torch.zeros(n, device="cuda")
    if state == rs.RS_STATE_F32:
        m, v, amax = m0.float(), v0.float(), [[None], [None]]
        m0, v0 = m.double(), v.double()
    else:
        # one size a block, the codes of the moments all near their tops
        nb = -(-n // block)
        am, av = (top_m * torch.ones(nb, device="cuda")).float(), v0[::block].float()
        m = (rand() * 254 - 127).round().to(torch.int8)
        v = (200 + rand() * 55).round().to(torch.uint8)
        amax = [[am], [av]]
        spread = lambda x: x.double().repeat_interleave(block)[:n]  # noqa: E731
        m0, v0 = m.double() / 127 * spread(am), v.double() / 255 * spread(av)
    h = rs.AdamW([(n, rs.RS_F32, rs.RS_F32, state, block if state else 0, 0)]).upload()
    h.bind([params], [grads], [m], [v], *amax)
    hp = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=eps, weight_decay=0.0, step=400)
    m1, v1 = 0.9 * m0, 0.999 * v0
    size, kappa = 1e-3 / (1 - 0.9 ** 400), 1 / math.sqrt(1 - 0.999 ** 400)
    den = v1.sqrt() * kappa + float(torch.tensor(eps, dtype=torch.float32))
    want = -size * m1 / den
    h.step([hp])
    # 3 2^-150 in v: sqrt's slope is 1 / (2 sqrt v)
    off_v = (10 * U * v1 + 4 * 2.0 ** -150) / (2 * v1.sqrt()) * kappa / den
    off_m = (7 * U * m1.abs() + 3 * 2.0 ** -150) / den
    tol = 1e-8 + 1e-6 * want.abs() + want.abs() * off_v + size * off_m
    assert ((params.double() - want).abs() <= tol).all()
    assert top_v != 1e-38 or (v1 < 2.0 ** -126).any()
    h.free()


@pytest.mark.parametrize("eps,top_v,top_m", [(1e-30, 1e-38, 1e-30), (1e-16, 1e-38, 1e-16), (1e-8, 1e-36, 1e-8), (3e38, 1e30, 1e38)])
def test_the_planned_step_against_binary64(eps, top_v, top_m):
    """Blocks of 256 as rows of a planned tensor; tolerances as above."""
    log(f"planned step eps {eps}")
    rows, block = 41, 256
    n = rows * block
    plan = rs.Plan([TensorSpec("w", (rows, block), ROWS, 1)], 1, 16).upload()
    g = torch.Generator(device="cuda").manual_seed(6)
    am = torch.full((rows,), top_m, device="cuda")
    av = (top_v * 10.0 ** (-5 * torch.rand(rows, device="cuda", generator=g, dtype=torch.float64))).float()
    qm, qv = torch.zeros(plan.total, dtype=torch.int8, device="cuda"), torch.zeros(plan.total, dtype=torch.uint8, device="cuda")
    here = slice(plan.pos[0], plan.pos[0] + n)
    qm[here] = torch.randint(-127, 128, (n,), device="cuda", generator=g).to(torch.int8)
    qv[here] = torch.randint(200, 256, (n,), device="cuda", generator=g).to(torch.uint8)
    params = torch.zeros(plan.total, device="cuda")
    spread = lambda x: x.double().repeat_interleave(block)  # noqa: E731
    m1 = 0.9 * (qm[here].double() / 127 * spread(am))
    v1 = 0.999 * (qv[here].double() / 255 * spread(av))
    size, kappa = 1e-3 / (1 - 0.9 ** 400), 1 / math.sqrt(1 - 0.999 ** 400)
    den = v1.sqrt() * kappa + float(torch.tensor(eps, dtype=torch.float32))
    want = -size * m1 / den
    off_v = (10 * U * v1 + 4 * 2.0 ** -150) / (2 * v1.sqrt()) * kappa / den
    off_m = (7 * U * m1.abs() + 3 * 2.0 ** -150) / den
    rs.rs_adam8_step(plan.h, rs.RS_ALL, rs.RS_ALL, params, torch.zeros(plan.total, dtype=torch.int16, device="cuda"), qm, qv, am, av,
                     lr=1e-3, beta1=0.9, beta2=0.999, eps=eps, weight_decay=0.0, step=400)
    tol = 1e-8 + 1e-6 * want.abs() + want.abs() * off_v + size * off_m
    assert ((params[here].double() - want).abs() <= tol).all()
    plan.free()
