"""Short rows with more choices than are in flight at once, some of them not
taken: against binary64, with the tolerances of test_gpu_experts (a dot product
of one turn: a chain of at most 17 products and 9 sums of chains, lanes and
waves, 26 u)."""
import numpy as np
import pytest
import torch

import sharded_state_raggedshard_amd as rs
from gpu_harness import log
from test_gpu_experts import DTYPES, U, Case, check_padding, run_sort

pytestmark = pytest.mark.gpu

# one piece a lane and several, eight slots in flight, and four and two; as many
# tokens as take all their choices in one workgroup, and fewer
SHAPES = [(2100, 264, 64, 17, 1), (2100, 250, 64, 17, 4), (100, 264, 64, 17, 16), (2048, 512, 32, 9, 1), (300, 64, 40, 33, 1),
          (2047, 24, 16, 16, 1), (2100, 1032, 64, 11, 1)]


class SomeTaken(Case):
    """A fifth of the choices not taken, and now and then all of a token's."""

    def __init__(self, rows, hidden, experts, k, align, dtype, gap):
        super().__init__(rows, hidden, experts, k, align, dtype, 4, masked=False, gap=gap)
        rng = np.random.default_rng(17)
        topk = np.stack([rng.permutation(experts)[:k] for _ in range(rows)]).astype(np.int64)
        topk[rng.random((rows, k)) < 0.2] = -1
        topk[5::50] = experts
        self.start, self.count, self.slot = run_sort(topk, None, experts, align)
        self.end = int(self.start[-1])
        self.weight[:, :k] = torch.where(self.slot < 0, float("nan"), torch.rand(rows, k, device="cuda", generator=self.g))
        self.real = torch.zeros(self.slots, dtype=torch.bool, device="cuda")
        self.real[self.slot[self.slot >= 0].long()] = True


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("gap", [0, 5])
def test_there_and_back(shape, dtype, gap):
    log(f"short rows {shape} {dtype} {gap}")
    c = SomeTaken(*shape, dtype, gap)
    n, k, h, ld = c.rows, c.k, c.hidden, c.ld
    taken = (c.slot >= 0)[..., None]
    _, x = c.array(n)
    store, y = c.array(c.slots, fill=3.0)
    rs.rs_expert_dispatch(x, dtype, n, h, ld, c.slot, k, c.weight, k + 1, c.experts, c.start, c.count, y, c.slots, ld)
    check_padding(c, store, y, 3.0)
    expect = torch.where(taken, c.w[..., None] * x.double()[:, None], 0.0)
    assert ((c.picked(y) - expect).abs() <= U * expect.abs() + c.half(expect)).all()
    y.copy_(torch.randn(c.slots, h, device="cuda", generator=c.g))
    y[~c.real] = float("nan")
    picked = c.picked(y)
    _, add = c.array(n)
    for weight in (None, c.weight):
        w = 1.0 if weight is None else c.w[..., None]
        store, out = c.array(n, fill=3.0)
        rs.rs_expert_combine(y, dtype, c.slots, h, ld, c.slot, n, k, weight, k + 1, add, ld, out, ld)
        terms = picked * w
        expect = add.double() + terms.sum(1)
        assert ((out.double() - expect).abs() <= (k + 1) * U * (add.double().abs() + terms.abs().sum(1)) + c.half(expect)).all()
        assert (store[:, h:] == 77).all()
        store, dy = c.array(c.slots, fill=3.0)
        dw = torch.full((n, k + 2), 9.0, device="cuda")
        rs.rs_expert_combine_grad(x, dtype, n, h, ld, y, c.slots, ld, c.slot, k, weight, k + 1, c.experts, c.start, c.count, dy, ld, dw, k + 2)
        check_padding(c, store, dy, 3.0)
        terms = x.double()[:, None] * picked
        assert ((dw[:, :k].double() - terms.sum(-1)).abs() <= 26 * U * terms.abs().sum(-1)).all()
        assert not dw[:, :k][c.slot < 0].any() and (dw[:, k:] == 9).all()
        expect = torch.where(taken, x.double()[:, None] * w, 0.0)
        assert ((c.picked(dy) - expect).abs() <= U * expect.abs() + c.half(expect)).all()
