"""Tokens to experts and back against plain evaluations: the sort and the
copies exactly, the sums against binary64.

Tolerances, u = 2^-24: a token's sum of k products by fused multiply-adds in
binary32 is off by at most (k + 1) u of its absolute terms; a product w dout
by u; a dot product by its longest chain, at most 17 products a turn of a row
and 10 sums of lanes, waves and turns, so 40 u of its absolute terms for the
two turns at most here.  bf16 outputs add half a step, 2^-8 of the value (at
least 2^-134, half the least subnormal)."""
import numpy as np
import pytest
import torch

import sharded_state_raggedshard_amd as rs
from gpu_harness import log

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPE = {rs.RS_F32: torch.float32, rs.RS_BF16: torch.bfloat16}
DTYPES = [rs.RS_F32, rs.RS_BF16]


def sort_of(topk, mask, experts, align):
    """(start, count, slot) in numpy."""
    rows, k = topk.shape
    ids = topk.astype(np.int64).copy()
    taken = (ids >= 0) & (ids < experts)
    if mask is not None:
        taken &= mask[:, None] != 0
    flat = np.where(taken, ids, experts).reshape(-1)
    order = np.argsort(flat, kind="stable")
    count = np.bincount(flat, minlength=experts + 1)[:experts]
    start = np.concatenate([[0], np.cumsum(-(-count // align) * align)])
    slot = np.full(rows * k, -1, dtype=np.int64)
    place = {e: start[e] for e in range(experts)}
    first = np.cumsum(count) - count
    sorted_ids = flat[order]
    live = sorted_ids < experts
    slot[order[live]] = start[sorted_ids[live]] + np.arange(live.sum()) - first[sorted_ids[live]]
    assert len(place) == experts
    return start, count, slot.reshape(rows, k)


def run_sort(topk, mask, experts, align, ldk=None, junk=99):
    rows, k = topk.shape
    ldk = ldk or k
    d = torch.full((max(rows, 1), ldk), 12345, dtype=torch.int64, device="cuda")
    d[:rows, :k] = torch.from_numpy(topk).cuda()
    dm = None if mask is None else torch.from_numpy(mask).cuda()
    start = torch.full((experts + 2,), junk, dtype=torch.int64, device="cuda")
    count = torch.full((experts + 1,), junk, dtype=torch.int32, device="cuda")
    slot = torch.full((rows * k + 1,), junk, dtype=torch.int32, device="cuda")
    nb = rs.rs_expert_sort_bytes(rows, experts, k)
    work = torch.full((nb + 16,), 0xA5, dtype=torch.uint8, device="cuda")
    rs.rs_expert_sort(d, rows, experts, k, ldk, dm, align, start, count, slot, work, nb)
    assert start[-1] == junk and count[-1] == junk and slot[-1] == junk and (work[nb:] == 0xA5).all()
    return start[:-1], count[:-1], slot[:-1].view(rows, k)


@pytest.mark.parametrize("rows,experts,k,align", [
    (0, 4, 2, 1), (1, 1, 1, 1), (1, 256, 8, 128), (16, 32, 4, 1), (63, 7, 3, 16), (64, 64, 1, 2), (1000, 60, 6, 1),
    (1024, 513, 8, 1), (700, 1024, 11, 128), (8191, 128, 1, 4), (8192, 128, 1, 1), (8193, 128, 1, 1), (3000, 1000, 7, 1),
    (5000, 1024, 8, 16), (9001, 60, 6, 128), (65536, 256, 8, 128), (40001, 1, 1, 1), (33333, 2, 2, 3)])
def test_sort(rows, experts, k, align):
    log(f"expert sort {rows} x {k} of {experts}, align {align}")
    rng = np.random.default_rng(rows + experts)
    for kind in ("spread", "one", "strange"):
        topk = rng.integers(0, experts, (rows, k))
        if kind == "one":
            topk[:] = experts - 1
        mask = None
        if kind == "strange":  # ids out of range, the same one twice, rows left out
            topk = rng.integers(-2, experts + 2, (rows, k))
            topk[rng.random((rows, k)) < 0.01] = 1 << 40
            topk[rng.random((rows, k)) < 0.01] = -(1 << 40)
            mask = (rng.random(rows) < 0.7).astype(np.uint8) * 3
        start, count, slot = run_sort(topk, mask, experts, align, ldk=k + 3 if kind == "strange" else None)
        es, ec, ep = sort_of(topk, mask, experts, align)
        assert np.array_equal(start.cpu().numpy(), es), kind
        assert np.array_equal(count.cpu().numpy(), ec), kind
        assert np.array_equal(slot.cpu().numpy(), ep), kind
        assert es[-1] <= rs.rs_expert_slots(rows, experts, k, align)


class Case:
    """Sorted random choices and arrays with junk around the rows."""

    def __init__(self, rows, hidden, experts, k, align, dtype, seed, masked=True, gap=0):
        rng = np.random.default_rng(seed)
        self.rows, self.hidden, self.experts, self.k, self.dtype = rows, hidden, experts, k, dtype
        topk = np.stack([rng.permutation(experts)[:k] for _ in range(rows)]) if rows else np.zeros((0, k), dtype=np.int64)
        mask = (rng.random(rows) < 0.85).astype(np.uint8) if masked else None
        self.start, self.count, self.slot = run_sort(topk.astype(np.int64), mask, experts, align)
        self.end = int(self.start[-1])
        self.slots = rs.rs_expert_slots(rows, experts, k, align) + 2  # two rows behind
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.gap = gap
        self.weight = torch.rand(rows, k + 1, device="cuda", generator=self.g)  # row stride k + 1
        self.weight[:, :k][self.slot < 0] = float("nan")  # weights of choices that are not taken
        real = torch.zeros(self.slots, dtype=torch.bool, device="cuda")
        real[self.slot[self.slot >= 0].long()] = True
        self.real = real

    def array(self, n, fill=None):
        """[n, hidden] rows, `gap` junk columns behind each."""
        store = torch.full((n, self.hidden + self.gap), 77.0, device="cuda", dtype=TYPE[self.dtype])
        x = store[:, :self.hidden]
        if fill is None:
            x.copy_(torch.randn(n, self.hidden, device="cuda", generator=self.g))
        else:
            x.fill_(fill)
        return store, x

    @property
    def ld(self):
        return self.hidden + self.gap

    def half(self, x):
        """Half a step of the output's type."""
        return (2.0 ** -8 * x.abs()).clamp(min=2.0 ** -134) if self.dtype == rs.RS_BF16 else 0.0

    def picked(self, y):
        """Rows of every choice in binary64, 0 for one that is not taken."""
        got = y.double()[self.slot.clamp(min=0).long()]
        return torch.where((self.slot >= 0)[..., None], got, torch.zeros_like(got))

    @property
    def w(self):
        return torch.where(self.slot >= 0, self.weight[:, :self.k].double(), 0.0)


SHAPES = [(0, 64, 8, 2, 4), (1, 1, 1, 1, 1), (1, 2880, 32, 4, 1), (5, 7, 8, 3, 4), (40, 8, 4, 4, 16), (300, 1003, 60, 6, 1),
          (257, 520, 16, 5, 128), (64, 2880, 32, 4, 16), (33, 4100, 8, 2, 1), (20, 8203, 8, 3, 1), (1000, 256, 256, 8, 128),
          (50, 4, 64, 17, 1)]


def check_padding(c, store, x, before):
    """Padding rows 0, rows behind the end and columns behind the rows left."""
    inside = torch.arange(c.slots, device="cuda") < c.end
    assert not x[inside & ~c.real].any()
    assert (x[~inside] == before).all()
    assert (store[:, c.hidden:] == 77).all()


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("gap", [0, 5])
def test_dispatch(shape, dtype, gap):
    log(f"dispatch {shape} {dtype} {gap}")
    c = Case(*shape, dtype, seed=1, gap=gap)
    _, x = c.array(c.rows)
    for weight in (None, c.weight):
        store, y = c.array(c.slots, fill=3.0)
        rs.rs_expert_dispatch(x, dtype, c.rows, c.hidden, c.ld, c.slot, c.k, weight, c.k + 1, c.experts, c.start, c.count, y, c.slots, c.ld)
        check_padding(c, store, y, 3.0)
        got = c.picked(y)
        if weight is None:
            assert torch.equal(got, torch.where((c.slot >= 0)[..., None], x.double()[:, None], 0.0))
        else:
            expect = c.w[..., None] * x.double()[:, None]
            assert ((got - expect).abs() <= U * expect.abs() + c.half(expect)).all()
    # without the segments padding rows stay as they were
    store, y = c.array(c.slots, fill=3.0)
    rs.rs_expert_dispatch(x, dtype, c.rows, c.hidden, c.ld, c.slot, c.k, None, 0, 0, None, None, y, c.slots, c.ld)
    assert (y[~c.real] == 3).all() and (store[:, c.hidden:] == 77).all()


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("gap", [0, 5])
def test_combine(shape, dtype, gap):
    log(f"combine {shape} {dtype} {gap}")
    c = Case(*shape, dtype, seed=2, gap=gap)
    _, y = c.array(c.slots)
    y[~c.real] = float("nan")  # rows of no choice never reach a token
    for weight, added in ((None, False), (c.weight, False), (c.weight, True), (None, True)):
        _, add = c.array(c.rows)
        store, out = c.array(c.rows, fill=3.0)
        rs.rs_expert_combine(y, dtype, c.slots, c.hidden, c.ld, c.slot, c.rows, c.k, weight, c.k + 1, add if added else None, c.ld, out, c.ld)
        terms = c.picked(y) * (1.0 if weight is None else c.w[..., None])
        expect, size = terms.sum(1), terms.abs().sum(1)
        if added:
            expect, size = expect + add.double(), size + add.double().abs()
        assert ((out.double() - expect).abs() <= (c.k + 1) * U * size + c.half(expect)).all()
        assert (store[:, c.hidden:] == 77).all()
        if added:  # in place
            rs.rs_expert_combine(y, dtype, c.slots, c.hidden, c.ld, c.slot, c.rows, c.k, weight, c.k + 1, add, c.ld, add, c.ld)
            assert torch.equal(add, out)


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("gap", [0, 5])
def test_combine_grad(shape, dtype, gap):
    log(f"combine gradient {shape} {dtype} {gap}")
    c = Case(*shape, dtype, seed=3, gap=gap)
    _, dout = c.array(c.rows)
    ystore, y = c.array(c.slots)
    y[~c.real] = float("nan")
    picked = c.picked(y)
    for weight in (c.weight, None):
        store, dy = c.array(c.slots, fill=3.0)
        dw = torch.full((c.rows, c.k + 2), 9.0, device="cuda")
        rs.rs_expert_combine_grad(dout, dtype, c.rows, c.hidden, c.ld, y, c.slots, c.ld, c.slot, c.k, weight, c.k + 1, c.experts, c.start,
                                  c.count, dy, c.ld, dw, c.k + 2)
        check_padding(c, store, dy, 3.0)
        terms = dout.double()[:, None] * picked
        assert ((dw[:, :c.k].double() - terms.sum(-1)).abs() <= 40 * U * terms.abs().sum(-1)).all()
        assert not dw[:, :c.k][c.slot < 0].any() and (dw[:, c.k:] == 9).all()
        expect = torch.where((c.slot >= 0)[..., None], dout.double()[:, None] * (1.0 if weight is None else c.w[..., None]), 0.0)
        assert ((c.picked(dy) - expect).abs() <= U * expect.abs() + c.half(expect)).all()
    # the weights' gradient alone, then in place over y
    dw2 = torch.zeros(c.rows, c.k, device="cuda")
    rs.rs_expert_combine_grad(dout, dtype, c.rows, c.hidden, c.ld, y, c.slots, c.ld, c.slot, c.k, None, 0, 0, None, None, None, 0, dw2, c.k)
    assert torch.equal(dw2, dw[:, :c.k])
    dw2.fill_(5.0)
    rs.rs_expert_combine_grad(dout, dtype, c.rows, c.hidden, c.ld, y, c.slots, c.ld, c.slot, c.k, None, 0, c.experts, c.start, c.count, y, c.ld,
                              dw2, c.k)
    assert torch.equal(dw2, dw[:, :c.k]) and torch.equal(c.picked(y), c.picked(dy))
    assert torch.equal(y[c.real], dy[c.real]) and (ystore[:, c.hidden:] == 77).all()


@pytest.mark.parametrize("shape", [(2500, 40, 1000, 6, 8), (2100, 523, 60, 5, 128), (3, 2880, 700, 8, 256)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_many_tokens_and_many_segments(shape, dtype):
    """More tokens than share workgroups, more experts than are read at once, few tokens with much padding."""
    log(f"many tokens and segments {shape} {dtype}")
    c = Case(*shape, dtype, seed=9, gap=0)
    _, dout = c.array(c.rows)
    _, y = c.array(c.slots)
    store, got = c.array(c.slots, fill=3.0)
    rs.rs_expert_dispatch(dout, dtype, c.rows, c.hidden, c.ld, c.slot, c.k, None, 0, c.experts, c.start, c.count, got, c.slots, c.ld)
    check_padding(c, store, got, 3.0)
    assert torch.equal(c.picked(got), torch.where((c.slot >= 0)[..., None], dout.double()[:, None], 0.0))
    store, dy = c.array(c.slots, fill=3.0)
    dw = torch.full((c.rows, c.k), 9.0, device="cuda")
    rs.rs_expert_combine_grad(dout, dtype, c.rows, c.hidden, c.ld, y, c.slots, c.ld, c.slot, c.k, c.weight, c.k + 1, c.experts, c.start,
                              c.count, dy, c.ld, dw, c.k)
    check_padding(c, store, dy, 3.0)
    terms = dout.double()[:, None] * c.picked(y)
    assert ((dw.double() - terms.sum(-1)).abs() <= 40 * U * terms.abs().sum(-1)).all()
    # a few of the tokens alone: the same bits
    some = min(c.rows, 100)
    dw2 = torch.zeros(some, c.k, device="cuda")
    rs.rs_expert_combine_grad(dout, dtype, some, c.hidden, c.ld, y, c.slots, c.ld, c.slot, c.k, None, 0, 0, None, None, None, 0, dw2, c.k)
    assert torch.equal(dw2, dw[:some])


def test_slots_outside_the_rows_are_not_taken():
    """A sort of more choices than y has rows for, or a slot map of anything."""
    log("slots out of range")
    rows, hidden, k, slots = 20, 100, 3, 40
    slot = torch.arange(rows * k, dtype=torch.int32, device="cuda").view(rows, k)
    slot[3] = torch.tensor([-1, -(1 << 31), (1 << 31) - 1], dtype=torch.int32)
    x = torch.randn(rows, hidden, device="cuda")
    store = torch.zeros(slots + 30, hidden, device="cuda")
    start = torch.tensor([-5, 1 << 60], device="cuda")
    count = torch.tensor([-7], dtype=torch.int32, device="cuda")
    rs.rs_expert_dispatch(x, rs.RS_F32, rows, hidden, hidden, slot, k, None, 0, 1, None, None, store, slots, hidden)
    live = (slot >= 0) & (slot < slots)
    assert torch.equal(store[slot[live].long()], x[:, None].expand(-1, k, -1)[live]) and not store[slots:].any()
    out = torch.zeros_like(x)
    rs.rs_expert_combine(store, rs.RS_F32, slots, hidden, hidden, slot, rows, k, None, 0, None, 0, out, hidden)
    assert torch.allclose(out, x * live.sum(1, keepdim=True), rtol=4 * U)
    dw = torch.ones(rows, k, device="cuda")
    rs.rs_expert_combine_grad(x, rs.RS_F32, rows, hidden, hidden, store, slots, hidden, slot, k, None, 0, 1, None, None, None, 0, dw, k)
    assert not dw[~live].any()
    store[slots:] = 1.0
    rs.rs_expert_dispatch(x, rs.RS_F32, 0, hidden, hidden, slot, k, None, 0, 1, start, count, store, slots, hidden)
    assert not store[:slots].any() and (store[slots:] == 1).all()


@pytest.mark.parametrize("first", [(1 << 63) - 1, -(1 << 63), 39, 40])
def test_padding_of_any_table_stays_inside(first):
    """Starts and counts that no sort wrote: rows of [0, slots) alone change."""
    log(f"padding from {first}")
    slots, hidden = 40, 24
    store = torch.ones(slots + 8, hidden, device="cuda")
    start = torch.tensor([first, (1 << 63) - 1], device="cuda")
    for count in (-(1 << 31), 0, 1, (1 << 31) - 1):
        store.fill_(1.0)
        rs.rs_expert_dispatch(store[:1], rs.RS_F32, 0, hidden, hidden, torch.zeros(1, 1, dtype=torch.int32, device="cuda"), 1, None, 0, 1, start,
                              torch.tensor([count], dtype=torch.int32, device="cuda"), store[4:], slots, hidden)
        assert (store[:4] == 1).all() and (store[4 + slots:] == 1).all()
        used = min(max(first, 0), slots) + max(count, 0)
        assert not store[4 + used:4 + slots].any() and (store[4:4 + min(used, slots)] == 1).all()


def test_gradients_against_differences():
    """dispatch -> a row function -> combine, every gradient by central
    differences of the binary64 definition."""
    log("expert gradients against differences")
    rows, hidden, experts, k = 6, 5, 4, 2
    c = Case(rows, hidden, experts, k, 2, rs.RS_F32, seed=9, masked=False)
    x, gain = torch.randn(rows, hidden, device="cuda"), torch.rand(experts, device="cuda") + 0.5
    w = torch.rand(rows, k, device="cuda")
    dout = torch.randn(rows, hidden, device="cuda")
    of = torch.zeros(c.slots, dtype=torch.long, device="cuda")
    for e in range(experts):
        of[int(c.start[e]):int(c.start[e + 1])] = e

    def loss(x, w):
        y = torch.tanh(x.double()) ** 2
        z = (gain.double()[of[c.slot.long()]] * w.double())[..., None] * y[:, None]
        return (z.sum(1) * dout.double()).sum().item()
    xs = torch.zeros(c.slots, hidden, device="cuda")
    rs.rs_expert_dispatch(x, rs.RS_F32, rows, hidden, hidden, c.slot, k, None, 0, experts, c.start, c.count, xs, c.slots, hidden)
    y = gain[of][:, None] * torch.tanh(xs) ** 2
    dy, dw, dx = torch.zeros_like(y), torch.zeros_like(w), torch.zeros_like(x)
    rs.rs_expert_combine_grad(dout, rs.RS_F32, rows, hidden, hidden, y, c.slots, hidden, c.slot, k, w, k, experts, c.start, c.count, dy, hidden,
                              dw, k)
    dxs = dy * gain[of][:, None] * 2 * torch.tanh(xs) * (1 - torch.tanh(xs) ** 2)
    rs.rs_expert_combine(dxs, rs.RS_F32, c.slots, hidden, hidden, c.slot, rows, k, None, 0, None, 0, dx, hidden)
    h = 1e-4  # the difference's own error is h^2 times a third derivative below 20; binary32 values below 10 add 1e-5
    for value, grad in ((x, dx), (w, dw)):
        v = value.double()
        for i in range(v.numel()):
            up, down = v.clone().view(-1), v.clone().view(-1)
            up[i] += h
            down[i] -= h
            a = (up.view(v.shape), w) if value is x else (x, up.view(v.shape))
            b = (down.view(v.shape), w) if value is x else (x, down.view(v.shape))
            assert abs((loss(*a) - loss(*b)) / (2 * h) - grad.view(-1)[i].item()) <= 2e-5


def test_captured_pass_replays():
    log("experts graph")
    rows, hidden, experts, k, align = 4000, 136, 64, 4, 16
    slots = rs.rs_expert_slots(rows, experts, k, align)
    g = torch.Generator(device="cuda").manual_seed(0)
    x, w = torch.randn(rows, hidden, device="cuda", generator=g), torch.rand(rows, k, device="cuda", generator=g)
    topk = torch.zeros(rows, k, dtype=torch.int64, device="cuda")
    nb = rs.rs_expert_sort_bytes(rows, experts, k)

    def buffers():
        return dict(start=torch.zeros(experts + 1, dtype=torch.int64, device="cuda"), count=torch.zeros(experts, dtype=torch.int32, device="cuda"),
                    slot=torch.zeros(rows, k, dtype=torch.int32, device="cuda"), work=torch.zeros(nb, dtype=torch.uint8, device="cuda"),
                    y=torch.zeros(slots, hidden, device="cuda"), out=torch.zeros(rows, hidden, device="cuda"), dw=torch.zeros(rows, k, device="cuda"))

    def call(b):
        rs.rs_expert_sort(topk, rows, experts, k, k, None, align, b["start"], b["count"], b["slot"], b["work"], nb)
        rs.rs_expert_dispatch(x, rs.RS_F32, rows, hidden, hidden, b["slot"], k, None, 0, experts, b["start"], b["count"], b["y"], slots, hidden)
        rs.rs_expert_combine(b["y"], rs.RS_F32, slots, hidden, hidden, b["slot"], rows, k, w, k, None, 0, b["out"], hidden)
        rs.rs_expert_combine_grad(x, rs.RS_F32, rows, hidden, hidden, b["y"], slots, hidden, b["slot"], k, w, k, experts, b["start"], b["count"],
                                  b["y"], hidden, b["dw"], k)
    a, e = buffers(), buffers()
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        call(a)
    for turn in range(3):
        topk.copy_(torch.rand(rows, experts, device="cuda", generator=g).topk(k).indices)
        for b in (a, e):
            b["y"].zero_()
        graph.replay()
        call(e)
        torch.cuda.synchronize()
        for name in ("start", "count", "slot", "y", "out", "dw"):
            assert torch.equal(a[name], e[name]), (turn, name)


def test_rows_beyond_32_bit_offsets():
    """Sorted rows past element 2^32."""
    log("experts, far rows")
    rows, hidden, experts, k = 76_000, 7168, 16, 8
    slots = rows * k
    assert slots * hidden > 1 << 32
    g = torch.Generator(device="cuda").manual_seed(4)
    topk = torch.rand(rows, experts, device="cuda", generator=g).topk(k).indices
    x = torch.randn(rows, hidden, device="cuda", dtype=torch.bfloat16, generator=g)
    start, count, slot = run_sort(topk.cpu().numpy(), None, experts, 1)
    y = torch.zeros(slots, hidden, device="cuda", dtype=torch.bfloat16)
    rs.rs_expert_dispatch(x, rs.RS_BF16, rows, hidden, hidden, slot, k, None, 0, experts, start, count, y, slots, hidden)
    out, dw = torch.zeros_like(x), torch.zeros(rows, k, device="cuda")
    rs.rs_expert_combine(y, rs.RS_BF16, slots, hidden, hidden, slot, rows, k, None, 0, None, 0, out, hidden)
    assert torch.equal(out, x * 8)
    rs.rs_expert_combine_grad(x, rs.RS_BF16, rows, hidden, hidden, y, slots, hidden, slot, k, None, 0, experts, start, count, y, hidden, dw, k)
    for t in range(0, rows, 997):
        s = x[t].double().square().sum().item()
        assert ((dw[t].double() - s).abs() <= 40 * U * s).all()
        assert torch.equal(y[slot[t].long()], x[t].expand(k, -1))


@pytest.mark.parametrize("dtype", DTYPES)
def test_through_an_expert_layer(dtype):
    """Router to sorted rows to a product per expert over whole tiles and back,
    with every gradient, against autograd in binary64 on a dense layer."""
    log(f"expert layer {dtype}")
    rows, hidden, experts, k, align = 70, 64, 8, 2, 16
    g = torch.Generator(device="cuda").manual_seed(21)
    randn = lambda *n: torch.randn(*n, device="cuda", generator=g)  # noqa: E731
    x, we = randn(rows, hidden).to(TYPE[dtype]), randn(experts, hidden, hidden) / 8
    scores = randn(rows, experts)
    values, topk = torch.topk(scores, k)
    w = torch.softmax(values, -1)
    dout = randn(rows, hidden).to(TYPE[dtype])
    slots = rs.rs_expert_slots(rows, experts, k, align)
    start, count, slot = run_sort(topk.cpu().numpy(), None, experts, align)
    xs = torch.full((slots, hidden), float("nan"), device="cuda", dtype=TYPE[dtype])
    rs.rs_expert_dispatch(x, dtype, rows, hidden, hidden, slot, k, None, 0, experts, start, count, xs, slots, hidden)
    y = torch.zeros_like(xs)
    s = start.tolist()
    for e in range(experts):
        y[s[e]:s[e + 1]] = (xs[s[e]:s[e + 1]].float() @ we[e]).to(y.dtype)
    out = torch.zeros_like(x)
    rs.rs_expert_combine(y, dtype, slots, hidden, hidden, slot, rows, k, w, k, None, 0, out, hidden)
    dy, dw = torch.full_like(xs, float("nan")), torch.zeros_like(w)
    rs.rs_expert_combine_grad(dout, dtype, rows, hidden, hidden, y, slots, hidden, slot, k, w, k, experts, start, count, dy, hidden, dw, k)
    dxs, dwe = torch.zeros_like(xs), torch.zeros_like(we)
    for e in range(experts):  # whole tiles, padding among them
        dxs[s[e]:s[e + 1]] = (dy[s[e]:s[e + 1]].float() @ we[e].T.contiguous()).to(y.dtype)
        dwe[e] = xs[s[e]:s[e + 1]].float().T.contiguous() @ dy[s[e]:s[e + 1]].float()
    dx = torch.zeros_like(x)
    rs.rs_expert_combine(dxs, dtype, slots, hidden, hidden, slot, rows, k, None, 0, None, 0, dx, hidden)
    X, W, WE = (t.double().requires_grad_(True) for t in (x, w, we))
    full = torch.stack([X @ WE[e] for e in range(experts)], 1)
    picked = torch.gather(full, 1, topk[..., None].expand(-1, -1, hidden))
    expect = (W[..., None] * picked).sum(1)
    ex, ew, ewe = torch.autograd.grad((expect * dout.double()).sum(), (X, W, WE))
    # products over 64 values: 64 u of sizes of some 10; bf16 rounds y, dy, dxs and the result: 4 half steps
    step = 4 * 2.0 ** -8 if dtype == rs.RS_BF16 else 64 * U
    for got, want, depth in ((out, expect, 1), (dx, ex, 1), (dw, ew, 8), (dwe, ewe, 8)):
        size = want.detach().abs().max().item() + 1.0
        assert (got.double() - want).abs().max().item() <= step * size * depth
    assert torch.isfinite(dwe).all()
