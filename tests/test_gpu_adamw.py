"""AdamW over many tensors against a plain evaluation in binary64.

Tolerances, u = 2^-24 (half a step of binary32): m = b1 m0 + w1 g is two
products and a sum of rounded scalars and a g scaled in binary32, so off by at
most 5 u of its absolute terms (7 u where m0 is a code's value: a quotient and
a product more); v likewise with g g, 8 u and 10 u.  The step lr' m / (sqrt(v)
kappa + eps) carries m's error, half of v's (at most 5 u), and at most 10 u of
its own (scalars, product, sum, root, reciprocal, two products); the new
parameter two roundings of its terms.  bf16 outputs add half a step, 2^-8 of
the value.  A code is at most one off, and only where the value in binary64
lies within its error of the border between two codes."""
import math

import pytest
import torch

import sharded_state_raggedshard_amd as rs
from gpu_harness import log
from synth import ROWS, TensorSpec

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F32, BF16 = rs.RS_F32, rs.RS_BF16
TYPE = {F32: torch.float32, BF16: torch.bfloat16}
HP = dict(lr=1e-2, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.1, step=7)
SIZES = [1, 3, 4, 5, 0, 63, 64, 255, 257, 1023, 4095, 4096, 4097, 9001]


class Store:
    """Arrays carved out of one byte store, `gap` bytes around each, so that
    they start anywhere their elements may and what lies between is seen."""

    def __init__(self, nbytes):
        self.bytes = torch.full((nbytes,), 0x5A, dtype=torch.uint8, device="cuda")
        self.at = 0
        self.used = torch.zeros(nbytes, dtype=torch.bool, device="cuda")

    def take(self, x, gap):
        size = x.element_size()
        self.at = -(-(self.at + gap) // size) * size
        n = x.numel() * size
        if self.at % 16 == 0 and gap % 16:
            self.at += size
        raw = self.bytes[self.at:self.at + n]
        self.used[self.at:self.at + n] = True
        self.at += n
        view = raw.view(x.dtype)
        view.copy_(x)
        return view

    def intact(self):
        return bool((self.bytes[~self.used] == 0x5A).all())


def make(tensors, seed, aligned, out):
    """(plan, dict of lists) with random arrays for the tensors."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda n: torch.rand(n, device="cuda", generator=g)  # noqa: E731
    store = Store(sum(t[0] for t in tensors) * 24 + 400 * len(tensors) + 4096)
    gap = 16 if aligned else 5
    a = {name: [] for name in ("params", "grads", "m", "v", "amax_m", "amax_v", "bf16_out")}
    for numel, p, gr, state, block, _ in tensors:
        a["params"].append(store.take((rand(numel) - 0.5).to(TYPE[p]), gap))
        a["grads"].append(store.take(((rand(numel) - 0.5) * 1e-2).to(TYPE[gr]), gap))
        if state == rs.RS_STATE_INT8:
            nb = -(-numel // block)
            a["m"].append(store.take((rand(numel) * 255).floor().sub(127).to(torch.int8), gap))
            a["v"].append(store.take((rand(numel) * 256).floor().clamp(max=255).to(torch.uint8), gap))
            a["amax_m"].append(store.take(rand(nb) * 1e-2, gap))
            a["amax_v"].append(store.take(rand(nb) * 1e-4, gap))
        else:
            a["m"].append(store.take((rand(numel) - 0.5) * 1e-2, gap))
            a["v"].append(store.take(rand(numel) * 1e-4, gap))
            a["amax_m"].append(None)
            a["amax_v"].append(None)
        a["bf16_out"].append(store.take(torch.zeros(numel, dtype=torch.bfloat16, device="cuda"), gap)
                             if out and p == F32 else None)
    h = rs.AdamW(tensors).upload().bind(**a)
    return h, a, store


def clone(a):
    return {k: [None if x is None else x.clone() for x in v] for k, v in a.items()}


def spread(amax, block, numel):
    return amax.double().repeat_interleave(block)[:numel]


def check(tensors, before, after, hps, s, what):
    for i, (numel, p, _, state, block, group) in enumerate(tensors):
        if numel == 0:
            continue
        hp = hps[group]
        name = f"{what}: tensor {i} of {numel}"
        b1, b2, t = hp["beta1"], hp["beta2"], hp["step"]
        g = before["grads"][i].double() * s
        m0, v0 = before["m"][i].double(), before["v"][i].double()
        eight = state == rs.RS_STATE_INT8
        if eight:
            m0 = m0 * spread(before["amax_m"][i], block, numel) / 127
            v0 = v0 * spread(before["amax_v"][i], block, numel) / 255
        m, v = b1 * m0 + (1 - b1) * g, b2 * v0 + (1 - b2) * g * g
        em = (7 if eight else 5) * U * (b1 * m0.abs() + (1 - b1) * g.abs())
        ev = (10 if eight else 8) * U * (b2 * v0 + (1 - b2) * g * g)
        size, kappa = hp["lr"] / (1 - b1 ** t), 1 / math.sqrt(1 - b2 ** t)
        den = v.sqrt() * kappa + hp["eps"]
        step = size * m / den
        th0 = before["params"][i].double()
        th = th0 * (1 - hp["lr"] * hp["weight_decay"]) - step
        tol = abs(size) * em / den + 15 * U * step.abs() + 3 * U * (th0.abs() + step.abs())
        got = after["params"][i].double()
        extra = 2.0 ** -8 * th.abs() if p == BF16 else 0.0
        assert ((got - th).abs() <= tol + extra).all(), name
        if after["bf16_out"][i] is not None:
            assert torch.equal(after["bf16_out"][i], after["params"][i].bfloat16()), name
        if not eight:
            assert ((after["m"][i].double() - m).abs() <= em).all(), name
            assert ((after["v"][i].double() - v).abs() <= ev).all(), name
            continue
        pad = -numel % block
        fold = lambda x: torch.nn.functional.pad(x, (0, pad)).view(-1, block)  # noqa: E731
        for x, e, levels, code, amax in ((m, em, 127, after["m"][i], after["amax_m"][i]),
                                         (v, ev, 255, after["v"][i], after["amax_v"][i])):
            top = fold(x.abs()).amax(1)
            err = fold(e).amax(1)
            assert ((amax.double() - top).abs() <= err).all(), name
            at = spread(top, block, numel)
            ideal = torch.where(at > 0, x / at * levels, torch.zeros_like(x))
            slack = torch.where(at > 0, (e + spread(err, block, numel)) / at * levels + 4 * U * levels, torch.zeros_like(x))
            assert ((code.double() - ideal).abs() <= 0.5 + slack).all(), name


KINDS = [(p, g, st) for p in (F32, BF16) for g in (F32, BF16) for st in (0, 64, 256, 512, 1024, 2048, 4096)]


@pytest.mark.parametrize("p,g,block", KINDS)
@pytest.mark.parametrize("aligned", [True, False])
def test_step_against_binary64(p, g, block, aligned):
    log(f"adamw {p} {g} block {block} aligned {aligned}")
    state = rs.RS_STATE_INT8 if block else rs.RS_STATE_F32
    tensors = [(n, p, g, state, block, i % 2) for i, n in enumerate(SIZES)]
    h, a, store = make(tensors, 3 + block, aligned, out=True)
    hps = [HP, {**HP, "lr": 3e-2, "beta1": 0.8, "beta2": 0.95, "weight_decay": 0.0, "eps": 1e-6, "step": 1}]
    scale = torch.tensor([0.37], device="cuda")
    for s in (None, scale):
        before = clone(a)
        h.step(hps, grad_scale=s)
        check(tensors, before, a, hps, 1.0 if s is None else s.double().item(), f"scale {s}")
    assert store.intact()
    h.free()


def test_tensors_of_all_kinds_in_one_step():
    log("adamw all kinds at once")
    tensors = [(n, p, g, rs.RS_STATE_INT8 if b else rs.RS_STATE_F32, b, j % 3)
               for j, (p, g, b) in enumerate(KINDS) for n in (1, 700, 5000)]
    h, a, store = make(tensors, 5, False, out=False)
    hps = [HP, {**HP, "beta2": 0.9}, {**HP, "lr": -1e-3, "step": 1000}]
    before = clone(a)
    h.step(hps)
    check(tensors, before, a, hps, 1.0, "all kinds")
    assert store.intact()
    h.free()


@pytest.mark.parametrize("block", [64, 256])
def test_codes_equal_the_planned_step_bit_for_bit(block):
    """Rows of one block each, m = 1: the planned buffer holds the tensor whole."""
    log(f"adamw against the planned step, block {block}")
    rows = 37
    spec = TensorSpec("w", (rows, block), ROWS, 1)
    plan = rs.Plan([spec], 1, 16).upload()
    n = rows * block
    t = (n, F32, BF16, rs.RS_STATE_INT8, block, 0)
    h, a, _ = make([t], 11, True, out=True)
    planned = {k: torch.zeros(plan.total, dtype=v[0].dtype, device="cuda") for k, v in a.items() if k[:4] != "amax"}
    at = plan.pos[0]
    for k, x in planned.items():
        x[at:at + n] = a[k][0]
    am, av = a["amax_m"][0].clone(), a["amax_v"][0].clone()
    assert plan.n_blocks == rows
    scale = torch.tensor([0.5], device="cuda")
    for step in (7, 8, 9):
        hp = {**HP, "lr": 1e-3, "step": step}
        rs.rs_adam8_step(plan.h, rs.RS_ALL, rs.RS_ALL, planned["params"], planned["grads"], planned["m"], planned["v"], am, av,
                         **hp, grad_scale=scale, bf16_out=planned["bf16_out"])
        h.step([hp], grad_scale=scale)
        for k, x in planned.items():
            assert torch.equal(x[at:at + n], a[k][0]), (step, k)
        assert torch.equal(am, a["amax_m"][0]) and torch.equal(av, a["amax_v"][0])
    plan.free()
    h.free()


@pytest.mark.parametrize("block", [0, 64, 4096])
def test_zero_gradients_and_states(block):
    """No gradient ever: a pure decay, and states that stay 0."""
    log(f"adamw zeros, block {block}")
    t = (5000, F32, BF16, rs.RS_STATE_INT8 if block else rs.RS_STATE_F32, block, 0)
    h, a, _ = make([t], 1, False, out=False)
    for k in ("grads", "m", "v", "amax_m", "amax_v"):
        if a[k][0] is not None:
            a[k][0].zero_()
    th = a["params"][0].clone()
    h.step([HP])
    decay = torch.tensor(1 - HP["lr"] * HP["weight_decay"], dtype=torch.float64).float()
    assert torch.equal(a["params"][0], th * decay.cuda())
    for k in ("m", "v", "amax_m", "amax_v"):
        assert a[k][0] is None or not a[k][0].any()
    h.free()


def test_tiny_and_subnormal_blocks():
    """Blocks whose absmax is below 2^-60 take the plain division; zeros among
    others stay 0."""
    log("adamw tiny blocks")
    t = (256, F32, F32, rs.RS_STATE_INT8, 64, 0)
    h, a, _ = make([t], 2, True, out=False)
    for k in ("m", "v"):
        a[k][0].zero_()
    g = torch.linspace(-1, 1, 256, device="cuda")
    g[:64] *= 1e-25
    g[64:128] = 0
    g[128] = 1e-12
    a["grads"][0].copy_(g)
    before = clone(a)
    h.step([{**HP, "beta1": 0.0, "step": 1}])
    hp = {**HP, "beta1": 0.0, "step": 1}
    m = a["m"][0].double() * spread(a["amax_m"][0], 64, 256) / 127
    # a code's value is within half a level of the gradient; below 2^-126 a gradient's own rounding counts
    level = spread(a["amax_m"][0], 64, 256) / 127
    assert ((m - before["grads"][0].double()).abs() <= 0.5 * level * (1 + 1e-5) + 2.0 ** -149).all()
    assert not a["m"][0][64:128].any()
    assert hp["step"] == 1
    h.free()


@pytest.mark.parametrize("g", [F32, BF16])
def test_norm_and_coefficient(g):
    log(f"adamw norm {g}")
    tensors = [(n, F32, g, rs.RS_STATE_F32, 0, 0) for n in SIZES + [100_003]]
    h, a, store = make(tensors, 9, False, out=False)
    sumsq, scale = torch.zeros(1, dtype=torch.float64, device="cuda"), torch.zeros(1, device="cuda")
    exact = sum(x.double().square().sum() for x in a["grads"]).item()
    for max_norm in (1e-3, 1e3):
        h.l2norm_clip(max_norm, sumsq, scale)
        # binary64 sums of N positive terms: N 2^-53 at most
        assert abs(sumsq.item() - exact) <= 2e5 * 2.0 ** -53 * exact
        expect = torch.zeros(1, device="cuda")
        rs.rs_clip_coef(sumsq, max_norm, expect)
        assert scale.item() == expect.item()
    first = sumsq.item()
    h.l2norm_clip(1.0, sumsq)  # no coefficient
    assert sumsq.item() == first
    for bad in (float("inf"), float("nan")):
        a["grads"][7][0] = bad
        h.l2norm_clip(1.0, sumsq, scale)
        assert (math.isinf if math.isinf(bad) else math.isnan)(sumsq.item())
        assert scale.item() == 0.0 if math.isinf(bad) else math.isnan(scale.item())
    assert store.intact()
    h.free()


def test_a_bad_gradient_stays_in_its_tensor():
    log("adamw NaN gradient")
    tensors = [(n, F32, F32, st, b, 0) for n in (100, 5000) for st, b in ((0, 0), (1, 64))]
    h, a, store = make(tensors, 4, False, out=True)
    before = clone(a)
    for x in (a["grads"][0], a["grads"][3]):
        x[37] = float("nan")
        x[38] = float("inf")
    h.step([HP])
    for i in (1, 2):
        check([tensors[i]], {k: [v[i]] for k, v in before.items()}, {k: [v[i]] for k, v in a.items()}, [HP], 1.0, "others")
    assert torch.isnan(a["params"][0][37]) and store.intact()
    h.free()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_moments_as_values(dtype):
    log(f"adamw moments {dtype}")
    tensors = [(n, F32, F32, rs.RS_STATE_INT8 if b else rs.RS_STATE_F32, b, 0) for n in SIZES for b in (0, 64, 1024)]
    h, a, store = make(tensors, 6, False, out=False)
    total = sum(t[0] for t in tensors)
    m, v = (torch.full((total + 3,), 7.0, dtype=TYPE[dtype], device="cuda") for _ in range(2))
    # bf16 from an address that is no multiple of 16 bytes
    h.moments(m[1:total + 1], None, dtype)
    h.moments(None, v[1:total + 1], dtype)
    at = 1
    for i, (n, _, _, _, b, _) in enumerate(tensors):
        for got, code, amax, levels in ((m, a["m"][i], a["amax_m"][i], 127), (v, a["v"][i], a["amax_v"][i], 255)):
            x = code.float()
            if b:
                x = (code.double() / levels).float() * amax.repeat_interleave(b)[:n]
            assert torch.equal(got[at:at + n], x.to(TYPE[dtype])), (i, n, b)
        at += n
    assert (m[[0, -2, -1]] == 7).all() and (v[[0, -2, -1]] == 7).all() and store.intact()
    h.free()


def test_bound_arrays_are_not_outputs():
    log("adamw refusals of bound arrays")
    h, a, _ = make([(1000, F32, BF16, rs.RS_STATE_F32, 0, 0)], 8, True, out=False)
    for bad in (lambda: h.step([HP], grad_scale=a["m"][0][:1]), lambda: h.moments(a["grads"][0], None, BF16),
                lambda: h.l2norm_clip(1.0, a["v"][0].view(torch.uint8)[:8].view(torch.float64)),
                lambda: h.moments(h.workspace.view(torch.float32), None)):
        with pytest.raises(rs.RaggedShardError) as e:
            bad()
        assert e.value.status == rs.RS_EINVAL
    h.free()


def test_captured_step_replays_and_follows_a_new_binding():
    log("adamw graph")
    tensors = [(n, F32, BF16, rs.RS_STATE_INT8 if n % 2 else rs.RS_STATE_F32, 64 if n % 2 else 0, 0) for n in SIZES]
    h, a, _ = make(tensors, 12, False, out=True)
    e, b, _ = make(tensors, 12, False, out=True)
    state = {k: [torch.zeros(1, dtype=torch.float64, device="cuda"), torch.zeros(1, device="cuda")] for k in "he"}
    total = sum(SIZES)
    out = {k: [torch.zeros(total, device="cuda") for _ in range(2)] for k in "he"}

    def call(o, key):
        o.l2norm_clip(1e-2, *state[key])
        o.step([HP], grad_scale=state[key][1])
        o.moments(*out[key])
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        call(h, "h")
    other = [x.clone().mul_(-0.5) for x in a["grads"]]
    for turn in range(4):
        if turn == 2:  # gradients that have moved
            for o, lists in ((h, a), (e, b)):
                lists["grads"] = [x.clone() for x in other]
                o.bind(**lists)
        graph.replay()
        call(e, "e")
        torch.cuda.synchronize()
        for k in a:
            for x, y in zip(a[k], b[k]):
                assert x is None or torch.equal(x, y), (turn, k)
        assert state["h"][0].item() == state["e"][0].item() and torch.equal(out["h"][0], out["e"][0])
    h.free()
    e.free()


def test_on_another_stream():
    log("adamw on a stream of its own")
    t = [(50_000, F32, F32, rs.RS_STATE_F32, 0, 0)]
    h, a, _ = make(t, 13, True, out=False)
    before = clone(a)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        torch.cuda._sleep(20_000_000)
        a["grads"][0].mul_(2.0)
        h.step([HP])
    torch.cuda.current_stream().wait_stream(stream)
    check(t, {**before, "grads": [before["grads"][0] * 2]}, a, [HP], 1.0, "stream")
    h.free()


@pytest.mark.parametrize("block,numel", [(0, (1 << 30) + 4099), (4096, (1 << 31) + 4099)])
def test_offsets_beyond_32_bits(block, numel):
    """Byte offsets of binary32 moments pass 2^32, element offsets 2^31."""
    log(f"adamw {numel} elements, block {block}")
    state = rs.RS_STATE_INT8 if block else rs.RS_STATE_F32
    t = (numel, BF16, BF16, state, block, 0)
    dev = dict(device="cuda")
    a = dict(params=[torch.full((numel,), 0.5, dtype=torch.bfloat16, **dev)],
             grads=[torch.full((numel,), 1e-3, dtype=torch.bfloat16, **dev)],
             m=[torch.zeros(numel, dtype=torch.int8 if block else torch.float32, **dev)],
             v=[torch.zeros(numel, dtype=torch.uint8 if block else torch.float32, **dev)],
             amax_m=[torch.zeros(-(-numel // block), **dev) if block else None],
             amax_v=[torch.zeros(-(-numel // block), **dev) if block else None], bf16_out=[None])
    where = [0, 4096, numel // 2 // 4096 * 4096, numel - 4099, numel - 1]
    for i, w in enumerate(where):
        a["grads"][0][w:w + 3] = 1e-2 * (i + 1)
    h = rs.AdamW([t]).upload().bind(**a)
    hp = {**HP, "step": 1}
    h.step([hp])
    for w in where:
        lo = w // 4096 * 4096
        hi = min(lo + 4096, numel)
        n = hi - lo
        part = {k: [None if x[0] is None else x[0][lo // 4096:lo // 4096 + 1] if k[:4] == "amax" else x[0][lo:hi]] for k, x in a.items()}
        before = dict(params=[torch.full((n,), 0.5, dtype=torch.bfloat16, **dev)], grads=part["grads"],
                      m=[torch.zeros(n, **dev)], v=[torch.zeros(n, **dev)], amax_m=[torch.zeros(1, **dev)], amax_v=[torch.zeros(1, **dev)])
        check([(n, BF16, BF16, state, block, 0)], before, part, [hp], 1.0, f"at {w}")
    h.free()


ROOT = rs.RS_STATE_INT8_ROOT


@pytest.mark.parametrize("block", [64, 256, 1024, 4096])
@pytest.mark.parametrize("p,g", [(F32, BF16), (BF16, F32)])
def test_root_codes_against_binary64(block, p, g):
    """The second moment by its root: v0 = (q / 255)^2 amax takes two products
    and a quotient more (2 u), the rest as above; the root of a quotient off by
    r of itself is off by r / 2, and a u more."""
    log(f"adamw root codes {block} {p} {g}")
    for aligned in (True, False):
        tensors = [(n, p, g, ROOT, block, i % 2) for i, n in enumerate(SIZES)]
        as_codes = [(n, p, g, rs.RS_STATE_INT8, block, i % 2) for i, n in enumerate(SIZES)]
        h, a, store = make(as_codes, 40 + block, aligned, out=True)
        h.free()
        h = rs.AdamW(tensors).upload().bind(**a)
        hps = [HP, {**HP, "beta2": 0.95, "weight_decay": 0.0, "step": 1}]
        for turn in range(2):
            before = clone(a)
            h.step(hps)
            for i, (numel, _, _, _, _, group) in enumerate(tensors):
                if numel == 0:
                    continue
                hp = hps[group]
                b1, b2, t = hp["beta1"], hp["beta2"], hp["step"]
                gr = before["grads"][i].double()
                m0 = before["m"][i].double() * spread(before["amax_m"][i], block, numel) / 127
                v0 = (before["v"][i].double() / 255) ** 2 * spread(before["amax_v"][i], block, numel)
                m, v = b1 * m0 + (1 - b1) * gr, b2 * v0 + (1 - b2) * gr * gr
                em, ev = 7 * U * (b1 * m0.abs() + (1 - b1) * gr.abs()), 12 * U * v
                den = v.sqrt() / math.sqrt(1 - b2 ** t) + hp["eps"]
                size = hp["lr"] / (1 - b1 ** t)
                step = size * m / den
                th0 = before["params"][i].double()
                th = th0 * (1 - hp["lr"] * hp["weight_decay"]) - step
                tol = size * em / den + 17 * U * step.abs() + 3 * U * (th0.abs() + step.abs()) + (2.0 ** -8 * th.abs() if p == BF16 else 0.0)
                assert ((a["params"][i].double() - th).abs() <= tol).all(), (numel, turn)
                pad = -numel % block
                top = torch.nn.functional.pad(v, (0, pad)).view(-1, block).amax(1)
                assert ((a["amax_v"][i].double() - top).abs() <= 12 * U * top).all()
                at = spread(top, block, numel)
                ideal = torch.where(at > 0, (v / at).sqrt() * 255, 0.0)
                code = a["v"][i].double()
                near = ((code - ideal).abs() <= 0.5 + (12 + 12 + 4) * U * 255) | ((code == 1) & (ideal < 1) & (v > 0))
                assert near.all() and (code[v > 0] > 0).all(), (numel, turn)
        assert store.intact()
        total = sum(SIZES)
        out = torch.zeros(total, device="cuda")
        h.moments(None, out, F32)
        at = 0
        for i, n in enumerate(SIZES):
            x = (a["v"][i].double() / 255).float()
            assert torch.equal(out[at:at + n], (x * x) * a["amax_v"][i].repeat_interleave(block)[:n]), n
            at += n
        h.free()


def test_root_codes_hold_what_linear_ones_lose():
    """Elements whose gradients pause after a hundredth of the block's largest:
    their v survives, so their steps stay near lr; kept states change nothing
    where no gradient comes."""
    log("adamw root codes, rare rows")
    n, block = 4096, 256
    g = torch.full((n,), 1.0, device="cuda")
    g[::2] = 1e-2
    arrays = dict(params=[torch.zeros(n, device="cuda")], grads=[g], m=[torch.zeros(n, dtype=torch.int8, device="cuda")],
                  v=[torch.zeros(n, dtype=torch.uint8, device="cuda")], amax_m=[torch.zeros(n // block, device="cuda")],
                  amax_v=[torch.zeros(n // block, device="cuda")], bf16_out=[None])
    h = rs.AdamW([(n, F32, F32, ROOT, block, 0)]).upload().bind(**arrays)
    hp = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0)
    h.step([{**hp, "step": 1}])
    assert (arrays["v"][0][::2] == 3).all()  # 255 / 100, to the nearest
    arrays["grads"][0].zero_()
    before = arrays["params"][0].clone()
    h.step([{**hp, "step": 2}])
    move = (arrays["params"][0] - before).abs()
    # m / sqrt(v) is within (1 / 127 / 0.01 / 2 and 3 / 2.55 - 1, together a factor 2) of 1
    assert (move < 2e-3).all() and (move[::2] > 2e-4).all()
    codes = arrays["v"][0].clone()
    for t in range(3, 40):  # v shrinks everywhere alike: its codes stay
        h.step([{**hp, "step": t}])
    assert torch.equal(arrays["v"][0], codes)
    h.free()


def test_no_elements_at_all():
    log("adamw without elements")
    h = rs.AdamW([(0, F32, F32, rs.RS_STATE_F32, 0, 0), (0, BF16, F32, ROOT, 64, 0)]).upload()
    none = [None, None]
    h.bind(none, none, none, none, none, none, [None, torch.zeros(4, dtype=torch.bfloat16, device="cuda").data_ptr()])
    sumsq, scale = torch.ones(1, dtype=torch.float64, device="cuda"), torch.zeros(1, device="cuda")
    h.l2norm_clip(1.0, sumsq, scale)
    assert sumsq.item() == 0.0 and scale.item() == 1.0
    h.step([HP])
    out = torch.ones(3, device="cuda")
    h.moments(out, None)
    assert (out == 1).all()
    h.free()


def test_two_plans_on_two_streams():
    """Each with its own workspace: what they give does not depend on the other."""
    log("adamw two plans at once")
    tensors = [(300_000, F32, BF16, rs.RS_STATE_F32, 0, 0), (5000, F32, BF16, rs.RS_STATE_INT8, 256, 0)]
    made = [make(tensors, 70, True, out=False) for _ in range(3)]
    results = [(torch.zeros(1, dtype=torch.float64, device="cuda"), torch.zeros(1, device="cuda")) for _ in made]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for turn in range(5):
        for (h, _, _), r, s in zip(made, results, [*streams, torch.cuda.current_stream()]):
            with torch.cuda.stream(s):
                h.l2norm_clip(1e-2, *r)
                h.step([HP], grad_scale=r[1])
    torch.cuda.synchronize()
    for k in ("params", "m", "v"):
        for x, y, z in zip(*(m[1][k] for m in made)):
            assert torch.equal(x, y) and torch.equal(x, z), k
    assert results[0][0].item() == results[1][0].item() == results[2][0].item()
    for h, _, _ in made:
        h.free()
