"""Token statistics and their gradient against binary64.

Tolerances, u = 2^-24, x_i = (z_i - m) / T <= 0: an exponent is a difference, a
rounded factor and a product, so e_i is off by e_i = (3 |x_i| + 15) u of itself
with the exponential's ulp and a chain of eight sums and two joins; the token,
outside the sums, by 3 |x_y| u (and the ulp where it is not the maximum).  With
E = sum p_i e_i over the others and the token:
  ln S is off by E, log p by E + 3 |x_y| u, and for a token that is the maximum
  by what the others are off, relative to their share;
  the entropy by sum p_i e_i (1 + |x_i| + mean |x|);
  a gradient by its factors: p_i (e_i + E + 8 u) of the bracket's absolute
  terms, and |b| times the error of mean |x|.
Results in binary32 add u of themselves, bf16 ones 2^-8 (2^-134 at least)."""
import math

import numpy as np
import pytest
import torch

import sharded_state_raggedshard_amd as rs
from gpu_harness import log

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPE = {rs.RS_F32: torch.float32, rs.RS_BF16: torch.bfloat16}
DTYPES = [rs.RS_F32, rs.RS_BF16]


def logits_of(rows, vocab, dtype, seed, gap=0, width=2.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    store = torch.full((rows, vocab + gap), 1e4, device="cuda", dtype=TYPE[dtype])
    z = store[:, :vocab]
    z.copy_(torch.randn(rows, vocab, device="cuda", generator=g) * width)
    target = torch.randint(0, vocab, (rows,), device="cuda", generator=g)
    return z, target, g


def run(z, dtype, target, top, temperature=1.0, want=("logp", "entropy", "saved")):
    rows, vocab = z.shape
    nb = rs.rs_token_stats_bytes(rows, vocab, top)
    work = torch.full((nb + 64,), 0xFF, dtype=torch.uint8, device="cuda")
    out = dict(logp=torch.full((rows + 1,), 5.0, device="cuda"), entropy=torch.full((rows + 1,), 5.0, device="cuda"),
               saved=torch.full((rows + 1, 4), 5.0, device="cuda"), top_id=torch.full((rows * top + 1,), 5, dtype=torch.int64, device="cuda"),
               top_logp=torch.full((rows * top + 1,), 5.0, device="cuda"))
    give = {k: out[k] if k in want else None for k in ("logp", "entropy", "saved")}
    if target is None:
        give["logp"] = None
    rs.rs_token_stats(z, dtype, rows, vocab, z.stride(0) if rows > 1 else vocab, target, give["logp"], give["entropy"], top,
                      out["top_id"] if top else None, out["top_logp"] if top else None, give["saved"], work, nb, temperature=temperature)
    assert (work[nb:] == 0xFF).all()
    for k, n in (("logp", rows), ("entropy", rows), ("top_id", rows * top), ("top_logp", rows * top)):
        assert (out[k][n:] == 5).all(), k
    assert (out["saved"][rows:] == 5).all()
    return dict(logp=out["logp"][:rows], entropy=out["entropy"][:rows], saved=out["saved"][:rows].contiguous(),
                top_id=out["top_id"][:rows * top].view(rows, top), top_logp=out["top_logp"][:rows * top].view(rows, top))


class Exact:
    """Everything in binary64, for rows that take part and hold no NaN or +inf."""

    def __init__(self, z, target, temperature):
        z = z.double()
        self.m = z.amax(-1, keepdim=True)
        self.x = ((z - torch.where(torch.isinf(self.m), 0.0, self.m)) / temperature)
        e = torch.exp(self.x)
        self.S = e.sum(-1, keepdim=True)
        self.p = e / self.S
        finite = self.x.clamp(min=-1e6)
        self.ax = torch.where(self.p > 0, finite.abs(), 0.0)
        # ln S from the others than the largest: 1 + rest would round the rest away
        rest = e.scatter(1, self.x.argmax(1, keepdim=True), 0.0).sum(-1, keepdim=True)
        ln_s = torch.log1p(rest)
        self.logp_all = self.x - ln_s
        self.down = (self.p * self.ax).sum(-1, keepdim=True)  # mean |x|
        self.entropy = ln_s[:, 0] + self.down[:, 0]
        err = (3 * self.ax + 15) * U
        if target is not None:
            t = target.clamp(min=0)[:, None]
            self.xy = self.ax.gather(1, t)
            err.scatter_(1, t, torch.where(self.xy > 0, (3 * self.xy + 2) * U, 0.0))
            self.logp = self.logp_all.gather(1, t)[:, 0]
        self.err = err
        self.E = (self.p * err).sum(-1, keepdim=True)
        self.derr = (self.p * (err + self.E) * (self.ax + self.down)).sum(-1, keepdim=True)
        self.herr = (self.p * err * (1 + self.ax + self.down)).sum(-1) + 2 * U * self.entropy


def check(z, dtype, target, got, temperature, top):
    rows, vocab = z.shape
    some = max(1, (1 << 25) // vocab)
    for a in range(0, rows, some):
        here = slice(a, min(rows, a + some))
        t = None if target is None else target[here]
        live = torch.ones(here.stop - a, dtype=torch.bool, device="cuda") if t is None else (t >= 0) & (t < vocab)
        x = Exact(z[here], None if t is None else torch.where(live, t, 0), temperature)
        live &= ~torch.isinf(x.m[:, 0])
        zero = torch.zeros_like(x.entropy)
        if t is not None:
            tol = x.E[:, 0] + 3 * U * x.xy[:, 0] + 2 * U * x.logp.abs()
            gone = torch.isinf(x.logp)
            off = torch.where(live & ~gone, got["logp"][here].double() - x.logp, zero)
            assert (off.abs() <= tol.nan_to_num(0.0, 0.0, 0.0)).all()
            assert (got["logp"][here][live & gone] == -math.inf).all() and not got["logp"][here][~live].any()
        off = torch.where(live, got["entropy"][here].double() - x.entropy, zero)
        assert (off.abs() <= torch.where(live, x.herr, zero)).all()
        assert not got["entropy"][here][~live].any()
        if not top:
            continue
        values = z[here].float().cpu().numpy()
        n = min(top, vocab)
        for r in range(values.shape[0]):
            v = values[r]
            if live[r]:
                if vocab > 4 * n:
                    edge = np.partition(v, vocab - n)[vocab - n]
                    cand = np.flatnonzero(v >= edge)
                else:
                    cand = np.arange(vocab)
                order = cand[np.lexsort((cand, -v[cand].astype(np.float64)))][:n]
                order = order[v[order] > -np.inf]
            else:
                order = np.zeros(0, dtype=np.int64)
            ids = np.full(top, -1, dtype=np.int64)
            ids[:len(order)] = order
            assert np.array_equal(got["top_id"][a + r].cpu().numpy(), ids), (a + r, top)
            lp = got["top_logp"][a + r]
            assert (lp[len(order):] == -math.inf).all()
            if len(order):
                o = torch.from_numpy(order).cuda()
                want = x.logp_all[r][o]
                assert ((lp[:len(order)].double() - want).abs() <= x.E[r] + 3 * U * x.ax[r][o] + 2 * U * want.abs()).all()


SHAPES = [(1, 1), (3, 2), (5, 7), (2, 8), (4, 31), (40, 33), (7, 1000), (600, 513), (9, 4099), (5, 8192), (6, 8193), (520, 8200), (3, 32003),
          (700, 32003), (61, 50000), (1, 128256), (16, 128256), (2, 201088)]


@pytest.mark.parametrize("rows,vocab", SHAPES)
@pytest.mark.parametrize("dtype", DTYPES)
def test_against_binary64(rows, vocab, dtype):
    log(f"token stats {rows} x {vocab} {dtype}")
    for top, gap, temperature in ((0, 0, 1.0), (5, 3, 0.7), (32, 0, 1.0), (1, 1, 3.0)):
        z, target, g = logits_of(rows, vocab, dtype, 10 + top, gap)
        z.scatter_(1, target[:, None], torch.where(torch.rand(rows, 1, device="cuda", generator=g) < 0.5, 25.0, 3.0).to(z.dtype))
        target[::4] = -1
        target[1::7] = vocab
        check(z, dtype, target, run(z, dtype, target, top, temperature), temperature, top)


@pytest.mark.parametrize("dtype", DTYPES)
def test_without_tokens(dtype):
    log(f"token stats without tokens {dtype}")
    for rows, vocab in ((5, 33), (600, 4000), (4, 128256)):
        z, _, _ = logits_of(rows, vocab, dtype, 3)
        check(z, dtype, None, run(z, dtype, None, 8), 1.0, 8)


@pytest.mark.parametrize("rows,vocab", [(700, 1031), (3, 1031), (520, 40000), (8, 128256), (600, 128256)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_ties_masks_and_crowds(rows, vocab, dtype):
    """Ties beyond what is gathered, few values above -inf, masks of the type's
    lowest value, the best values in few threads' shares."""
    log(f"token stats ties {rows} x {vocab} {dtype}")
    z, target, g = logits_of(rows, vocab, dtype, 5)
    low = torch.finfo(TYPE[dtype]).min
    rand = lambda n: torch.rand(n, device="cuda", generator=g)  # noqa: E731
    kinds = 8
    for r in range(rows):
        kind = r % kinds
        row = z[r]
        if kind == 0:
            row.zero_()
        elif kind == 1:
            row.fill_(-math.inf)
            row[(rand(4) * vocab).long()] = 1.0
        elif kind == 2:
            row.copy_(torch.where(rand(vocab) < 0.9, low, row.float()).to(row.dtype))
        elif kind == 3:
            row.copy_(torch.round(row.float()).to(row.dtype))  # many equal values
            row[::3] = -0.0
        elif kind == 4:
            row.fill_(low)
        elif kind == 5:
            row[:7 % vocab] = 30.0
            row[-5:] = 30.0
        elif kind == 6 and vocab > 4096:
            at = torch.arange(0, vocab, 512, device="cuda")
            row[at] = (20 + rand(len(at))).to(row.dtype)
            at = (torch.arange(0, vocab // 2048, device="cuda")[:, None] * 2048 + torch.arange(16, device="cuda")).view(-1)
            row[at] = (25 + rand(len(at))).to(row.dtype)
        else:
            row[vocab // 2:] = 40.0
    for top in (1, 20, 32):
        check(z, dtype, target, run(z, dtype, target, top), 1.0, top)


@pytest.mark.parametrize("rows,vocab", [(4, 77), (4, 100_000), (600, 9000)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_rows_that_are_not_numbers(rows, vocab, dtype):
    log(f"token stats NaN {rows} x {vocab} {dtype}")
    z, target, g = logits_of(rows, vocab, dtype, 6)
    z[0, vocab // 3] = float("nan")
    z[1, vocab // 5] = float("inf")
    z[2] = -math.inf
    z[2, 5] = float("nan")
    target[2] = 5
    z[3] = -math.inf
    got = run(z, dtype, target, 8)
    assert torch.isnan(got["logp"][:3]).all() and torch.isnan(got["entropy"][:3]).all()
    assert torch.isnan(got["top_logp"][:3]).all() and (got["top_id"][:4] == -1).all()
    assert got["logp"][3] == 0 and got["entropy"][3] == 0 and (got["top_logp"][3] == -math.inf).all()
    if rows > 4:
        check(z[4:], dtype, target[4:], {k: v[4:] for k, v in got.items()}, 1.0, 8)
    # a row without a token hides what it holds
    target[:4] = -1
    got = run(z, dtype, target, 8)
    assert not got["logp"][:4].any() and not got["entropy"][:4].any() and not got["saved"][:4].any()
    assert (got["top_id"][:4] == -1).all() and (got["top_logp"][:4] == -math.inf).all()


def test_nearly_certain_tokens_keep_their_digits():
    """1 - p, log p and the entropy of a token 10 to 60 above the rest."""
    log("token stats nearly certain")
    for vocab in (50, 5000, 130_000):
        z, target, _ = logits_of(50, vocab, rs.RS_F32, 8, width=1.0)
        z.scatter_(1, target[:, None], torch.arange(10.0, 60.0, device="cuda")[:, None])
        z[:, 0] = torch.where(target == 0, z[:, 0], 5.0)
        got = run(z, rs.RS_F32, target, 2)
        x = Exact(z, target, 1.0)
        # what the others weigh is known to (3 |x| + 15) u of itself
        rest = -torch.expm1(torch.log_softmax(z.double(), -1).gather(1, target[:, None])[:, 0])
        others = torch.where(torch.arange(vocab, device="cuda") == target[:, None], 0.0, torch.exp(x.x))
        rest = others.sum(1) / (1 + others.sum(1))
        rel = (3 * 70 + 20) * U
        assert ((got["saved"][:, 3].double() - rest).abs() <= rel * rest + 2.0 ** -126).all()
        assert ((got["logp"].double() + torch.log1p(others.sum(1))).abs() <= rel * rest + 2.0 ** -126).all()
        h = torch.log1p(others.sum(1)) - (others * x.x).sum(1) / (1 + others.sum(1))
        assert ((got["entropy"].double() - h).abs() <= 2 * rel * h + 2.0 ** -126).all()


@pytest.mark.parametrize("shift", [0.0, -90.0, 600.0, -1500.0, 2.0 ** 40])
@pytest.mark.parametrize("rows,vocab,top", [(50, 40_000, 0), (530, 40_000, 0), (530, 40_000, 3), (3, 5000, 3)])
def test_bf16_rows_far_from_zero(rows, vocab, top, shift):
    """Rows around any value, the token a lot above the rest or not at all: as the others, and 1 - p keeps its digits."""
    log(f"token stats {rows} x {vocab} bf16 around {shift}")
    z, target, g = logits_of(rows, vocab, rs.RS_BF16, 21, width=1.0)
    z.copy_(z.float() + shift)
    lift = torch.arange(rows, device="cuda")[:, None] % 60 + 1.0
    z.scatter_(1, target[:, None], (lift + shift).to(z.dtype))
    got = run(z, rs.RS_BF16, target, top)
    check(z, rs.RS_BF16, target, got, 1.0, top)
    x = Exact(z, target, 1.0)
    others = torch.where(torch.arange(vocab, device="cuda") == target[:, None], 0.0, torch.exp(x.x)).sum(1)
    sure = (x.xy[:, 0] == 0) & (others < 1e-3)
    # three rows are lifted by 3 at most: 5000 e^0.5 / e^3 = 400 of the others' weight
    assert sure.any() or rows == 3 or abs(shift) > 1e9
    rel = (3 * x.ax.amax(1) + 20) * U
    rest = others / (1 + others)
    assert ((got["saved"][:, 3].double() - rest).abs() <= rel * rest + 2.0 ** -126)[sure].all()
    assert ((got["logp"].double() + torch.log1p(others)).abs() <= rel * rest + 2.0 ** -126)[sure].all()


def test_large_bf16_values():
    """The ends of the type in rows that are taken in many pieces, ruled out values between them."""
    log("token stats large bf16 values")
    for rows, vocab, top in ((6, 40_000, 0), (530, 40_000, 2)):
        z = torch.zeros(rows, vocab, device="cuda", dtype=torch.bfloat16)
        z[0], z[1] = 3e38, -3e38
        z[2, ::2] = -3e38
        z[2, 1::2] = 3e38
        z[3, ::2] = -math.inf
        z[4] = -math.inf
        z[5, 20_000] = math.inf
        target = torch.full((rows,), 7, device="cuda")
        got = run(z, rs.RS_BF16, target, top)
        want = torch.tensor([math.log(vocab), math.log(vocab), math.log(vocab / 2), math.log(vocab / 2), 0.0], dtype=torch.float64, device="cuda")
        assert ((got["entropy"][:5].double() - want).abs() <= 20 * U * (1 + want)).all()
        assert ((got["logp"][:5].double() + want).abs() <= 20 * U * (1 + want)).all()
        assert torch.isnan(got["entropy"][5]) and torch.isnan(got["logp"][5])
        if top:
            assert got["top_id"][:6].tolist() == [[0, 1], [0, 1], [1, 3], [1, 3], [-1, -1], [-1, -1]]


def expected_gradient(x, t, live, c, b, temperature):
    """(gradient, tolerance without the output's rounding) in binary64."""
    c, b = c.double()[:, None], b.double()[:, None]
    bracket = c + b * torch.where(x.p > 0, x.x.clamp(min=-1e6) + x.down, 0.0)
    g = -x.p * bracket
    size = c.abs() + b.abs() * (x.down + x.ax)
    tol = x.p * ((x.err + x.E + 8 * U) * size + b.abs() * x.derr)
    if t is not None:
        py, xy = x.p.gather(1, t[:, None]), x.xy
        others = (1 - torch.zeros_like(py)) * (x.p.sum(1, keepdim=True) - py)
        others = torch.where(torch.arange(x.p.shape[1], device="cuda") == t[:, None], 0.0, x.p).sum(1, keepdim=True)
        own = c * others - b * py * torch.where(py > 0, x.down - xy, 0.0)
        oerr = torch.where(torch.arange(x.p.shape[1], device="cuda") == t[:, None], 0.0, x.p * (x.err + x.E + 8 * U)).sum(1, keepdim=True)
        otol = c.abs() * oerr + b.abs() * py * (((3 * xy + 2) * U + x.E + 8 * U) * (x.down + xy) + x.derr)
        g.scatter_(1, t[:, None], own)
        tol.scatter_(1, t[:, None], otol)
    dead = ~live[:, None]
    return torch.where(dead, 0.0, g) / temperature, torch.where(dead, 0.0, tol) / temperature


@pytest.mark.parametrize("rows,vocab", SHAPES)
@pytest.mark.parametrize("dtype", DTYPES)
def test_gradient_against_binary64(rows, vocab, dtype):
    log(f"token stats gradient {rows} x {vocab} {dtype}")
    for gap, temperature, parts in ((0, 1.0, "both"), (3, 0.7, "both"), (0, 2.0, "logp"), (5, 1.0, "entropy"), (0, 1.0, "no token")):
        z, target, g = logits_of(rows, vocab, dtype, 20, gap)
        z.scatter_(1, target[:, None], torch.where(torch.rand(rows, 1, device="cuda", generator=g) < 0.5, 25.0, 3.0).to(z.dtype))
        z[:, 1::5] = torch.where(target[:, None] % 2 == 0, -math.inf, z[:, 1::5].float()).to(z.dtype)
        z.scatter_(1, target[:, None], 4.0)
        c, b = torch.randn(rows, device="cuda", generator=g), torch.randn(rows, device="cuda", generator=g)
        if parts == "no token":
            target = None
        else:
            target[::4] = -1
            c[3::9] = 0.0
            b[3::18] = 0.0
        saved = run(z, dtype, target, 0, temperature, want=("saved",))["saved"]
        live = torch.ones(rows, dtype=torch.bool, device="cuda") if target is None else (target >= 0)
        gc = c if parts in ("both", "logp") else None
        gb = b if parts in ("both", "entropy", "no token") else None
        store = torch.full((rows, vocab + gap + 2), 9.0, device="cuda", dtype=z.dtype)
        d = store[:, :vocab]
        before = z.clone()
        rs.rs_token_stats_grad(z, dtype, rows, vocab, vocab + gap, target, saved, gc, gb, d, vocab + gap + 2, temperature=temperature)
        assert (store[:, vocab:] == 9).all() and torch.equal(before, z)
        zero = torch.zeros(rows, device="cuda")
        some = max(1, (1 << 24) // vocab)
        for a in range(0, rows, some):
            here = slice(a, a + some)
            t = None if target is None else torch.where(live[here], target[here], 0)
            x = Exact(z[here], t, temperature)
            want, tol = expected_gradient(x, t, live[here], zero[here] if gc is None else c[here], zero[here] if gb is None else b[here], temperature)
            # products below 2^-126 count as 0
            out = U * want.abs() if dtype == rs.RS_F32 else (2.0 ** -8 * want.abs()).clamp(min=2.0 ** -134)
            assert ((d[here].double() - want).abs() <= tol + out + 2.0 ** -126).all(), (parts, a)
        if parts == "both":  # in place
            rs.rs_token_stats_grad(z, dtype, rows, vocab, vocab + gap, target, saved, gc, gb, z, vocab + gap, temperature=temperature)
            assert torch.equal(z, d)


def test_gradient_against_differences():
    log("token stats gradient against differences")
    rows, vocab, T = 4, 9, 0.8
    z, target, g = logits_of(rows, vocab, rs.RS_F32, 30, width=1.0)
    c, b = torch.randn(rows, device="cuda", generator=g), torch.randn(rows, device="cuda", generator=g)

    def loss(z):
        ls = torch.log_softmax(z / T, -1)
        return (c.double() * ls.gather(1, target[:, None])[:, 0] - b.double() * (ls.exp() * ls).sum(-1)).sum().item()
    saved = run(z, rs.RS_F32, target, 0, T)["saved"]
    d = torch.zeros_like(z)
    rs.rs_token_stats_grad(z, rs.RS_F32, rows, vocab, vocab, target, saved, c, b, d, vocab, temperature=T)
    h = 1e-5  # h^2 times a third derivative below 100; 16 digits of values below 10 over h: 1e-10
    for i in range(rows):
        for j in range(vocab):
            up, down = z.double().clone(), z.double().clone()
            up[i, j] += h
            down[i, j] -= h
            assert abs((loss(up) - loss(down)) / (2 * h) - d[i, j].item()) <= 2e-8 + 200 * U


def test_zero_gradients_and_bad_rows_stay_apart():
    log("token stats gradient of bad rows")
    for rows, vocab in ((4, 300), (600, 9000)):
        z, target, g = logits_of(rows, vocab, rs.RS_F32, 31)
        z[0, 1] = float("nan")
        z[1, 1] = float("nan")
        z[2] = -math.inf
        c = torch.ones(rows, device="cuda")
        c[1] = 0.0
        saved = run(z, rs.RS_F32, target, 0)["saved"]
        d = torch.full_like(z, 3.0)
        rs.rs_token_stats_grad(z, rs.RS_F32, rows, vocab, vocab, target, saved, c, None, d, vocab)
        assert torch.isnan(d[0]).all() and not d[1].any() and not d[2].any()
        assert torch.isfinite(d[3:]).all() and d[3:].any()


def test_large_values():
    """Logits at the ends of binary32: differences overflow to -inf, no further."""
    log("token stats large values")
    vocab = 1000
    z = torch.zeros(5, vocab, device="cuda")
    z[0], z[1] = 3e38, -3e38
    z[2, ::2] = -3e38
    z[2, 1::2] = 3e38
    z[3] = torch.linspace(-3e38, 3e38, vocab, device="cuda")  # its step overflows: infinities and NaN
    z[4] = torch.linspace(-3e38, 3e38, vocab, device="cuda", dtype=torch.float64)
    assert torch.isnan(z[3]).any() or torch.isinf(z[3]).any()
    target = torch.tensor([5, 6, 7, vocab - 1, vocab - 1], device="cuda")
    got = run(z, rs.RS_F32, target, 3)
    fine = [0, 1, 2, 4]
    want = torch.tensor([math.log(vocab), math.log(vocab), math.log(vocab / 2), 0.0], dtype=torch.float64, device="cuda")
    assert ((got["entropy"][fine].double() - want).abs() <= 20 * U * (1 + want)).all()
    assert ((got["logp"][fine].double() + want).abs() <= 20 * U * (1 + want)).all()
    assert got["top_id"][fine].tolist() == [[0, 1, 2], [0, 1, 2], [1, 3, 5], [vocab - 1, vocab - 2, vocab - 3]]
    assert torch.isnan(got["entropy"][3]) and torch.isnan(got["logp"][3]) and got["top_id"][3].tolist() == [-1] * 3


def test_equal_calls_and_captured_calls_give_equal_bits():
    log("token stats graph")
    for rows, vocab, top in ((16, 60_000, 20), (700, 20_001, 8)):
        z, target, g = logits_of(rows, vocab, rs.RS_BF16, 40)
        c, b = torch.randn(rows, device="cuda", generator=g), torch.randn(rows, device="cuda", generator=g)
        nb = rs.rs_token_stats_bytes(rows, vocab, top)

        def buffers():
            return dict(work=torch.zeros(nb, dtype=torch.uint8, device="cuda"), logp=torch.zeros(rows, device="cuda"),
                        entropy=torch.zeros(rows, device="cuda"), top_id=torch.zeros(rows, top, dtype=torch.int64, device="cuda"),
                        top_logp=torch.zeros(rows, top, device="cuda"), saved=torch.zeros(rows, 4, device="cuda"), d=torch.zeros_like(z))

        def call(o):
            rs.rs_token_stats(z, rs.RS_BF16, rows, vocab, vocab, target, o["logp"], o["entropy"], top, o["top_id"], o["top_logp"], o["saved"],
                              o["work"], nb)
            rs.rs_token_stats_grad(z, rs.RS_BF16, rows, vocab, vocab, target, o["saved"], c, b, o["d"], vocab)
        a, e = buffers(), buffers()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
            call(a)
        for turn in range(3):
            z.copy_(torch.randn(rows, vocab, device="cuda", generator=g) * 3)
            graph.replay()
            call(e)
            torch.cuda.synchronize()
            for name in ("logp", "entropy", "top_id", "top_logp", "saved", "d"):
                assert torch.equal(a[name], e[name]), (turn, name)


def test_logits_beyond_32_bit_offsets():
    log("token stats far rows")
    rows, vocab = 17_000, 128_256
    assert rows * vocab > 1 << 31
    g = torch.Generator(device="cuda").manual_seed(50)
    z = torch.randn(rows, vocab, device="cuda", dtype=torch.bfloat16, generator=g).mul_(3)
    target = torch.randint(0, vocab, (rows,), device="cuda", generator=g)
    c, b = torch.randn(rows, device="cuda", generator=g), torch.randn(rows, device="cuda", generator=g)
    got = run(z, rs.RS_BF16, target, 4)
    d = torch.zeros_like(z)
    rs.rs_token_stats_grad(z, rs.RS_BF16, rows, vocab, vocab, target, got["saved"], c, b, d, vocab)
    n = 1030  # as many rows as are not split
    tail = slice(rows - n, rows)
    part = run(z[tail], rs.RS_BF16, target[tail], 4)
    for k in got:
        assert torch.equal(got[k][tail], part[k]), k
    e = torch.zeros(n, vocab, device="cuda", dtype=torch.bfloat16)
    rs.rs_token_stats_grad(z[tail], rs.RS_BF16, n, vocab, vocab, target[tail], part["saved"], c[tail], b[tail], e, vocab)
    assert torch.equal(d[tail], e)
    check(z[-20:], rs.RS_BF16, target[-20:], {k: v[-20:] for k, v in got.items()}, 1.0, 4)


def test_more_rows_than_a_grid():
    log("token stats many rows")
    rows, vocab = (1 << 22) + 77, 3
    z, target, g = logits_of(rows, vocab, rs.RS_F32, 60)
    target[::5] = -1
    got = run(z, rs.RS_F32, target, 2)
    live = target >= 0
    x = Exact(z, target.clamp(min=0), 1.0)
    assert (torch.where(live, got["entropy"].double() - x.entropy, 0.0).abs() <= x.herr).all() and not got["entropy"][~live].any()
    ids = torch.where(live[:, None], torch.sort(z, dim=-1, descending=True, stable=True).indices[:, :2], -1)
    assert torch.equal(got["top_id"], ids)
    c = torch.ones(rows, device="cuda")
    d = torch.zeros_like(z)
    rs.rs_token_stats_grad(z, rs.RS_F32, rows, vocab, vocab, target, got["saved"], c, None, d, vocab)
    want, tol = expected_gradient(x, target.clamp(min=0), live, c, torch.zeros_like(c), 1.0)
    assert ((d.double() - want).abs() <= tol + U * want.abs()).all()
