"""GPU parity of the training objectives with the binary64 oracle
(oracle/objectives.py): token log-probability, clipped policy loss,
preference loss.

Tolerances, from the arithmetic of the kernels (u = 2^-24, half a step of
binary32; R = max |z - max z| / T of the row):
  an exponential: exponent scale, difference and product each rounded once
      on values of size R, and one ulp of exp2: (3 R + 3) u of its value;
  the row sum: that, four binary32 additions in a chain and binary64 ones,
      up to 8 rescalings by an exponential that are not by 1:
      d_s = (3 R + 3 + 4 + 8 (3 R + 3)) u;
  logp: d_l = d_s, and u |logp| for the output;
  dloss/dlogp: |c'(l)| d_l with c' bounded from its formula, and u |c|;
  a gradient value: c p off by (d_s + (3 R + 3) u + 4 u) |c| p + dc p, the
      token's own also by 2 u |c| (c - c p), then half a step of the type.
"""
import math

import numpy as np
import pytest
import torch

import sharded_state_raggedshard_amd as rs
from gpu_harness import log
from oracle import objectives as ob

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {rs.RS_F32: 2.0 ** -24, rs.RS_BF16: 2.0 ** -8}
TORCH = {rs.RS_F32: torch.float32, rs.RS_BF16: torch.bfloat16}
SENT = 7.25  # exact in both types


def make_logits(rows, vocab, ld, dtype, seed, shift=0, sigma=2.5):
    """(view [rows, vocab] of stride ld, `shift` elements into its storage)."""
    g = torch.Generator().manual_seed(seed)
    store = torch.full((shift + rows * ld + 8,), SENT, dtype=TORCH[dtype])
    v = store[shift:shift + rows * ld].view(rows, ld)[:, :vocab]
    v.copy_((torch.randn(rows, vocab, generator=g) * sigma).to(TORCH[dtype]))
    dev = store.cuda()
    return dev, dev[shift:shift + rows * ld].view(rows, ld)[:, :vocab]


def np64(t):
    return t.detach().cpu().double().numpy()


def row_bounds(z, temperature):
    """(R, d_s) per row."""
    with np.errstate(all="ignore"):
        top = np.max(np.where(np.isfinite(z), z, -1e300), axis=1)
        # values far below the top count as 0 on either side
        fall = np.where(np.isfinite(z), top[:, None] - z, 0.0) / temperature
        R = np.minimum(fall.max(axis=1), 90.0)
    return R, (9 * (3 * R + 3) + 4) * U


def check_gradient(got, exp, z, target, temperature, dcoef, dtype, what):
    R, ds = row_bounds(z, temperature)
    for t in range(z.shape[0]):
        if not exp["live"][t]:
            assert not got[t].any(), f"{what}: row {t} is not zero"
            continue
        c, p = abs(exp["coef"][t]) / temperature, exp["p"][t]
        rel = ds[t] + (3 * R[t] + 7) * U
        tol = c * p * rel + dcoef[t] / temperature * p
        y = int(target[t])
        tol[y] = c * (p[y] * rel + 2 * U) + dcoef[t] / temperature * (1 - p[y])
        tol = tol * 1.01 + HALF[dtype] * np.abs(exp["dlogits"][t]) + 1e-37
        bad = ~(np.abs(got[t] - exp["dlogits"][t]) <= tol)
        assert not bad.any(), (f"{what}: row {t} columns {np.nonzero(bad)[0][:5]} got "
                               f"{got[t][bad][:5]} expected {exp['dlogits'][t][bad][:5]}")


def work_for(rows, vocab, n_seq=0):
    n = rs.rs_objective_bytes(rows, vocab, n_seq)
    return torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda"), n  # NaN-filled: nothing may be taken from it


def close(got, exp, tol, what):
    got, exp = np.asarray(got, dtype=np.float64), np.asarray(exp, dtype=np.float64)
    same = (got == exp) | (np.isnan(got) & np.isnan(exp))
    with np.errstate(invalid="ignore"):
        bad = ~(same | (np.abs(got - exp) <= tol))
    at = np.nonzero(bad)[0][:4]
    assert not bad.any(), f"{what}[{at}]: got {got[at]} expected {exp[at]} within {np.broadcast_to(tol, exp.shape)[at]}"


# (rows, vocab, ld - vocab, start shift, dtype, temperature)
SHAPES = [
    (1, 1, 0, 0, rs.RS_F32, 1.0), (3, 2, 1, 1, rs.RS_BF16, 1.0), (5, 3, 0, 3, rs.RS_F32, 0.5),
    (4, 7, 2, 1, rs.RS_BF16, 1.0), (4, 8, 0, 0, rs.RS_BF16, 2.0), (6, 9, 0, 0, rs.RS_BF16, 1.0),
    (33, 63, 0, 0, rs.RS_F32, 1.0), (9, 64, 3, 0, rs.RS_BF16, 1.0), (2, 511, 0, 5, rs.RS_BF16, 1.0),
    (17, 1000, 24, 0, rs.RS_F32, 0.7), (5, 2047, 0, 0, rs.RS_BF16, 1.0), (5, 2048, 0, 0, rs.RS_F32, 1.0),
    (5, 2049, 0, 1, rs.RS_F32, 1.0), (130, 4099, 0, 0, rs.RS_BF16, 1.0),
    (3, 8192, 0, 0, rs.RS_BF16, 1.0), (2, 16391, 0, 1, rs.RS_BF16, 1.3), (3, 32003, 5, 0, rs.RS_F32, 1.0),
    (1, 50001, 0, 0, rs.RS_BF16, 1.0), (2, 131071, 0, 0, rs.RS_BF16, 1.0), (1, 201088, 0, 0, rs.RS_F32, 1.0),
    (3, 262149, 3, 1, rs.RS_BF16, 1.0),
]
IDS = [f"{r}x{v}+{p}@{s}-{'f32' if d == rs.RS_F32 else 'bf16'}-T{t}" for r, v, p, s, d, t in SHAPES]


# more rows than are split over workgroups: every workgroup size, with all of a
# row in registers and with a rest
ROW_SHAPES = [
    (65, 2047, 0, 1, rs.RS_F32, 1.0), (66, 40001, 0, 0, rs.RS_BF16, 1.0), (65, 70001, 3, 0, rs.RS_BF16, 1.0),
    (65, 110003, 0, 1, rs.RS_BF16, 1.0), (67, 60001, 0, 0, rs.RS_F32, 0.8), (65, 70016, 0, 0, rs.RS_F32, 1.0),
    (300, 40003, 0, 0, rs.RS_BF16, 1.0), (300, 60007, 1, 3, rs.RS_BF16, 1.0), (300, 3001, 0, 0, rs.RS_F32, 1.0),
    (520, 9001, 0, 0, rs.RS_BF16, 1.3), (520, 30011, 0, 0, rs.RS_BF16, 1.0), (2100, 5003, 0, 0, rs.RS_BF16, 1.0),
    (2100, 8111, 2, 1, rs.RS_BF16, 1.0), (2100, 7, 0, 0, rs.RS_F32, 1.0), (2050, 4095, 0, 0, rs.RS_F32, 1.0),
]
ROW_IDS = [f"{r}x{v}+{p}@{s}-{'f32' if d == rs.RS_F32 else 'bf16'}-T{t}" for r, v, p, s, d, t in ROW_SHAPES]


def targets_of(rows, vocab, seed):
    """A token for most rows; some at the ends of the row, some without."""
    y = np.random.default_rng(seed).integers(0, vocab, rows)
    y[0] = vocab - 1
    if rows > 2:
        y[1], y[2] = 0, -1
    if rows > 4:
        y[4] = vocab  # one past the row: no token
    return y


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_token_logp(shape):
    rows, vocab, pad, shift, dtype, temp = shape
    log(f"token_logp {shape}")
    store, z = make_logits(rows, vocab, vocab + pad, dtype, 3, shift)
    before = store.clone()
    y = targets_of(rows, vocab, 4)
    yt = torch.from_numpy(y).cuda()
    logp, lse = torch.full((rows + 1,), SENT, device="cuda"), torch.full((rows + 1,), SENT, device="cuda")
    work, n = work_for(rows, vocab)
    rs.rs_token_logp(z, dtype, rows, vocab, vocab + pad, yt, logp, work, n, lse=lse, temperature=temp)
    torch.cuda.synchronize()
    z64 = np64(z)
    el, ee, live, _ = ob.token_logp(z64, y, temp)
    R, ds = row_bounds(z64, temp)
    close(np64(logp)[:rows], el, ds + 1.01 * U * np.abs(el), "logp")
    close(np64(lse)[:rows], ee, ds + 1.01 * U * np.abs(ee), "lse")
    assert logp[rows] == SENT and lse[rows] == SENT and torch.equal(store, before)
    # without the optional output: the same bits
    again = torch.zeros(rows, device="cuda")
    rs.rs_token_logp(z, dtype, rows, vocab, vocab + pad, yt, again, work, n, temperature=temp)
    assert torch.equal(again, logp[:rows])


def policy_inputs(rows, z64, y, temp, seed):
    rng = np.random.default_rng(seed)
    l = ob.token_logp(z64, y, temp)[0]
    # ratios well inside, above and below the clipping range, both signs of A
    old = (l - rng.choice([0.0, 0.05, -0.1, 0.6, -0.5], rows)).astype(np.float32)
    ref = (l + rng.normal(0, 0.3, rows)).astype(np.float32)
    adv = rng.normal(0, 1, rows).astype(np.float32)
    w = rng.uniform(0.2, 1, rows).astype(np.float32) / rows
    if rows > 5:
        w[5] = 0
    return old, ref, adv, w


def policy_bounds(exp, z64, old, ref, adv, w, temp, kl):
    """(dcoef, dstats): errors of the coefficients and of the four sums."""
    _, ds = row_bounds(z64, temp)
    dl = ds * np.abs(exp["live"])
    r = np.exp(exp["logp"] - old.astype(np.float64))
    q = np.exp(ref.astype(np.float64) - exp["logp"])
    slope = np.abs(adv) * r * dl
    dcoef = np.abs(w) * (slope + kl * q * dl) * 1.01 + U * np.abs(exp["coef"])
    dkl = np.abs(w) * np.abs(1 - q) * dl + np.abs(w) * q * dl * dl
    pg = (np.abs(w) * slope)[exp["live"]].sum() * 1.01
    k = dkl[exp["live"]].sum() * 1.01
    return dcoef, np.array([pg + kl * k, pg, k, 0.0]) + 1.01 * U * np.abs(exp["stats"])


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
@pytest.mark.parametrize("kl", [0.0, 0.1])
def test_policy_loss(shape, kl):
    check_policy(shape, kl)


@pytest.mark.parametrize("shape", ROW_SHAPES, ids=ROW_IDS)
def test_policy_loss_a_workgroup_a_row(shape):
    check_policy(shape, 0.1)


def check_policy(shape, kl):
    rows, vocab, pad, shift, dtype, temp = shape
    log(f"policy_loss {shape} kl={kl}")
    _, z = make_logits(rows, vocab, vocab + pad, dtype, 5, shift)
    y = targets_of(rows, vocab, 6)
    z64 = np64(z)
    old, ref, adv, w = policy_inputs(rows, z64, y, temp, 7)
    dev = [torch.from_numpy(a).cuda() for a in (old, ref, adv, w)]
    yt = torch.from_numpy(y).cuda()
    ldd = vocab + (3 if pad else 0)  # its own stride
    dstore = torch.full((rows * ldd + 9,), SENT, dtype=TORCH[dtype], device="cuda")
    d = dstore[1:1 + rows * ldd].view(rows, ldd)
    logp = torch.zeros(rows, device="cuda")
    stats = torch.full((5,), SENT, device="cuda")
    work, n = work_for(rows, vocab)
    args = dict(temperature=temp, clip_low=0.2, clip_high=0.28, kl_coef=kl)
    rs.rs_policy_loss(z, dtype, rows, vocab, vocab + pad, yt, dev[0], dev[1] if kl else None, dev[2],
                      dev[3], d, ldd, logp, stats, work, n, **args)
    torch.cuda.synchronize()
    exp = ob.policy_loss(z64, y, old, ref if kl else None, adv, w, **args)
    dcoef, dstats = policy_bounds(exp, z64, old, ref, adv, w, temp, kl)
    _, ds = row_bounds(z64, temp)
    close(np64(logp), exp["logp"], ds + 1.01 * U * np.abs(exp["logp"]), "logp")
    close(np64(stats)[:4], exp["stats"], dstats, "stats")
    check_gradient(np64(d)[:, :vocab], exp, z64, y, temp, dcoef, dtype, "dlogits")
    assert (d[:, vocab:] == SENT).all() and dstore[0] == SENT and (dstore[1 + rows * ldd:] == SENT).all()
    assert stats[4] == SENT
    # loss alone, and in place: the same bits
    stats2, first = torch.zeros(4, device="cuda"), d[:, :vocab].clone()
    rs.rs_policy_loss(z, dtype, rows, vocab, vocab + pad, yt, dev[0], dev[1] if kl else None, dev[2],
                      dev[3], None, vocab, None, stats2, work, n, **args)
    close(np64(stats2), exp["stats"], dstats, "stats of the loss alone")
    rs.rs_policy_loss(z, dtype, rows, vocab, vocab + pad, yt, dev[0], dev[1] if kl else None, dev[2],
                      dev[3], z, vocab + pad, None, stats2, work, n, **args)
    assert torch.equal(stats2, stats[:4]) and torch.equal(z, first)


def test_policy_gradient_against_differences():
    """The gradient of the kernel's own loss, by central differences along
    random directions: a step of 2^-6 leaves the losses' own error (dstats)
    and that of the moved logits (below 8 u, as gradients add up to less
    than 2) over the step, and step^2 / 6 of a third derivative that is
    below 30 here (|A| r <= 4, kl below 1, directions of unit maximum)."""
    log("policy differences")
    rows, vocab = 6, 96
    rng = np.random.default_rng(1)
    z = torch.from_numpy(rng.normal(0, 1, (rows, vocab)).astype(np.float32)).cuda()
    y = targets_of(rows, vocab, 2)
    old, ref, adv, w = policy_inputs(rows, np64(z), y, 1.0, 3)
    dev = [torch.from_numpy(a).cuda() for a in (old, ref, adv, w)]
    yt = torch.from_numpy(y).cuda()
    work, n = work_for(rows, vocab)

    def call(x, d):
        s = torch.zeros(4, device="cuda")
        rs.rs_policy_loss(x, rs.RS_F32, rows, vocab, vocab, yt, *dev, d, vocab, None, s, work, n,
                          kl_coef=0.1)
        return s[0].item()

    d = torch.zeros(rows, vocab, device="cuda")
    call(z, d)
    step = 2.0 ** -6
    exp = ob.policy_loss(np64(z), y, old, ref, adv, w, kl_coef=0.1)
    noise = 2 * policy_bounds(exp, np64(z), old, ref, adv, w, 1.0, 0.1)[1][0] + 8 * U
    for seed in range(4):
        v = torch.from_numpy(np.random.default_rng(seed).uniform(-1, 1, (rows, vocab)).astype(np.float32)).cuda()
        num = (call(z + step * v, None) - call(z - step * v, None)) / (2 * step)
        ana = (d.double() * v.double()).sum().item()
        assert abs(num - ana) <= 30 * step * step / 6 + noise / step, (num, ana)


@pytest.mark.parametrize("dtype", [rs.RS_F32, rs.RS_BF16])
@pytest.mark.parametrize("vocab", [100, 5000, 40000])
def test_values_that_take_no_part_leave_no_trace(dtype, vocab):
    """NaN and infinities in rows without a token, of weight 0 or of nothing
    but -inf; masked vocabulary; a NaN row that keeps to itself."""
    log(f"masked values vocab={vocab} dtype={dtype}")
    rows = 8
    _, z = make_logits(rows, vocab, vocab, dtype, 11)
    y = np.random.default_rng(12).integers(vocab // 2, vocab, rows)
    z[0] = float("nan"); y[0] = -1                    # no token
    z[1, 3] = float("inf")                            # weight 0
    z[2] = -float("inf")                              # nothing to score
    z[3, :vocab // 2] = -float("inf")                 # masked vocabulary
    z[4] = torch.finfo(TORCH[dtype]).min              # masks of the lowest value
    z[4, int(y[4])] = 1.0
    z[7] = torch.finfo(TORCH[dtype]).min              # a row of nothing but them: even shares
    z64 = np64(z)
    old, ref, adv, w = policy_inputs(rows, np.where(np.isfinite(z64), z64, -1e30), y, 1.0, 13)
    w[1] = 0
    old[0] = adv[0] = ref[0] = old[1] = adv[1] = ref[2] = adv[2] = np.nan
    w[5] = 0.1
    dev = [torch.from_numpy(a).cuda() for a in (old, ref, adv, w)]
    yt = torch.from_numpy(y).cuda()
    d = torch.full((rows, vocab), SENT, dtype=TORCH[dtype], device="cuda")
    logp, stats = torch.zeros(rows, device="cuda"), torch.zeros(4, device="cuda")
    work, n = work_for(rows, vocab)
    rs.rs_policy_loss(z, dtype, rows, vocab, vocab, yt, *dev, d, vocab, logp, stats, work, n, kl_coef=0.1)
    exp = ob.policy_loss(z64, y, old, ref, adv, w, kl_coef=0.1)
    assert list(np.nonzero(~exp["live"])[0]) == [0, 1, 2] and np.isfinite(exp["stats"]).all()
    dcoef, dstats = policy_bounds(exp, z64, old, np.nan_to_num(ref), adv, w, 1.0, 0.1)
    _, ds = row_bounds(z64, 1.0)
    close(np64(logp), exp["logp"], ds + 1.01 * U * np.abs(exp["logp"]), "logp")
    close(np64(stats), exp["stats"], dstats, "stats")
    check_gradient(np64(d), exp, z64, y, 1.0, dcoef, dtype, "dlogits")
    assert not d[3, :vocab // 2].any()
    # a NaN in one live row makes that row and the loss NaN, nothing else
    good = d.clone()
    z[6, vocab - 1] = float("nan")
    rs.rs_policy_loss(z, dtype, rows, vocab, vocab, yt, *dev, d, vocab, logp, stats, work, n, kl_coef=0.1)
    assert torch.isnan(stats[0]) and torch.isnan(logp[6]) and torch.isnan(d[6]).all()
    keep = [0, 1, 2, 3, 4, 5, 7]
    assert torch.equal(d[keep], good[keep])
    # a token of probability 0 in a row of others
    z[6] = 0
    z[6, int(y[6])] = -float("inf")
    rs.rs_token_logp(z, dtype, rows, vocab, vocab, yt, logp, work, n)
    assert logp[6].item() == -math.inf and logp[2].item() == 0


def test_no_rows():
    log("no rows")
    work, n = work_for(0, 10)
    stats = torch.full((4,), SENT, device="cuda")
    rs.rs_token_logp(None, rs.RS_F32, 0, 10, 10, None, None, work, n)
    rs.rs_policy_loss(None, rs.RS_F32, 0, 10, 10, None, None, None, None, None, None, 10, None, stats, work, n)
    assert not stats.any()
    stats.fill_(SENT)
    start = torch.zeros(5, dtype=torch.int64, device="cuda")
    work, n = work_for(0, 10, 4)
    seq = torch.full((4,), SENT, device="cuda")
    rs.rs_preference_loss(None, rs.RS_F32, 0, 10, 10, None, start, 2, None, None, None, 10, seq, stats, work, n)
    assert not seq.any() and abs(stats[0].item() - math.log(2)) < 1e-6 and stats[3] == SENT


# ------------------------------------------------------------ preference

def preference_bounds(exp, z64, start, pairs, w, temp, beta, kind, average):
    _, ds = row_bounds(z64, temp)
    dl = np.where(exp["live"], ds, 0)
    dseq = np.zeros(2 * pairs)
    cnt = np.ones(2 * pairs)
    for s in range(2 * pairs):
        a, b = int(start[s]), int(start[s + 1])
        cnt[s] = max(exp["live"][a:b].sum(), 1) if average else 1
        dseq[s] = dl[a:b].sum() / cnt[s]
    dD = dseq[:pairs] + dseq[pairs:]
    curve = 2.0 if kind == ob.IPO else beta * beta / 4  # |d2 loss / dD2|
    dper = np.tile(np.abs(w) * curve * dD, 2)
    dcoef = np.zeros(len(dl))
    for s in range(2 * pairs):
        dcoef[int(start[s]):int(start[s + 1])] = dper[s] / cnt[s]
    dcoef = dcoef * 1.01 + U * np.abs(exp["coef"])
    slope = np.abs(exp["per_seq"][:pairs])
    dstats = np.array([(slope * dD + np.abs(w) * curve * dD * dD).sum(), (np.abs(w) * beta * dD).sum(), 0.0])
    return dseq, dcoef, dstats * 1.01 + 1.01 * U * np.abs(exp["stats"]) + 1e-12


PREF = [
    # lengths (preferred, then others), rows in front, behind, vocab, pad, dtype, kind, smoothing, margin, average
    ([1], [1], 0, 0, 17, 0, rs.RS_F32, ob.SIGMOID, 0.0, 0.0, False),
    ([3, 0], [2, 5], 1, 2, 65, 2, rs.RS_BF16, ob.SIGMOID, 0.1, 0.3, False),
    ([4, 9, 2], [1, 1, 7], 0, 3, 1031, 0, rs.RS_F32, ob.IPO, 0.0, 0.0, True),
    ([5, 0, 1], [2, 0, 3], 2, 0, 3001, 0, rs.RS_BF16, ob.HINGE, 0.0, -0.4, False),
    ([6, 30], [20, 11], 0, 5, 8209, 0, rs.RS_BF16, ob.SIGMOID, 0.0, 0.0, True),
    ([2, 3], [4, 2], 0, 1, 70001, 0, rs.RS_BF16, ob.SIGMOID, 0.0, 0.1, True),
    ([1] * 300, [1] * 300, 3, 4, 24, 0, rs.RS_F32, ob.SIGMOID, 0.05, 0.0, False),
]


@pytest.mark.parametrize("case", PREF, ids=[f"pref{i}" for i in range(len(PREF))])
@pytest.mark.parametrize("refs", [True, False])
def test_preference_loss(case, refs):
    first, second, front, behind, vocab, pad, dtype, kind, ls, margin, average = case
    log(f"preference_loss {case[2:]} refs={refs}")
    pairs = len(first)
    start = front + np.concatenate([[0], np.cumsum(first + second)]).astype(np.int64)
    rows = int(start[-1]) + behind
    _, z = make_logits(rows, vocab, vocab + pad, dtype, 21)
    z64 = np64(z)
    rng = np.random.default_rng(22)
    y = rng.integers(0, vocab, rows)
    y[rng.uniform(size=rows) < 0.2] = -1
    w = rng.uniform(0.3, 1, pairs).astype(np.float32)
    if pairs > 2:
        w[1] = 0
    beta, temp = 0.2, 0.9
    args = dict(temperature=temp, beta=beta, label_smoothing=ls, margin=margin, kind=kind, average=average)
    seq = ob.preference_loss(z64, y, start, pairs, None, np.ones(pairs), **args)["seq_logp"]
    ref = (seq + rng.normal(0, 1.5, 2 * pairs)).astype(np.float32) if refs else None
    exp = ob.preference_loss(z64, y, start, pairs, ref, w, **args)
    yt, st = torch.from_numpy(y).cuda(), torch.from_numpy(start).cuda()
    rt = torch.from_numpy(ref).cuda() if refs else None
    wt = torch.from_numpy(w).cuda()
    d = torch.full((rows, vocab + 1), SENT, dtype=TORCH[dtype], device="cuda")
    seq_logp, stats = torch.zeros(2 * pairs, device="cuda"), torch.full((4,), SENT, device="cuda")
    work, n = work_for(rows, vocab, 2 * pairs)
    rs.rs_preference_loss(z, dtype, rows, vocab, vocab + pad, yt, st, pairs, rt, wt, d, vocab + 1,
                          seq_logp, stats, work, n, **args)
    torch.cuda.synchronize()
    dseq, dcoef, dstats = preference_bounds(exp, z64, start, pairs, w, temp, beta, kind, average)
    close(np64(seq_logp), exp["seq_logp"], dseq * 1.01 + 1.01 * U * np.abs(exp["seq_logp"]), "seq_logp")
    close(np64(stats)[:3], exp["stats"], dstats, "stats")
    assert stats[3] == SENT and (d[:, vocab] == SENT).all()
    ins = exp["inside"]
    assert (d[torch.from_numpy(~ins).cuda()] == SENT).all()
    sub = {k: exp[k][ins] for k in ("live", "coef", "p", "dlogits")}
    check_gradient(np64(d)[ins][:, :vocab], sub, z64[ins], y[ins], temp, dcoef[ins], dtype, "dlogits")
    # loss alone; in place: the same bits, rows outside kept
    stats2 = torch.zeros(3, device="cuda")
    rs.rs_preference_loss(z, dtype, rows, vocab, vocab + pad, yt, st, pairs, rt, wt, None, vocab, None,
                          stats2, work, n, **args)
    assert torch.equal(stats2, stats[:3])
    zin = z.clone()
    z0 = z.clone()
    rs.rs_preference_loss(zin, dtype, rows, vocab, vocab, yt, st, pairs, rt, wt, zin, vocab, None,
                          stats2, work, n, **args)
    keep = torch.from_numpy(ins).cuda()
    assert torch.equal(stats2, stats[:3]) and torch.equal(zin[~keep], z0[~keep])
    assert torch.equal(zin[keep], d[keep][:, :vocab])
    # equal weights are the default
    rs.rs_preference_loss(z, dtype, rows, vocab, vocab + pad, yt, st, pairs, rt, None, None, vocab,
                          None, stats2, work, n, **args)
    e = ob.preference_loss(z64, y, start, pairs, ref, None, **args)
    close(np64(stats2), e["stats"],
          preference_bounds(e, z64, start, pairs, np.full(pairs, 1 / pairs), temp, beta, kind, average)[2], "mean")


def test_preference_extremes():
    """Very sure pairs on either side, in binary32 logits: finite losses and
    slopes that go to 0 and to beta."""
    log("preference extremes")
    rows, vocab = 4, 16
    z = torch.zeros(rows, vocab, device="cuda")
    z[0, 1] = z[1, 2] = 3000.0   # preferred: certain, others impossible-like
    y = torch.tensor([1, 0, 0, 2], device="cuda")      # l: 0, -3000, 0-ish, ...
    z[2] = z[0]
    z[3] = z[1]
    start = torch.arange(5, device="cuda")
    d = torch.zeros(rows, vocab, device="cuda")
    stats, seq = torch.zeros(3, device="cuda"), torch.zeros(4, device="cuda")
    work, n = work_for(rows, vocab, 4)
    rs.rs_preference_loss(z, rs.RS_F32, rows, vocab, vocab, y, start, 2, None, None, d, vocab, seq, stats,
                          work, n, beta=1.0)
    # pair 0: l = 0 against l(z[2], 0) = -3000; pair 1: -3000 against 0
    assert seq.tolist() == [0.0, -3000.0, -3000.0, 0.0]
    assert stats.tolist() == [1500.0, 0.0, 0.5]
    exp = ob.preference_loss(np64(z), y.cpu().numpy(), np.arange(5), 2, None, None, beta=1.0)
    assert np.allclose(np64(d), exp["dlogits"], atol=1e-6)


# ---------------------------------------------------- streams and graphs

def test_captured_and_replayed_on_another_stream():
    """Both losses and the log-probability captured once with one scratch
    area; every replay equals eager calls bit for bit, on inputs that change
    between replays."""
    log("objectives graph")
    rows, vocab, pairs = 40, 9001, 3
    _, z = make_logits(rows, vocab, vocab, rs.RS_BF16, 31)
    y = torch.from_numpy(targets_of(rows, vocab, 32)).cuda()
    old, ref, adv, w = [torch.from_numpy(a).cuda() for a in policy_inputs(rows, np64(z), targets_of(rows, vocab, 32), 1.0, 33)]
    start = torch.tensor([0, 5, 9, 20, 22, 30, 38], device="cuda")
    nb = rs.rs_objective_bytes(rows, vocab, 2 * pairs)

    def arrays():
        return {"work": torch.full((nb,), 0xFF, dtype=torch.uint8, device="cuda"),
                "d": torch.zeros(rows, vocab, dtype=torch.bfloat16, device="cuda"),
                "e": torch.zeros(rows, vocab, dtype=torch.bfloat16, device="cuda"),
                "logp": torch.zeros(rows, device="cuda"), "l2": torch.zeros(rows, device="cuda"),
                "s": torch.zeros(4, device="cuda"), "t": torch.zeros(3, device="cuda"),
                "seq": torch.zeros(2 * pairs, device="cuda")}

    def sequence(a):
        rs.rs_token_logp(z, rs.RS_BF16, rows, vocab, vocab, y, a["l2"], a["work"], nb)
        rs.rs_policy_loss(z, rs.RS_BF16, rows, vocab, vocab, y, old, ref, adv, w, a["d"], vocab,
                          a["logp"], a["s"], a["work"], nb, kl_coef=0.1)
        rs.rs_preference_loss(z, rs.RS_BF16, rows, vocab, vocab, y, start, pairs, None, None, a["e"],
                              vocab, a["seq"], a["t"], a["work"], nb)

    eager, graphed = arrays(), arrays()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        sequence(graphed)
    torch.cuda.synchronize()
    assert not graphed["d"].any() and not graphed["s"].any()  # capture ran nothing
    for k in range(4):
        z.add_(torch.randn(rows, vocab, device="cuda", generator=torch.Generator(device="cuda").manual_seed(k)) * 0.5)
        sequence(eager)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for name in eager:
            if name != "work":
                assert torch.equal(eager[name], graphed[name]), (k, name)
    # on a stream of its own with its own scratch, beside the current one
    other = arrays()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        sequence(other)
    sequence(eager)
    torch.cuda.synchronize()
    for name in eager:
        if name != "work":
            assert torch.equal(eager[name], other[name]), name
    del graph


def test_rows_behind_32_bit_offsets():
    """33500 rows of 128256 bf16 logits: more than 2^32 elements.  The rows
    at both ends against the oracle, the rest by their sums (a gradient row
    adds up to 0)."""
    log("beyond 2^32 elements")
    rows, vocab = 33500, 128256
    g = torch.Generator(device="cuda").manual_seed(1)
    z = torch.empty(rows, vocab, dtype=torch.bfloat16, device="cuda")
    z.normal_(0, 2.5, generator=g)
    ends = [0, 1, rows // 2, rows - 2, rows - 1]
    y = torch.full((rows,), -1, dtype=torch.int64, device="cuda")
    y[::7] = 128255
    y[ends] = torch.tensor([0, 5, 77, 128255, 64000], device="cuda")
    one, adv = torch.zeros(rows, device="cuda"), torch.ones(rows, device="cuda")
    work, n = work_for(rows, vocab)
    logp, stats = torch.zeros(rows, device="cuda"), torch.zeros(4, device="cuda")
    rs.rs_token_logp(z, rs.RS_BF16, rows, vocab, vocab, y, logp, work, n)
    old = logp.clone()
    z64 = np64(z[ends])
    rs.rs_policy_loss(z, rs.RS_BF16, rows, vocab, vocab, y, old, None, adv, adv, z, vocab, logp, stats, work, n)
    torch.cuda.synchronize()
    yn = y[ends].cpu().numpy()
    oldn = old[ends].cpu().numpy()
    exp = ob.policy_loss(z64, yn, oldn, None, np.ones(5), np.ones(5))
    dcoef, _ = policy_bounds(exp, z64, oldn, oldn, np.ones(5), np.ones(5), 1.0, 0.0)
    check_gradient(np64(z[ends]), exp, z64, yn, 1.0, dcoef, rs.RS_BF16, "ends")
    live = y >= 0
    assert not z[~live].any()
    # r = 1 up to the rounding of old: the token's value is p - 1, the others p
    off = z[live].float().sum(1).abs().max().item()
    assert off < 2.0 ** -8 * 2.0  # half a step on each of values that add up to 2 in size


def test_more_rows_than_one_launch_takes():
    """2^22 + 9 rows of 3 values: the launches are cut into slices or stride
    over the rows; against torch in binary64, row sums of the gradient 0."""
    log("more rows than a launch takes")
    rows, vocab = (1 << 22) + 9, 3
    g = torch.Generator(device="cuda").manual_seed(2)
    z = torch.randn(rows, vocab, device="cuda", generator=g)
    y = torch.randint(-1, vocab, (rows,), device="cuda", generator=g)
    work, n = work_for(rows, vocab)
    logp, again = torch.full((rows,), SENT, device="cuda"), torch.full((rows,), SENT, device="cuda")
    rs.rs_token_logp(z, rs.RS_F32, rows, vocab, vocab, y, logp, work, n)
    full = torch.log_softmax(z.double(), -1)
    exp = torch.where(y >= 0, full.gather(1, y.clamp(min=0)[:, None])[:, 0], torch.zeros_like(full[:, 0]))
    bound = (9 * (3 * 12 + 3) + 4 + 12) * U  # values within 12 of each other
    assert (logp.double() - exp).abs().max().item() < bound
    one, d, stats = torch.ones(rows, device="cuda"), torch.full_like(z, SENT), torch.zeros(4, device="cuda")
    rs.rs_policy_loss(z, rs.RS_F32, rows, vocab, vocab, y, logp, None, one, one, d, vocab, again, stats, work, n)
    assert (again.double() - exp).abs().max().item() < bound
    p = full.exp()
    p[y >= 0] = p[y >= 0].scatter_add(1, y[y >= 0][:, None], -torch.ones_like(p[y >= 0][:, :1]))
    p[y < 0] = 0
    # r = exp(logp - its rounding) is off by u |logp|, and the bounds above
    assert (d.double() - p).abs().max().item() < 2 * bound
    live = int((y >= 0).sum())
    assert abs(stats[0].item() + live) <= live * (bound + 2 * U)


def test_kl_weight_of_zero_leaves_the_reference_out():
    log("policy kl_coef 0 with a reference")
    rows, vocab = 5, 50
    z = torch.randn(rows, vocab, device="cuda")
    y = torch.arange(rows, device="cuda")
    one = torch.ones(rows, device="cuda")
    work, n = work_for(rows, vocab)
    a, b = torch.zeros(rows, vocab, device="cuda"), torch.zeros(rows, vocab, device="cuda")
    s, t = torch.zeros(4, device="cuda"), torch.zeros(4, device="cuda")
    far = torch.full((rows,), 1e5, device="cuda")  # exp(ref - logp) overflows
    rs.rs_policy_loss(z, rs.RS_F32, rows, vocab, vocab, y, one, far, one, one, a, vocab, None, s, work, n)
    rs.rs_policy_loss(z, rs.RS_F32, rows, vocab, vocab, y, one, None, one, one, b, vocab, None, t, work, n)
    assert torch.equal(a, b) and s[0] == t[0] and torch.isfinite(s[:2]).all()
