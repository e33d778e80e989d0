"""GPU parity of the router balance loss with the binary64 oracle
(oracle/objectives.py).

Tolerances, from the arithmetic of the kernel (u = 2^-24, half a step of
binary32; X the larger of a row's largest |z| and its range, held at 90
where exponentials are 0 anyway):
  a share p: exponential e = (3 X + 7) u, sum 30 additions in a chain,
      quotient: d_p = 2 e + 34 u of it;
  f (count times a rounded share) 2 u, sum f p: d_p + 44 u of it;
  a gradient value slope c1 (f - dot): slope c1 ((d_p + 4 u) |f - dot|
      + 2 u f + (d_p + 44 u) dot), with 2 zc / n (p d_lse + |lse| p d_p),
      d_lse = e + 32 u + 3 u |lse|, and half a step of its type;
  a mean: d_p and a chain of at most 96 binary32 additions;
  the losses: the same errors summed, and half a step.
"""
import numpy as np
import pytest
import torch

import sharded_state_raggedshard_amd as rs
from gpu_harness import log
from oracle import objectives as ob
from test_gpu_objectives import HALF, SENT, TORCH, U, close, make_logits, np64

pytestmark = pytest.mark.gpu

SCORES = {"softmax": (rs.RS_SCORE_SOFTMAX, ob.SOFTMAX), "sigmoid": (rs.RS_SCORE_SIGMOID, ob.NORMALISED_SIGMOID)}


def bounds(exp, z, mask, start, k, balance_coef, z_coef, score):
    """(dlogits, mean, stats) tolerances."""
    rows, experts = z.shape
    dg, dm = np.zeros_like(z), np.zeros_like(exp["mean_prob"])
    ds = np.zeros(2)
    for s in range(len(start) - 1):
        a, b = int(start[s]), int(start[s + 1])
        tokens = [t for t in range(a, b) if mask is None or mask[t]]
        n = max(len(tokens), 1)
        f = exp["counts"][s] * (experts / (k * n))
        for t in tokens:
            x = z[t]
            fin = x[np.isfinite(x)]
            if not fin.size:
                continue
            X = min(max(np.abs(fin).max(), fin.max() - fin.min()), 90.0)
            e = (3 * X + 7) * U
            dp = 2 * e + 34 * U
            p, lse = ob.softmax_row(x, 1.0)
            slope = p
            if score == ob.NORMALISED_SIGMOID:
                ls = -np.logaddexp(0.0, -x)
                p = np.exp(ls - ls.max())
                p /= p.sum()
                slope = p * np.exp(-np.logaddexp(0.0, x))
                dp += e + 6 * U
            dot = f @ p
            dlse = e + 32 * U + 3 * U * abs(lse)
            dg[t] = (balance_coef / n * slope * ((dp + 4 * U) * np.abs(f - dot) + 2 * U * f + (dp + 44 * U) * dot)
                     + 2 * z_coef / n * p * (dlse + abs(lse) * (dp + 3 * U)))
            dm[s] += dp * p / n
            ds += np.array([balance_coef * (dp + 44 * U) * dot / n, z_coef * 2 * abs(lse) * dlse / n])
    return (dg * 1.01, dm * 1.01 + 97 * U * exp["mean_prob"], ds * 1.01 + 1.01 * U * np.abs(exp["stats"]))


def run(z, dtype, ld, topk, mask, start, d, ldd, **kw):
    rows, experts = z.shape
    n_seq = 1 if start is None else len(start) - 1
    counts = torch.full((n_seq * experts + 1,), 77, dtype=torch.int32, device="cuda")
    mean = torch.full((n_seq * experts + 1,), SENT, device="cuda")
    stats = torch.full((3,), SENT, device="cuda")
    nb = rs.rs_router_balance_bytes(rows, experts, n_seq)
    work = torch.full((nb,), 0xFF, dtype=torch.uint8, device="cuda")
    rs.rs_router_balance(z, dtype, rows, experts, ld, topk, topk.shape[1], topk.stride(0), mask, start, n_seq,
                         d, ldd, counts, mean, stats, work, nb, **kw)
    torch.cuda.synchronize()
    assert counts[-1] == 77 and mean[-1] == SENT and stats[2] == SENT
    return counts[:-1].view(n_seq, experts), mean[:-1].view(n_seq, experts), stats[:2]


# (sequence starts or None, rows, experts, k, ld - experts, shift, dtype, masked share)
CASES = [
    (None, 1, 1, 1, 0, 0, rs.RS_F32, 0), (None, 1, 8, 2, 0, 0, rs.RS_BF16, 0),
    (None, 7, 2, 1, 1, 1, rs.RS_F32, 0), (None, 96, 32, 4, 0, 0, rs.RS_F32, 0),
    ([0, 5, 5, 40, 61], 61, 31, 3, 0, 0, rs.RS_BF16, 0.3), ([2, 64, 65, 200], 203, 33, 2, 3, 1, rs.RS_F32, 0),
    (None, 130, 60, 6, 0, 0, rs.RS_BF16, 0.5), ([0, 300], 300, 64, 8, 0, 0, rs.RS_F32, 0),
    ([0, 0, 129, 129, 129, 700], 700, 100, 4, 4, 3, rs.RS_BF16, 0.1), (None, 1000, 128, 4, 0, 0, rs.RS_F32, 0.05),
    ([7, 90, 91, 92, 400], 401, 160, 6, 0, 0, rs.RS_BF16, 0), ([0, 64, 128, 192, 256], 256, 256, 8, 0, 0, rs.RS_BF16, 0),
    (None, 257, 257, 8, 0, 0, rs.RS_F32, 0), (None, 65, 384, 6, 0, 0, rs.RS_F32, 0.2),
    ([0, 30, 77], 77, 512, 8, 0, 0, rs.RS_BF16, 0), ([1, 30, 70], 70, 513, 8, 1, 0, rs.RS_BF16, 0),
    (None, 40, 1000, 1, 0, 0, rs.RS_F32, 0), (None, 33, 1024, 16, 0, 0, rs.RS_BF16, 0),
    (None, 20, 1023, 4, 0, 5, rs.RS_F32, 0), ([i * 3 for i in range(200)] + [700], 700, 16, 2, 0, 0, rs.RS_BF16, 0.1),
    (None, 150001, 8, 2, 0, 0, rs.RS_BF16, 0),
    # shorter on average than a counting workgroup's share; as many sequences as rows; more; few long ones
    ([min(5 + i * i // 3, 1300) for i in range(64)], 1302, 40, 4, 0, 0, rs.RS_F32, 0.1),
    (list(range(91)), 90, 48, 2, 0, 0, rs.RS_BF16, 0),
    ([i // 3 for i in range(121)], 40, 24, 2, 0, 0, rs.RS_F32, 0.2),
    ([0, 900, 901, 4000, 4000, 9000, 9000, 9000, 9000, 9001, 9700], 9700, 24, 2, 0, 0, rs.RS_BF16, 0.1),
]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("case", CASES, ids=[f"{c[1]}x{c[2]}k{c[3]}" for c in CASES])
def test_router_balance(case, score):
    starts, rows, experts, k, pad, shift, dtype, masked = case
    log(f"router_balance {case[1:]} {score}")
    ld = experts + pad
    _, z = make_logits(rows, experts, ld, dtype, 41, shift, sigma=1.5)
    rng = np.random.default_rng(42)
    z64 = np64(z)
    topk = np.argsort(-z64, axis=1, kind="stable")[:, :k].copy()
    if rows > 4 and experts > 3:
        topk[1, 0], topk[2, -1] = -1, experts       # no expert
        topk[3] = 2                                 # one expert k times
    mask = None if not masked else (rng.uniform(size=rows) >= masked)
    start = [0, rows] if starts is None else starts
    kw = dict(balance_coef=0.3, z_coef=0.05 if score == "softmax" else 0.0)
    exp = ob.router_balance(z64, topk, mask, start, score=SCORES[score][1], **kw)
    ldk = k + 1
    tk = torch.full((rows, ldk), -5, dtype=torch.int64, device="cuda")
    tk[:, :k] = torch.from_numpy(topk).cuda()
    mt = None if mask is None else torch.from_numpy(mask.astype(np.uint8) * 3).cuda()
    st = None if starts is None else torch.tensor(starts, dtype=torch.int64, device="cuda")
    d = torch.full((rows, experts + 1), SENT, dtype=TORCH[dtype], device="cuda")
    args = (mt, st)
    counts, mean, stats = run(z, dtype, ld, tk[:, :k], *args, d, experts + 1, score=SCORES[score][0], **kw)
    assert np.array_equal(counts.cpu().numpy(), exp["counts"])
    tol_d, tol_m, tol_s = bounds(exp, z64, mask, start, k, kw["balance_coef"], kw["z_coef"], SCORES[score][1])
    close(np64(mean).ravel(), exp["mean_prob"].ravel(), tol_m.ravel(), "mean_prob")
    close(np64(stats), exp["stats"], tol_s, "stats")
    ins = exp["inside"]
    got = np64(d)
    assert (got[:, experts] == SENT).all() and (got[~ins] == SENT).all()
    close(got[ins][:, :experts].ravel(), exp["dlogits"][ins].ravel(),
          (tol_d[ins] + HALF[dtype] * np.abs(exp["dlogits"][ins]) + 1e-37).ravel(), "dlogits")
    if mask is not None:
        assert not got[ins & ~mask][:, :experts].any()
    # loss alone, and in place: the same bits
    c2, m2, s2 = run(z, dtype, ld, tk[:, :k], *args, None, experts, score=SCORES[score][0], **kw)
    assert torch.equal(c2, counts) and torch.equal(m2, mean) and torch.equal(s2, stats)
    inside = torch.from_numpy(ins).cuda()
    before = z.clone()
    c2, m2, s2 = run(z, dtype, ld, tk[:, :k], *args, z, ld, score=SCORES[score][0], **kw)
    assert torch.equal(s2, stats) and torch.equal(m2, mean)
    assert torch.equal(z[inside], d[inside][:, :experts]) and torch.equal(z[~inside], before[~inside])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [rs.RS_F32, rs.RS_BF16])
def test_far_and_masked_logits(dtype, score):
    """Rows far from 0 on either side, masked experts, a row of nothing but
    -inf, NaN in rows that take no part, and a NaN that stays in its row."""
    log(f"router far logits dtype={dtype} {score}")
    rows, experts, k = 70, 48, 3
    _, z = make_logits(rows, experts, experts, dtype, 51, sigma=1.5)
    topk = torch.randint(0, experts, (rows, k), device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    z[3] += 200
    z[4] -= 200
    z[5, ::2] = -float("inf")
    z[6] = -float("inf")
    z[7] = torch.finfo(TORCH[dtype]).min
    z[8, 5:] = torch.finfo(TORCH[dtype]).min
    z[9] = float("nan")
    mask = np.ones(rows, dtype=bool)
    mask[[9, 30]] = False
    z64 = np64(z)
    kw = dict(balance_coef=0.3, z_coef=0.0)
    ref = z64.copy()
    ref[9] = 0
    exp = ob.router_balance(ref, topk.cpu().numpy(), mask, [0, rows], score=SCORES[score][1], **kw)
    d = torch.full((rows, experts), SENT, dtype=TORCH[dtype], device="cuda")
    mt = torch.from_numpy(mask).cuda()
    counts, mean, stats = run(z, dtype, experts, topk, mt, None, d, experts, score=SCORES[score][0], **kw)
    assert np.array_equal(counts.cpu().numpy(), exp["counts"])
    tol_d, tol_m, tol_s = bounds(exp, ref, mask, [0, rows], k, 0.3, 0.0, SCORES[score][1])
    close(np64(mean).ravel(), exp["mean_prob"].ravel(), tol_m.ravel(), "mean_prob")
    close(np64(stats), exp["stats"], tol_s, "stats")
    close(np64(d).ravel(), exp["dlogits"].ravel(), (tol_d + HALF[dtype] * np.abs(exp["dlogits"]) + 1e-37).ravel(), "dlogits")
    assert not d[6].any() and not d[9].any() and not d[30].any()
    good = d.clone()
    z[20, 7] = float("nan")
    _, mean, stats = run(z, dtype, experts, topk, mt, None, d, experts, score=SCORES[score][0], **kw)
    assert torch.isnan(d[20]).all() and torch.isnan(stats[0]) and torch.isnan(mean).all()
    keep = [t for t in range(rows) if t != 20]
    assert torch.equal(d[keep], good[keep])


def test_no_rows_and_no_live_rows():
    log("router empty")
    counts, mean, stats = run(torch.empty(0, 8, device="cuda"), rs.RS_F32, 8, torch.empty(0, 2, dtype=torch.int64, device="cuda"),
                              None, torch.tensor([0, 0, 0], device="cuda"), None, 8)
    assert not counts.any() and not mean.any() and not stats.any()
    z = torch.randn(5, 8, device="cuda")
    d = torch.full((5, 8), SENT, device="cuda")
    counts, mean, stats = run(z, rs.RS_F32, 8, torch.zeros(5, 2, dtype=torch.int64, device="cuda"),
                              torch.zeros(5, dtype=torch.uint8, device="cuda"), None, d, 8, z_coef=0.1)
    assert not counts.any() and not mean.any() and not stats.any() and not d.any()


def test_captured_balance_replays_like_eager_calls():
    log("router graph")
    rows, experts, k = 3000, 128, 4
    z = torch.randn(rows, experts, device="cuda")
    start = torch.tensor([0, 700, 701, 3000], device="cuda")
    nb = rs.rs_router_balance_bytes(rows, experts, 3)
    topk = torch.zeros(rows, k, dtype=torch.int64, device="cuda")

    def arrays():
        return [torch.zeros(rows, experts, device="cuda"), torch.zeros(3, experts, dtype=torch.int32, device="cuda"),
                torch.zeros(3, experts, device="cuda"), torch.zeros(2, device="cuda"),
                torch.full((nb,), 0xFF, dtype=torch.uint8, device="cuda")]

    def call(a):
        rs.rs_router_balance(z, rs.RS_F32, rows, experts, experts, topk, k, k, None, start, 3, a[0], experts,
                             a[1], a[2], a[3], a[4], nb, z_coef=0.01)

    eager, graphed = arrays(), arrays()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(graphed)
    torch.cuda.synchronize()
    assert not graphed[0].any() and not graphed[1].any()
    for i in range(4):
        z.normal_(0, 1.5, generator=torch.Generator(device="cuda").manual_seed(i))
        topk.copy_(torch.topk(z, k).indices)
        call(eager)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(eager[:4], graphed[:4]):
            assert torch.equal(a, b), i
    del graph
