"""Pins of the objectives' oracle (oracle/objectives.py): log-probabilities
and losses against torch's own functions in binary64, gradients against
central differences of the losses."""
import numpy as np
import pytest
import torch

from oracle import objectives as ob


def _case(seed, rows=7, vocab=11):
    rng = np.random.default_rng(seed)
    z = rng.normal(0, 2, (rows, vocab))
    y = rng.integers(0, vocab, rows)
    y[2] = -1
    return rng, z, y


def _differences(f, z, step=1e-6):
    d = np.zeros_like(z)
    for i in np.ndindex(z.shape):
        hi, lo = z.copy(), z.copy()
        hi[i] += step
        lo[i] -= step
        d[i] = (f(hi) - f(lo)) / (2 * step)
    return d


def test_token_logp_is_torchs_log_softmax():
    _, z, y = _case(0)
    z[4, 3] = -np.inf
    logp, lse, live, p = ob.token_logp(z, y, 0.7)
    ref = torch.log_softmax(torch.from_numpy(z) / 0.7, -1).numpy()
    for t in range(len(y)):
        assert live[t] == (y[t] >= 0)
        if live[t]:
            assert abs(logp[t] - ref[t, y[t]]) < 1e-12
            assert np.allclose(p[t], np.exp(ref[t]), atol=1e-14)
    logp, lse, live, _ = ob.token_logp(np.full((1, 3), -np.inf), np.array([1]))
    assert logp[0] == 0 and not live[0]


@pytest.mark.parametrize("kl", [0.0, 0.3])
def test_policy_loss_value_and_gradient(kl):
    rng, z, y = _case(1)
    base = ob.token_logp(z, y, 1.3)[0]
    old = base - np.array([0.0, 0.5, 0, -0.5, 0.5, -0.5, 0.01])
    adv = np.array([1.0, 1.0, 5.0, 1.0, -1.0, -1.0, -0.3])
    ref = base + rng.normal(0, 0.3, 7)
    w = rng.uniform(0.1, 1, 7)
    w[6] = 0
    args = dict(temperature=1.3, clip_low=0.2, clip_high=0.28, kl_coef=kl)
    got = ob.policy_loss(z, y, old, ref, adv, w, **args)
    zt = torch.from_numpy(z).requires_grad_(True)
    keep = torch.tensor([t for t in range(7) if y[t] >= 0 and w[t] != 0])
    l = torch.log_softmax(zt / 1.3, -1)[keep, torch.from_numpy(y)[keep]]
    a, wt = torch.from_numpy(adv)[keep], torch.from_numpy(w)[keep]
    r = torch.exp(l - torch.from_numpy(old)[keep])
    pg = -torch.minimum(a * r, a * r.clamp(0.8, 1.28))
    away = torch.from_numpy(ref)[keep] - l
    loss = (wt * (pg + kl * (torch.exp(away) - 1 - away))).sum()
    loss.backward()
    assert abs(got["stats"][0] - loss.item()) < 1e-12
    assert np.allclose(got["dlogits"], zt.grad.numpy(), atol=1e-13)
    assert got["stats"][3] == pytest.approx(w[1] + w[5])  # r > 1.28 with A > 0, r < 0.8 with A < 0
    diff = _differences(lambda x: ob.policy_loss(x, y, old, ref, adv, w, **args)["stats"][0], z)
    assert np.allclose(got["dlogits"], diff, atol=1e-8)


@pytest.mark.parametrize("kind,ls,margin", [(ob.SIGMOID, 0.0, 0.0), (ob.SIGMOID, 0.1, 0.2),
                                            (ob.HINGE, 0.0, 0.1), (ob.IPO, 0.0, 0.0)])
@pytest.mark.parametrize("average", [False, True])
def test_preference_loss_value_and_gradient(kind, ls, margin, average):
    rng, z, y = _case(2, rows=14)
    y[2] = 5
    y[6] = 99
    start = np.array([1, 4, 4, 9, 12])     # row 0 and rows 12, 13 outside; sequence 1 empty
    ref, w = rng.normal(-5, 1, 4), np.array([0.6, 0.4])
    args = dict(beta=0.3, label_smoothing=ls, margin=margin, kind=kind, average=average)
    got = ob.preference_loss(z, y, start, 2, ref, w, **args)
    lt = torch.log_softmax(torch.from_numpy(z), -1)
    L = torch.zeros(4, dtype=torch.float64)
    for s in range(4):
        rows = [t for t in range(start[s], start[s + 1]) if y[t] < 11]
        for t in rows:
            L[s] += lt[t, y[t]] / (len(rows) if average else 1)
    d = (L - torch.from_numpy(ref))[:2] - (L - torch.from_numpy(ref))[2:]
    h = 0.3 * d - margin
    each = {ob.SIGMOID: -(1 - ls) * torch.nn.functional.logsigmoid(h)
            - ls * torch.nn.functional.logsigmoid(-h),
            ob.HINGE: torch.relu(1 - h), ob.IPO: (d - 1 / 0.6) ** 2}[kind]
    assert np.allclose(got["seq_logp"], L.numpy())
    assert abs(got["stats"][0] - (torch.from_numpy(w) * each).sum().item()) < 1e-12
    diff = _differences(lambda x: ob.preference_loss(x, y, start, 2, ref, w, **args)["stats"][0], z)
    assert np.allclose(got["dlogits"], diff, atol=1e-8)
    assert not got["dlogits"][[0, 6, 12, 13]].any()


@pytest.mark.parametrize("score,zc", [(ob.SOFTMAX, 0.0), (ob.SOFTMAX, 0.05),
                                      (ob.NORMALISED_SIGMOID, 0.0)])
def test_router_balance_value_and_gradient(score, zc):
    rng = np.random.default_rng(3)
    z = rng.normal(0, 1.5, (12, 5))
    topk = np.argsort(-z, axis=1)[:, :2]
    topk[4] = [3, 3]
    topk[5, 1] = -1
    mask = np.ones(12)
    mask[6] = 0
    start = [1, 6, 6, 11]
    got = ob.router_balance(z, topk, mask, start, 0.4, zc, score)
    assert got["counts"][0, 3] >= 2 and got["counts"][1].sum() == 0
    assert got["counts"].sum() == 2 * 9 - 1
    p = torch.softmax(torch.from_numpy(z), -1) if score == ob.SOFTMAX else torch.sigmoid(torch.from_numpy(z))
    p = (p / p.sum(-1, keepdim=True)).numpy()
    loss = 0.0
    for s, rows in ((0, [1, 2, 3, 4, 5]), (2, [7, 8, 9, 10])):
        f = got["counts"][s] * 5 / (2 * len(rows))
        loss += 0.4 * (f * p[rows].mean(0)).sum()
        assert np.allclose(got["mean_prob"][s], p[rows].mean(0))
    assert abs(got["stats"][0] - loss) < 1e-12

    def total(x):
        return ob.router_balance(x, topk, mask, start, 0.4, zc, score)["stats"].sum()

    assert np.allclose(got["dlogits"], _differences(total, z), atol=1e-8)
    assert not got["dlogits"][[0, 6, 11]].any()


def test_router_sigmoid_shares_of_far_negative_rows():
    z = np.array([[-200.0, -201.0, -230.0]])
    got = ob.router_balance(z, np.array([[0]]), None, [0, 1], score=ob.NORMALISED_SIGMOID)
    assert np.allclose(got["mean_prob"][0], torch.softmax(torch.from_numpy(z), -1).numpy())
