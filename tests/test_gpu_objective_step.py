"""The objectives inside a training step, as they are used together: the old
policy's log-probabilities, the policy loss (or a preference loss) and the
router's balance loss give the parameters' gradients, which go through the
grad DBuffer, the clipping norm and the int8 AdamW step.  Gradients against
torch's autograd in binary64, the step against the oracle; and the package's
example runs on them.

Tolerance of a parameter gradient, a sum over T tokens of dlogits x in
binary32 (torch's product): the logits are binary32 products over 64 hidden
values, off by at most 64 u of the sum of |x w| (below 40 here, so
64 * 40 u), which moves every p and coefficient by that; the sum adds T u of
its absolute terms; then half a step of bf16."""
import numpy as np
import pytest
import torch

import oracle
import sharded_state_raggedshard_amd as rs
from gpu_harness import log
from sharded_state_raggedshard_amd import example
from synth import ROWS, TILE, TensorSpec

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
T, HIDDEN, VOCAB, EXPERTS, K = 80, 64, 320, 32, 4


def autograd(x, w, router, target, topk, kind, old, ref, adv, start):
    """(dw, drouter) of the sum of the losses, binary64."""
    w, router = w.double().requires_grad_(True), router.double().requires_grad_(True)
    x = x.double()
    l = torch.log_softmax(x @ w.T, -1).gather(1, target[:, None])[:, 0]
    if kind == "policy":
        r = torch.exp(l - old.double())
        pg = -torch.minimum(adv.double() * r, adv.double() * r.clamp(0.8, 1.2))
        away = ref.double() - l
        loss = ((pg + 0.05 * (torch.exp(away) - away - 1)) / T).sum()
    else:
        n = (len(start) - 1) // 2
        seq = torch.stack([l[start[i]:start[i + 1]].sum() for i in range(2 * n)])
        loss = -torch.nn.functional.logsigmoid(0.1 * (seq[:n] - seq[n:])).mean()
    p = torch.softmax(x @ router.T, -1)
    f = torch.bincount(topk.reshape(-1), minlength=EXPERTS).double() * EXPERTS / (K * T)
    loss = loss + 0.01 * (f * p.mean(0)).sum()
    return torch.autograd.grad(loss, (w, router)), loss.item()


@pytest.mark.parametrize("kind", ["policy", "preference"])
def test_losses_to_parameters(kind):
    log(f"losses to parameters: {kind}")
    specs = [TensorSpec("w", (VOCAB, HIDDEN), ROWS, 32), TensorSpec("router", (EXPERTS, HIDDEN), TILE, 32, 32)]
    m = 4
    plan = rs.Plan(specs, m, 16, chunk=256).upload()
    L = oracle.Layout(specs, m, 16)
    gen = torch.Generator().manual_seed(5)
    dev = lambda t: t.cuda()  # noqa: E731
    w, router = (torch.randn(s.shape, generator=gen) * 0.3 for s in specs)
    x = torch.randn(T, HIDDEN, generator=gen)
    target = torch.randint(0, VOCAB, (T,), generator=gen)
    adv = torch.randn(T, generator=gen)
    logits, scores = dev(x) @ dev(w).T, dev(x) @ dev(router).T
    topk = scores.topk(K).indices
    start = [0, 9, 20, 20, 47, 60, 80]
    nb = max(rs.rs_objective_bytes(T, VOCAB, 6), rs.rs_router_balance_bytes(T, EXPERTS))
    work = torch.empty(nb, dtype=torch.uint8, device="cuda")
    old, logp = torch.zeros(T, device="cuda"), torch.zeros(T, device="cuda")
    rs.rs_token_logp(logits, rs.RS_F32, T, VOCAB, VOCAB, dev(target), old, work, nb)
    old = old + dev(torch.randn(T, generator=gen).mul(0.3))
    ref = old + dev(torch.randn(T, generator=gen).mul(0.2))
    # ratios away from the clipping borders
    r = torch.exp(torch.log_softmax(logits.double(), -1).gather(1, dev(target)[:, None])[:, 0] - old.double())
    old = torch.where(((r - 0.8).abs() < 1e-3) | ((r - 1.2).abs() < 1e-3), old + 0.01, old)
    dlogits, drouter = torch.zeros_like(logits), torch.zeros_like(scores)
    counts, mean = torch.zeros(EXPERTS, dtype=torch.int32, device="cuda"), torch.zeros(EXPERTS, device="cuda")
    stats, rstats = torch.zeros(4, device="cuda"), torch.zeros(2, device="cuda")
    if kind == "policy":
        rs.rs_policy_loss(logits, rs.RS_F32, T, VOCAB, VOCAB, dev(target), old, ref, dev(adv),
                          torch.full((T,), 1.0 / T, device="cuda"), dlogits, VOCAB, logp, stats, work, nb, kl_coef=0.05)
    else:
        rs.rs_preference_loss(logits, rs.RS_F32, T, VOCAB, VOCAB, dev(target), torch.tensor(start, device="cuda"), 3,
                              None, None, dlogits, VOCAB, None, stats, work, nb)
    rs.rs_router_balance(scores, rs.RS_F32, T, EXPERTS, EXPERTS, topk, K, K, None, None, 1, drouter, EXPERTS, counts,
                         mean, rstats, work, nb)
    grads = [dlogits.T @ dev(x), drouter.T @ dev(x)]
    (ew, er), loss = autograd(dev(x), dev(w), dev(router), dev(target), topk, kind, old, ref, dev(adv), start)
    assert (dev(x).abs() @ dev(w).abs().T).max().item() < 40
    noise = 64 * 40 * U
    assert abs(stats[0].item() + rstats[0].item() - loss) <= 4 * noise * (abs(loss) + 1)
    buf = torch.zeros(plan.total, dtype=torch.int16, device="cuda")
    theta = np.zeros(L.total, dtype=np.float32)
    for i, (g, e, d, v) in enumerate(zip(grads, (ew, er), (dlogits, drouter), (w, router))):
        size = d.abs().double().T @ dev(x).abs().double()
        # a coefficient's own error: at most 4 of its relative noise (ratio, KL slope, share)
        assert ((g.double() - e).abs() <= (4 * noise + T * U) * size + noise * size.mean()).all(), specs[i].name
        buf[plan.pos[i]:plan.pos[i] + g.numel()] = g.to(torch.bfloat16).reshape(-1).view(torch.int16)
        theta[L.pos[i]:L.pos[i] + v.numel()] = v.numpy().reshape(-1)
    # the step takes them
    sumsq, clip = torch.zeros(1, dtype=torch.float64, device="cuda"), torch.zeros(1, device="cuda")
    rs.rs_group_l2norm_clip(plan.h, rs.RS_ALL, rs.RS_ALL, buf, rs.RS_BF16, 0.5, sumsq, clip)
    d_theta = torch.from_numpy(theta.copy()).cuda()
    qm, qv = torch.zeros(L.total, dtype=torch.int8, device="cuda"), torch.zeros(L.total, dtype=torch.uint8, device="cuda")
    am, av = torch.zeros(L.n_blocks, device="cuda"), torch.zeros(L.n_blocks, device="cuda")
    rs.rs_adam8_step(plan.h, rs.RS_ALL, rs.RS_ALL, d_theta, buf, qm, qv, am, av, step=1, grad_scale=clip)
    g16 = buf.cpu().numpy().view(np.uint16)
    hm, hv = np.zeros(L.total, dtype=np.int8), np.zeros(L.total, dtype=np.uint8)
    ha, hb = np.zeros(L.n_blocks, dtype=np.float32), np.zeros(L.n_blocks, dtype=np.float32)
    L.adam8_step(-1, -1, theta, g16, hm, hv, ha, hb, oracle.HParams(step=1), gscale=oracle.clip_coef(L.group_sumsq(-1, -1, g16), 0.5))
    got = d_theta.cpu().numpy()
    assert np.all(np.abs(got - theta) <= 1e-8 + 1e-6 * np.abs(theta))
    assert np.array_equal(qm.cpu().numpy(), hm) and np.array_equal(qv.cpu().numpy(), hv)
    plan.free()


def test_example_runs_the_objectives():
    log("example objectives")
    r = example.main(steps=2)
    for name in ("preference", "policy", "router"):
        assert torch.isfinite(r[name]).all() and r[name][0].item() != 0, name
    assert r["counts"].sum().item() == example.TOKENS * example.TOPK
    # on-policy ratios are 1: nothing is clipped, the KL part is above 0
    assert r["policy"][3].item() == 0 and r["policy"][2].item() > 0
    r["plan"].free()
