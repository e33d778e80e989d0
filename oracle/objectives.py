"""Plain CPU oracle of the training objectives -- TEST INFRASTRUCTURE ONLY.

Only tests/ uses this module; the library never imports it.  Row by row in
numpy binary64, straight from the formulas: token log-probability, clipped
policy loss with a KL term, preference loss over packed pairs, router
balance loss with per-expert counts, each with the gradient by the chain
rule.  tests/test_oracle_objectives.py holds the losses against torch's own
functions and the gradients against differences of the losses.
"""
from __future__ import annotations

from typing import Optional

import numpy as np

SIGMOID, HINGE, IPO = 0, 1, 2
SOFTMAX, NORMALISED_SIGMOID = 0, 1


def softmax_row(z: np.ndarray, scale: float):
    """(p, log sum exp) of one row of binary64 logits; (zeros, None) for a
    row of nothing but -inf."""
    m = z.max()
    if m == -np.inf:
        return np.zeros_like(z), None
    with np.errstate(invalid="ignore"):
        e = np.exp((z - m) * scale)
    s = e.sum()
    return e / s, m * scale + np.log(s)


def token_logp(z: np.ndarray, target: np.ndarray, temperature: float = 1.0, part=None):
    """(logp, lse, live rows, p): rows without a token (target outside the
    row, part[t] False, nothing but -inf) have logp 0, lse 0."""
    rows, vocab = z.shape
    logp, lse = np.zeros(rows), np.zeros(rows)
    live, p = np.zeros(rows, dtype=bool), np.zeros((rows, vocab))
    for t in range(rows):
        y = int(target[t])
        if not 0 <= y < vocab or (part is not None and not part[t]):
            continue
        q, l = softmax_row(z[t].astype(np.float64), 1.0 / temperature)
        if l is None:
            continue
        live[t], p[t], lse[t] = True, q, l
        # against the maximum: values of the type's lowest cancel exactly
        m = float(z[t].max())
        logp[t] = (float(z[t, y]) - m) / temperature - (l - m / temperature if abs(m) < 1e30 else
                                                        np.log((z[t] == m).sum()))
    return logp, lse, live, p


def _dlogits(p, target, live, coef, temperature):
    d = np.zeros_like(p)
    for t in np.nonzero(live)[0]:
        d[t] = -coef[t] * p[t]
        d[t, int(target[t])] += coef[t]
    return d / temperature


def policy_loss(z, target, old, ref, adv, weight, temperature=1.0, clip_low=0.2, clip_high=0.2,
                kl_coef=0.0):
    logp, lse, live, p = token_logp(z, target, temperature, weight != 0)
    coef = np.zeros(len(logp))
    pg = kl = clipped = 0.0
    for t in np.nonzero(live)[0]:
        r = np.exp(logp[t] - float(old[t]))
        a, w = float(adv[t]), float(weight[t])
        free, held = -a * r, -a * min(max(r, 1.0 - clip_low), 1.0 + clip_high)
        pg += w * max(free, held)
        slope = free if free >= held else 0.0
        if free < held:
            clipped += w
        if ref is not None:
            away = float(ref[t]) - logp[t]
            kl += w * (np.expm1(away) - away)
            slope -= kl_coef * np.expm1(away)
        coef[t] = w * slope
    return {"logp": logp, "live": live, "p": p, "coef": coef,
            "stats": np.array([pg + kl_coef * kl, pg, kl, clipped]),
            "dlogits": _dlogits(p, target, live, coef, temperature)}


def preference_loss(z, target, start, pairs, ref: Optional[np.ndarray], weight, temperature=1.0,
                    beta=0.1, label_smoothing=0.0, margin=0.0, kind=SIGMOID, average=False):
    """Rows outside every sequence have inside False; their gradient is
    whatever the caller's array held."""
    rows = z.shape[0]
    w = np.full(pairs, 1.0 / pairs) if weight is None else weight.astype(np.float64)
    seq_of = np.full(rows, -1)
    for s in range(2 * pairs):
        seq_of[int(start[s]):int(start[s + 1])] = s
    part = np.array([s >= 0 and w[s % pairs] != 0 for s in seq_of], dtype=bool)
    logp, lse, live, p = token_logp(z, target, temperature, part)
    total = np.zeros(2 * pairs)
    count = np.zeros(2 * pairs)
    for t in np.nonzero(live)[0]:
        total[seq_of[t]] += logp[t]
        count[seq_of[t]] += 1
    if average:
        total = total / np.maximum(count, 1)
    stats, per_seq = np.zeros(3), np.zeros(2 * pairs)
    for i in range(pairs):
        if w[i] == 0:
            continue
        d = total[i] - total[i + pairs]
        if ref is not None:
            d -= float(ref[i]) - float(ref[i + pairs])
        h = beta * d - margin
        if kind == IPO:
            loss, g = (d - 0.5 / beta) ** 2, 2.0 * (d - 0.5 / beta)
        elif kind == HINGE:
            loss, g = max(0.0, 1.0 - h), -beta if h < 1.0 else 0.0
        else:
            loss = ((1.0 - label_smoothing) * np.logaddexp(0.0, -h)
                    + label_smoothing * np.logaddexp(0.0, h))
            g = beta * (label_smoothing - np.exp(-np.logaddexp(0.0, h)))
        stats += w[i] * np.array([loss, h, float(h > 0)])
        per_seq[i], per_seq[i + pairs] = w[i] * g, -w[i] * g
    coef = np.zeros(rows)
    for t in np.nonzero(live)[0]:
        coef[t] = per_seq[seq_of[t]] / (max(count[seq_of[t]], 1) if average else 1)
    return {"seq_logp": total, "logp": logp, "live": live, "p": p, "coef": coef, "stats": stats,
            "inside": seq_of >= 0, "per_seq": per_seq,
            "dlogits": _dlogits(p, target, live, coef, temperature)}


def router_balance(z, topk, mask, start, balance_coef=1e-2, z_coef=0.0, score=SOFTMAX):
    rows, experts = z.shape
    k = topk.shape[1]
    n_seq = len(start) - 1
    counts = np.zeros((n_seq, experts), dtype=np.int64)
    mean = np.zeros((n_seq, experts))
    d = np.zeros((rows, experts))
    inside = np.zeros(rows, dtype=bool)
    balance = z_loss = 0.0
    for s in range(n_seq):
        a, b = int(start[s]), int(start[s + 1])
        inside[a:b] = True
        tokens = [t for t in range(a, b) if mask is None or mask[t]]
        n = max(len(tokens), 1)
        for t in tokens:
            for e in topk[t]:
                if 0 <= e < experts:
                    counts[s, int(e)] += 1
        f = counts[s] * (experts / (k * n))
        for t in tokens:
            x = z[t].astype(np.float64)
            p, lse = softmax_row(x, 1.0)
            if lse is None:
                continue
            slope = p
            if score == NORMALISED_SIGMOID:
                # log s(x), against its largest: far negative rows keep their shares
                ls = -np.logaddexp(0.0, -x)
                p = np.exp(ls - ls.max())
                p = p / p.sum()
                slope = p * np.exp(-np.logaddexp(0.0, x))
            mean[s] += p / n
            balance += balance_coef * (f @ p) / n
            d[t] = balance_coef / n * slope * (f - f @ p)
            if z_coef:
                z_loss += z_coef * lse * lse / n
                d[t] += 2.0 * z_coef / n * lse * p
    return {"counts": counts, "mean_prob": mean, "dlogits": d, "inside": inside,
            "stats": np.array([balance, z_loss])}
