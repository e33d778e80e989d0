"""Cases of the training objectives: the operators that turn a model's logits
into losses and into the gradients that a training step accumulates.

  token_logp   log-probability of one token per row of logits (what the
               behaviour and the reference policy of the losses below need)
  policy       clipped policy loss with a KL term, and its logits' gradient
  preference   paired log-ratio loss over ragged sequences, and its gradient
  balance      per-expert counts and load-balance loss of a router, and its
               gradient

Vocabularies and expert counts come from the model inventories in synth
(128256, 129280, 201088 tokens; 32, 128 and 256 experts, 4 or 8 of them per
token) or are generic.  Logits are a bell curve of width 2.5 with the row's
own token lifted to a probability between a few percent and nearly one, as a
trained model's are.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
LARGEST = 8192 * 128256  # logits of the largest listed case


def listed():
    return [
        # scoring one micro-batch of generated tokens: latency counts
        dict(name="logp_batch16", op="token_logp", rows=16, vocab=128256, pad=0, type="bf16", prompt=0, temperature=1.0),
        # the reference policy's pass over a packed batch of rollouts, odd vocabulary: rows start at any element
        dict(name="logp_odd_vocab", op="token_logp", rows=6001, vocab=32003, pad=0, type="bf16", prompt=300, temperature=0.7),
        # a tiny policy head (tests, debugging runs)
        dict(name="policy_small", op="policy", rows=48, vocab=1031, pad=0, type="f32", prompt=0, kl=0.04, clip_high=0.2, temperature=1.0),
        # one short rollout, large vocabulary: fewer rows than the card has units
        dict(name="policy_one_rollout", op="policy", rows=61, vocab=201088, pad=0, type="bf16", prompt=0, kl=0.0, clip_high=0.28, temperature=1.0),
        # binary32 logits of a padded vocabulary
        dict(name="policy_f32", op="policy", rows=1500, vocab=129280, pad=64, type="f32", prompt=100, kl=0.04, clip_high=0.2, temperature=0.9),
        # a packed micro-batch of rollouts, a quarter of the rows prompt
        dict(name="policy_packed", op="policy", rows=8192, vocab=128256, pad=0, type="bf16", prompt=256, kl=0.04, clip_high=0.28, temperature=1.0),
        # four short pairs, odd vocabulary
        dict(name="preference_short", op="preference", pairs=4, length=45, tail=3, vocab=32003, pad=0, type="bf16", prompt=0.4, kind="sigmoid", smoothing=0.0, average=False),
        # reference-scaled pairs in binary32
        dict(name="preference_f32", op="preference", pairs=6, length=250, tail=0, vocab=50000, pad=0, type="f32", prompt=0.3, kind="ipo", smoothing=0.0, average=True),
        # a packed batch of long pairs, rows of padding behind the last sequence
        dict(name="preference_packed", op="preference", pairs=8, length=600, tail=117, vocab=128256, pad=0, type="bf16", prompt=0.35, kind="sigmoid", smoothing=0.1, average=False),
        # a small batch through a 32-expert router: latency counts
        dict(name="balance_small", op="balance", rows=96, experts=32, k=4, type="f32", sequences=1, masked=0, score="softmax", z=1e-3),
        # one layer's tokens, 128 experts, four per token, one batch-wide loss
        dict(name="balance_batch", op="balance", rows=16383, experts=128, k=4, type="f32", sequences=1, masked=50, score="softmax", z=1e-3),
        # 256 experts, eight per token, sigmoid scores, a loss per sequence
        dict(name="balance_sequences", op="balance", rows=262144, experts=256, k=8, type="bf16", sequences=61, masked=0, score="sigmoid", z=0.0),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], evenly over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["token_logp", "policy", "policy", "preference", "preference", "balance", "balance"])
    kind = rng.choice(["bf16", "bf16", "f32"])
    if op == "balance":
        experts = rng.choice([8, 32, 60, 64, 128, 160, 256, 384])
        return dict(op=op, rows=_spread(rng, 1, 131072), experts=experts, k=rng.choice([1, 2, 4, 6, 8]), type=kind,
                    sequences=_spread(rng, 1, 64), masked=rng.choice([0, 0, 30, 200]), score=rng.choice(["softmax", "sigmoid"]), z=0.0)
    vocab = _spread(rng, 1000, 202000)
    pad = rng.choice([0, 0, 1, 64])
    most = LARGEST // 2 // (vocab + pad) // (2 if kind == "f32" else 1)
    if op == "preference":
        pairs = _spread(rng, 1, 24)
        length = _spread(rng, 2, max(3, min(1500, most // (2 * pairs) - 8)))
        return dict(op=op, pairs=pairs, length=length, tail=rng.choice([0, 5]), vocab=vocab, pad=pad, type=kind,
                    prompt=rng.choice([0.0, 0.3, 0.6]), kind=rng.choice(["sigmoid", "ipo"]), smoothing=0.0, average=rng.choice([False, True]))
    case = dict(op=op, rows=_spread(rng, 1, max(2, min(6000, most))), vocab=vocab, pad=pad, type=kind, prompt=rng.choice([0, 100, 500]),
                temperature=rng.choice([1.0, 1.0, 0.8]))
    if op == "policy":
        case.update(kl=rng.choice([0.0, 0.04]), clip_high=rng.choice([0.2, 0.28]))
    return case


# ------------------------------------------------------- shapes of a case

def _lengths(case):
    """Ragged lengths of the 2 * pairs sequences: 0.4 to 1 of the longest."""
    return [max(1, int(case["length"] * (0.4 + 0.6 * ((i * 0.618034 + 0.3) % 1.0)))) for i in range(2 * case["pairs"])]


def _starts(case):
    """Sequence starts of a router's packed batch: ragged, the last one longest."""
    n, rows = case["sequences"], case["rows"]
    return [int(rows * (i / n) ** 1.2) for i in range(n)] + [rows]


def _rows(case):
    return sum(_lengths(case)) + case["tail"] if case["op"] == "preference" else case["rows"]


def _scored(case):
    """Rows that have a token to score, as a list of truth values."""
    if case["op"] == "preference":
        got = []
        for n in _lengths(case):
            skip = min(n - 1, int(n * case["prompt"]))
            got += [False] * skip + [True] * (n - skip)
        return got + [False] * case["tail"]
    return [(t % 1024) >= case["prompt"] or case["rows"] < 600 for t in range(case["rows"])]


def work(case):
    size = 4 if case["type"] == "f32" else 2
    if case["op"] == "balance":
        n = case["rows"] * case["experts"]
        return {"bytes": 2 * n * size + case["rows"] * (8 * case["k"] + 1), "flops": 8 * n}
    rows, scored = _rows(case), sum(_scored(case))
    if case["op"] == "token_logp":
        return {"bytes": scored * case["vocab"] * size + 12 * rows, "flops": 3 * scored * case["vocab"]}
    written = rows - case.get("tail", 0)
    return {"bytes": (scored + written) * case["vocab"] * size + 24 * rows, "flops": 6 * scored * case["vocab"]}


# ---------------------------------------------------------------- inputs

def _softmax_parts(logits, target, scale):
    """exp((z - max) scale), its sum and the target's log-probability."""
    z = logits.float()
    top = z.amax(-1, keepdim=True)
    at = (z.gather(1, target[:, None]) - top).double()[:, 0] * scale
    e = torch.exp((z - top) * scale)
    total = e.sum(-1, dtype=torch.float64)  # long sums in 64 bits
    return e, total, at - torch.log(total)


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(int(seed) * 7919 + 17)
    kind = TYPES[case["type"]]
    rand = lambda *n: torch.rand(*n, device=dev, generator=g)  # noqa: E731
    randn = lambda *n: torch.randn(*n, device=dev, generator=g)  # noqa: E731
    s = {"case": case}
    if case["op"] == "balance":
        rows, experts, k = case["rows"], case["experts"], case["k"]
        s["logits"] = (randn(rows, experts) * 1.5 + randn(experts) * 0.5).to(kind)
        s["topk"] = torch.topk(s["logits"].float(), k, dim=-1).indices
        s["mask"] = ((torch.arange(rows, device=dev) * 7919 + 500) % 1000 >= case["masked"]).to(torch.uint8) if case["masked"] else None
        s["starts"] = torch.tensor(_starts(case), dtype=torch.int64, device=dev)
        s["dlogits"] = torch.zeros_like(s["logits"])
        s["counts"] = torch.zeros(case["sequences"], experts, dtype=torch.int32, device=dev)
        s["mean_prob"] = torch.zeros(case["sequences"], experts, device=dev)
        s["stats"] = torch.zeros(2, device=dev)
        s["work"] = _workspace(rows)
        return s
    rows, vocab = _rows(case), case["vocab"]
    # rows of vocab logits, `pad` unused columns behind each
    s["store"] = torch.randn(rows, vocab + case["pad"], device=dev, generator=g, dtype=kind).mul_(2.5)
    s["logits"] = s["store"][:, :vocab]
    scored = torch.tensor(_scored(case), device=dev)
    target = torch.randint(0, vocab, (rows,), device=dev, generator=g)
    lift = math.log(vocab) + 3.1 - 3.0 + 7.0 * rand(rows)
    s["logits"].scatter_(1, target[:, None], lift[:, None].to(kind))
    s["target"] = torch.where(scored, target, torch.full_like(target, -1))
    s["logp"] = torch.zeros(rows, device=dev)
    if case["op"] != "token_logp":
        s["dlogits"] = torch.zeros(rows, vocab, device=dev, dtype=kind)
        s["stats"] = torch.zeros(4 if case["op"] == "policy" else 3, device=dev)
        logp = _softmax_parts(s["logits"], target, 1.0 / case.get("temperature", 1.0))[2]
    if case["op"] == "policy":
        step = 0.12 * randn(rows).double()  # log ratio to the behaviour policy
        # no ratio within 1e-4 of a clipping border, where rounding decides
        for border in (math.log(0.8), math.log(1.0 + case["clip_high"])):
            step = torch.where((step - border).abs() < 1e-4, step + 3e-4, step)
        s["old_logp"] = (logp - step).float()
        s["ref_logp"] = (logp + 0.2 * randn(rows).double()).float()
        s["advantage"] = randn(rows)
        s["weight"] = scored.float() / max(1, sum(_scored(case)))
    if case["op"] == "preference":
        pairs = case["pairs"]
        ends = torch.tensor([0] + _lengths(case), device=dev).cumsum(0)
        s["starts"] = ends.to(torch.int64)
        total = torch.cat([torch.zeros(1, device=dev, dtype=torch.float64), torch.where(scored, logp, torch.zeros_like(logp)).cumsum(0)])
        seq = total[ends[1:]] - total[ends[:-1]]
        if case["average"]:
            hits = torch.cat([torch.zeros(1, device=dev, dtype=torch.float64), scored.double().cumsum(0)])
            seq = seq / (hits[ends[1:]] - hits[ends[:-1]])
        s["ref_logp"] = (seq + (0.5 if case["average"] else 6.0) * randn(2 * pairs).double()).float()
        s["weight"] = torch.full((pairs,), 1.0 / pairs, device=dev)
        s["seq_logp"] = torch.zeros(2 * pairs, device=dev)
    s["work"] = _workspace(rows)
    return s


def _workspace(rows):
    """Scratch memory that a training program keeps for the losses."""
    return torch.empty((32 << 20) + 256 * rows, dtype=torch.uint8, device="cuda")


# ------------------------------------------------------------ plain forms

def _row_sequences(starts, rows, device):
    return (torch.arange(rows, device=device)[:, None] >= starts[None, 1:]).sum(1)


def _plain_token_logp(s, case):
    valid = s["target"] >= 0
    logp = _softmax_parts(s["logits"], s["target"].clamp(min=0), 1.0 / case["temperature"])[2]
    return {"logp": torch.where(valid, logp, torch.zeros_like(logp)).float()}


def _logits_gradient(e, total, target, valid, coef, scale, kind):
    """coef (onehot - softmax) scale, zero for rows without a token."""
    c = torch.where(valid, coef * scale, torch.zeros_like(coef)).float()
    d = e * (-c / total.float())[:, None]
    d.scatter_add_(1, target[:, None], c[:, None])
    return torch.where(valid[:, None], d, torch.zeros_like(d)).to(kind)


def _plain_policy(s, case):
    valid = (s["target"] >= 0) & (s["weight"] != 0)
    target = s["target"].clamp(min=0)
    scale = 1.0 / case["temperature"]
    e, total, logp = _softmax_parts(s["logits"], target, scale)
    w, a = s["weight"].double(), s["advantage"].double()
    ratio = torch.exp(logp - s["old_logp"].double())
    free, held = -a * ratio, -a * ratio.clamp(0.8, 1.0 + case["clip_high"])
    clipped = free < held
    away = s["ref_logp"].double() - logp
    kl = torch.exp(away) - away - 1.0
    coef = w * (torch.where(clipped, torch.zeros_like(a), free) + case["kl"] * (1.0 - torch.exp(away)))
    zero = torch.zeros_like(w)
    parts = [torch.where(valid, w * x, zero).sum() for x in (torch.maximum(free, held), kl, clipped.double())]
    stats = torch.stack([parts[0] + case["kl"] * parts[1], *parts]).float()
    return {"dlogits": _logits_gradient(e, total, target, valid, coef, scale, s["logits"].dtype),
            "logp": torch.where(valid, logp, zero).float(), "stats": stats}


def _plain_preference(s, case):
    rows, pairs = s["logits"].shape[0], case["pairs"]
    valid = s["target"] >= 0
    target = s["target"].clamp(min=0)
    e, total, logp = _softmax_parts(s["logits"], target, 1.0)
    seq_of = _row_sequences(s["starts"], rows, logp.device)
    valid = valid & (seq_of < 2 * pairs)
    seq_of = seq_of.clamp(max=2 * pairs - 1)
    own_row = (seq_of[None, :] == torch.arange(2 * pairs, device=logp.device)[:, None]) & valid[None, :]
    share = own_row.double()
    if case["average"]:
        share = share / share.sum(1, keepdim=True).clamp(min=1.0)
    seq = (share * torch.where(valid, logp, torch.zeros_like(logp))[None, :]).sum(1)
    ref, w, beta = s["ref_logp"].double(), s["weight"].double(), 0.1
    delta = (seq - ref)[:pairs] - (seq - ref)[pairs:]
    if case["kind"] == "ipo":
        loss, slope, h = (delta - 0.5 / beta) ** 2, 2.0 * (delta - 0.5 / beta), beta * delta
    else:
        h, ls = beta * delta, case["smoothing"]
        loss = (1.0 - ls) * torch.log1p(torch.exp(-h)) + ls * torch.log1p(torch.exp(h))
        slope = beta * (ls - 1.0 / (1.0 + torch.exp(h)))
    per_seq = torch.cat([w * slope, -w * slope])
    coef = (share * per_seq[:, None]).sum(0)
    stats = torch.stack([(w * loss).sum(), (w * h).sum(), (w * (h > 0)).sum()]).float()
    return {"dlogits": _logits_gradient(e, total, target, valid, coef, 1.0, s["logits"].dtype),
            "seq_logp": seq.float(), "stats": stats}


def _sequence_sums(member, x):
    """member [sequences, rows] times x [rows, columns], in blocks of rows
    (one product over all rows is many times slower)."""
    more = -x.shape[0] % 512
    m = torch.nn.functional.pad(member, (0, more)).view(member.shape[0], -1, 512).transpose(0, 1).contiguous()
    return torch.bmm(m, torch.nn.functional.pad(x, (0, 0, 0, more)).view(-1, 512, x.shape[1])).sum(0)


def _plain_balance(s, case):
    z = s["logits"].float()
    rows, experts = z.shape
    n = case["sequences"]
    seq_of = _row_sequences(s["starts"], rows, z.device)
    live = s["mask"] != 0 if s["mask"] is not None else torch.ones(rows, device=z.device, dtype=torch.bool)
    chosen = torch.zeros_like(z).scatter_add_(1, s["topk"], live.float()[:, None].expand(-1, case["k"]))
    member = ((seq_of[None, :] == torch.arange(n, device=z.device)[:, None]) & live[None, :]).double()
    tokens = member.sum(1).clamp(min=1.0)
    if case["score"] == "softmax":
        e = torch.exp(z - z.amax(-1, keepdim=True))
        p = e / e.sum(-1, keepdim=True)
        slope = p
        lse = (z.amax(-1) + torch.log(e.sum(-1))).double()
    else:
        sig = 1.0 / (1.0 + torch.exp(-z))
        p = sig / sig.sum(-1, keepdim=True)
        slope = p * (1.0 / (1.0 + torch.exp(z)))
        lse = torch.zeros(rows, device=z.device, dtype=torch.float64)
    mean = _sequence_sums(member, p.double()) / tokens[:, None]
    counts = _sequence_sums(member, chosen.double())
    f = counts * experts / (case["k"] * tokens[:, None])
    balance = 0.01 * (f * mean).sum()
    z_loss = case["z"] * ((member * lse.square()).sum(1) / tokens).sum()
    f_row = f.float()[seq_of]
    per = (1.0 / tokens).float()[seq_of][:, None]
    d = per * (0.01 * slope * (f_row - (f_row * p).sum(-1, keepdim=True)) + (2.0 * case["z"]) * lse.float()[:, None] * p)
    d = torch.where(live[:, None], d, torch.zeros_like(d))
    return {"dlogits": d.to(s["logits"].dtype), "counts": counts.to(torch.int32), "mean_prob": mean.float(),
            "stats": torch.stack([balance, z_loss]).float()}


# ------------------------------------------------------------- one pass

def _run_own(s, case):
    import sharded_state_raggedshard_amd as rs
    kind = rs.RS_F32 if case["type"] == "f32" else rs.RS_BF16
    if case["op"] == "balance":
        rs.rs_router_balance(s["logits"], kind, case["rows"], case["experts"], case["experts"], s["topk"], case["k"], case["k"],
                             s["mask"], s["starts"], case["sequences"], s["dlogits"], case["experts"], s["counts"], s["mean_prob"], s["stats"],
                             s["work"], s["work"].numel(), balance_coef=0.01, z_coef=case["z"],
                             score=rs.RS_SCORE_SIGMOID if case["score"] == "sigmoid" else rs.RS_SCORE_SOFTMAX)
        return {"dlogits": s["dlogits"], "counts": s["counts"], "mean_prob": s["mean_prob"], "stats": s["stats"]}
    rows, vocab = s["logits"].shape
    ld = s["logits"].stride(0)
    if case["op"] == "token_logp":
        rs.rs_token_logp(s["logits"], kind, rows, vocab, ld, s["target"], s["logp"], s["work"], s["work"].numel(), temperature=case["temperature"])
        return {"logp": s["logp"]}
    if case["op"] == "policy":
        rs.rs_policy_loss(s["logits"], kind, rows, vocab, ld, s["target"], s["old_logp"], s["ref_logp"], s["advantage"], s["weight"],
                          s["dlogits"], vocab, s["logp"], s["stats"], s["work"], s["work"].numel(), temperature=case["temperature"],
                          clip_low=0.2, clip_high=case["clip_high"], kl_coef=case["kl"])
        return {"dlogits": s["dlogits"], "logp": s["logp"], "stats": s["stats"]}
    rs.rs_preference_loss(s["logits"], kind, rows, vocab, ld, s["target"], s["starts"], case["pairs"], s["ref_logp"], s["weight"],
                          s["dlogits"], vocab, s["seq_logp"], s["stats"], s["work"], s["work"].numel(), beta=0.1, label_smoothing=case["smoothing"],
                          kind=rs.RS_PREF_IPO if case["kind"] == "ipo" else rs.RS_PREF_SIGMOID, average=case["average"])
    return {"dlogits": s["dlogits"], "seq_logp": s["seq_logp"], "stats": s["stats"]}


def run(state):
    case = state["case"]
    if own:
        return _run_own(state, case)
    plain = {"token_logp": _plain_token_logp, "policy": _plain_policy, "preference": _plain_preference, "balance": _plain_balance}
    return plain[case["op"]](state, case)


# ---------------------------------------------------- 64-bit definitions

def _exact_logp(s, scale):
    """Log-probabilities of the targets (0 without one), some rows at a time."""
    rows, vocab = s["logits"].shape
    out = torch.zeros(rows, dtype=torch.float64, device="cuda")
    some = max(1, (1 << 27) // vocab)
    for a in range(0, rows, some):
        t = s["target"][a:a + some]
        ls = torch.log_softmax(s["logits"][a:a + some].double() * scale, dim=-1)
        out[a:a + some] = ls.gather(1, t.clamp(min=0)[:, None])[:, 0] * (t >= 0)
    return out


def _exact_dlogits(s, coef, scale):
    """Chain rule through log_softmax from dloss/dlogp, some rows at a time."""
    rows, vocab = s["logits"].shape
    out = torch.zeros(rows, vocab, dtype=torch.float64, device="cuda")
    some = max(1, (1 << 27) // vocab)
    for a in range(0, rows, some):
        t = s["target"][a:a + some]
        c = (coef[a:a + some] * (t >= 0))[:, None]
        d = torch.softmax(s["logits"][a:a + some].double() * scale, dim=-1) * (-c)
        d.scatter_add_(1, t.clamp(min=0)[:, None], c)
        out[a:a + some] = d * scale
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "balance":
        return _exact_balance(s, case)
    scale = 1.0 / case.get("temperature", 1.0)
    logp = _exact_logp(s, scale)
    if case["op"] == "token_logp":
        return {"logp": logp}
    leaf = logp.clone().requires_grad_(True)
    ref, w = s["ref_logp"].double(), s["weight"].double()
    if case["op"] == "policy":
        token = (s["target"] >= 0).double()
        ratio = torch.exp(leaf - s["old_logp"].double())
        gain = s["advantage"].double() * ratio
        bounded = s["advantage"].double() * torch.clamp(ratio, 0.8, 1.0 + case["clip_high"])
        surrogate = -torch.minimum(gain, bounded)
        kl = torch.expm1(ref - leaf) - (ref - leaf)
        w = w * token
        loss = (w * surrogate).sum() + case["kl"] * (w * kl).sum()
        stats = torch.stack([loss, (w * surrogate).sum(), (w * kl).sum(), (w * (gain > bounded)).sum()])
        extra = {"logp": logp}
    else:
        pairs, beta = case["pairs"], 0.1
        per = []
        for i in range(2 * pairs):
            a, b = int(s["starts"][i]), int(s["starts"][i + 1])
            n = (s["target"][a:b] >= 0).sum().clamp(min=1) if case["average"] else 1
            per.append(leaf[a:b].sum() / n)
        seq = torch.stack(per)
        delta = (seq[:pairs] - ref[:pairs]) - (seq[pairs:] - ref[pairs:])
        if case["kind"] == "ipo":
            each = torch.square(delta - 1.0 / (2.0 * beta))
        else:
            ls = torch.nn.functional.logsigmoid
            each = -(1.0 - case["smoothing"]) * ls(beta * delta) - case["smoothing"] * ls(-beta * delta)
        loss = (w * each).sum()
        stats = torch.stack([loss, (w * beta * delta).sum(), (w * (delta > 0)).sum()])
        extra = {"seq_logp": seq.detach()}
    (coef,) = torch.autograd.grad(loss, leaf)
    return {"dlogits": _exact_dlogits(s, coef, scale), "stats": stats.detach(), **extra}


def _exact_balance(s, case):
    z = s["logits"].double().requires_grad_(True)
    rows, experts, k = case["rows"], case["experts"], case["k"]
    if case["score"] == "softmax":
        p = torch.softmax(z, dim=-1)
    else:
        sig = torch.sigmoid(z)
        p = sig / sig.sum(-1, keepdim=True)
    live = torch.ones(rows, device="cuda", dtype=torch.bool) if s["mask"] is None else s["mask"].bool()
    starts = _starts(case)
    balance, z_loss = z.new_zeros(()), z.new_zeros(())
    counts, means = [], []
    for a, b in zip(starts[:-1], starts[1:]):
        keep = live[a:b]
        n = max(1, int(keep.sum()))
        c = torch.bincount(s["topk"][a:b][keep].reshape(-1), minlength=experts)
        mean = p[a:b][keep].sum(0) / n
        balance = balance + 0.01 * (c.double() * (experts / (k * n)) * mean).sum()
        if case["z"]:
            z_loss = z_loss + case["z"] * torch.logsumexp(z[a:b][keep], dim=-1).square().sum() / n
        counts.append(c)
        means.append(mean.detach())
    (d,) = torch.autograd.grad(balance + z_loss, z)
    return {"dlogits": d, "counts": torch.stack(counts).to(torch.int32), "mean_prob": torch.stack(means),
            "stats": torch.stack([balance, z_loss]).detach()}
