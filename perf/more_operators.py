"""Cases of the operators around a mixture-of-experts training step: what a
step does between the router and the experts, between the logits and a loss of
the caller's own, and with the parameters that no planned buffer holds.

  experts  tokens sorted by expert, carried to the experts and back with their
           weights (way "forward"); the gradients of both (way "backward")
  stats    log-probability of a token per row of logits with the row's entropy
           and its most probable alternatives (way "score"); the same with the
           logits' gradient from both upstream gradients (way "train")
  adamw    an AdamW step over many tensors in place, moments in 32 bits, or in
           8 bits with one scale per block and read out as the values they
           stand for (bf16); with "clip" the gradients' norm and coefficient
           first

Hidden sizes, expert counts, vocabularies and layers come from the model and
workload inventories in synth (2048, 2880, 4096, 7168 wide; 32, 128 and 256
experts, 4 or 8 a token; 128256, 129280 and 201088 tokens) or are generic.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
LARGEST_LOGITS = 4096 * 128256
LARGEST_MOVED = 8192 * 8 * 7168
LARGEST_STATE = 400_000_000


def listed():
    return [
        # one decoding step of a batch of 16: latency counts
        dict(name="experts_decode", op="experts", way="forward", rows=16, hidden=2880, experts=32, k=4, align=1, masked=0, type="bf16"),
        # a packed micro-batch with padding rows, odd hidden size, binary32
        dict(name="experts_odd", op="experts", way="backward", rows=3001, hidden=1003, experts=60, k=6, align=1, masked=40, type="f32"),
        # one layer's tokens, segments padded to the row tiles of the experts' products
        dict(name="experts_batch", op="experts", way="forward", rows=8192, hidden=7168, experts=256, k=8, align=128, masked=0, type="bf16"),
        # the backward pass of one layer's tokens
        dict(name="experts_gradient", op="experts", way="backward", rows=16384, hidden=2880, experts=128, k=4, align=1, masked=0, type="bf16"),
        # tokens just sampled, with the alternatives that a sampler reports: latency counts
        dict(name="stats_sampled", op="stats", way="score", rows=16, vocab=128256, top=20, prompt=0, banned=0, temperature=1.0, type="bf16"),
        # scoring given texts, odd vocabulary, a quarter of it ruled out, prompts left out
        dict(name="stats_odd_vocab", op="stats", way="score", rows=6001, vocab=32003, top=5, prompt=300, banned=250, temperature=0.7, type="f32"),
        # one short rollout, large vocabulary: fewer rows than the card has units
        dict(name="stats_one_rollout", op="stats", way="train", rows=61, vocab=201088, top=0, prompt=0, banned=0, temperature=1.0, type="bf16"),
        # a packed micro-batch of rollouts
        dict(name="stats_packed", op="stats", way="train", rows=4096, vocab=128256, top=8, prompt=128, banned=0, temperature=1.0, type="bf16"),
        # the norms and biases of a small model: latency counts
        dict(name="adamw_vectors", op="adamw", kind="vectors", count=65, width=2048, param="f32", grad="f32", state=32, out=False, clip=False),
        # adapters and other small odd tensors, 8-bit moments, clipped
        dict(name="adamw_odd_8bit", op="adamw", kind="ragged", count=211, width=400_000, param="f32", grad="bf16", state=8, out=False, clip=True),
        # one layer, binary32 master and moments, bf16 weights written beside them, clipped
        dict(name="adamw_layer", op="adamw", kind="layers", layers=1, hidden=2048, ffn=5632, kv=2048, param="f32", grad="bf16", state=32, out=True, clip=True),
        # bf16 weights trained in place, binary32 moments
        dict(name="adamw_bf16_weights", op="adamw", kind="layers", layers=1, hidden=4096, ffn=14336, kv=1024, param="bf16", grad="bf16", state=32, out=False, clip=False),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], evenly over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["experts", "stats", "adamw"])
    kind = rng.choice(["bf16", "bf16", "f32"])
    if op == "experts":
        experts, k = rng.choice([8, 32, 60, 64, 128, 160, 256]), rng.choice([1, 2, 4, 6, 8])
        hidden = _spread(rng, 64, 8192)
        if rng.random() < 0.6:
            hidden = hidden // 8 * 8
        most = LARGEST_MOVED // (k * hidden) // (4 if kind == "f32" else 2)
        return dict(op=op, way=rng.choice(["forward", "backward"]), rows=_spread(rng, 1, min(32768, most)), hidden=hidden, experts=experts, k=k,
                    align=rng.choice([1, 1, 16, 128]), masked=rng.choice([0, 0, 30, 200]), type=kind)
    if op == "stats":
        vocab, way = _spread(rng, 1000, 202000), rng.choice(["score", "train"])
        most = LARGEST_LOGITS // vocab // (4 if kind == "f32" else 2)
        return dict(op=op, way=way, rows=_spread(rng, 1, max(2, min(6000, most))), vocab=vocab, top=rng.choice([0, 1, 5, 8, 20, 32]),
                    prompt=rng.choice([0, 100, 500]), banned=rng.choice([0, 0, 400]), temperature=rng.choice([1.0, 1.0, 0.8]), type=kind)
    shape = rng.choice(["vectors", "ragged", "ragged"])
    count = _spread(rng, 1, 300)
    width = _spread(rng, 1, min(4_000_000, LARGEST_STATE // 4 // count))
    param = rng.choice(["f32", "f32", "bf16"])
    return dict(op=op, kind=shape, count=count, width=width, param=param, grad=param if param == "bf16" else kind, state=rng.choice([32, 8]),
                out=param == "f32" and rng.random() < 0.5, clip=rng.choice([True, False]))


# ------------------------------------------------------- shapes of a case

BLOCK = 256  # elements that share a scale, 8-bit moments
BETA1, BETA2, EPS, LR, DECAY, STEP, MAX_NORM = 0.9, 0.95, 1e-8, 3e-4, 0.1, 10, 1.0


def _sizes(case):
    """(elements of the tensors with weight decay, of those without)."""
    if case["kind"] == "layers":
        h, f, kv = case["hidden"], case["ffn"], case["kv"]
        return [h * h, kv * h, kv * h, h * h, f * h, f * h, h * f] * case["layers"], [h, h] * case["layers"]
    if case["kind"] == "vectors":
        return [], [case["width"]] * case["count"]
    # ragged: every third tensor a short one without decay
    n = [max(1, int(case["width"] * ((i * 0.618034 + 0.21) % 1.0) ** 3)) for i in range(case["count"])]
    return [x for i, x in enumerate(n) if i % 3], [min(x, 2880) for i, x in enumerate(n) if i % 3 == 0]


def _starts(sizes, align):
    """First element of each tensor in one store, and its end."""
    at, got = 0, []
    for n in sizes:
        got.append(at)
        at += -(-n // align) * align
    return got, at


def _slots(case):
    """Rows that the sorted tokens can take at most."""
    choices = case["rows"] * case["k"]
    return choices + min(case["experts"], choices) * (case["align"] - 1)


def _scored(case):
    """Rows that have a token to score, as a list of truth values."""
    return [(t % 1024) >= case["prompt"] or case["rows"] < 600 for t in range(case["rows"])]


def work(case):
    if case["op"] == "experts":
        size = 4 if case["type"] == "f32" else 2
        rows, k, h = case["rows"], case["k"], case["hidden"]
        taken = sum((t * 7919 + 500) % 1000 >= case["masked"] for t in range(rows)) * k
        if case["way"] == "forward":  # tokens in, sorted tokens out, experts' rows in, tokens out
            return {"bytes": (2 * rows + 2 * taken) * h * size + rows * k * 16, "flops": 2 * taken * h}
        # gradient of the tokens out and the experts' rows in, theirs out; the sorted tokens' gradient in, the tokens' out
        return {"bytes": (2 * rows + 3 * taken) * h * size + rows * k * 12, "flops": 4 * taken * h}
    if case["op"] == "stats":
        size = 4 if case["type"] == "f32" else 2
        rows, vocab, scored = case["rows"], case["vocab"], sum(_scored(case))
        if case["way"] == "score":
            return {"bytes": scored * vocab * size + rows * (16 + 12 * case["top"]), "flops": 5 * scored * vocab}
        return {"bytes": (scored + rows) * vocab * size + rows * (24 + 12 * case["top"]), "flops": 10 * scored * vocab}
    big, small = _sizes(case)
    n = sum(big) + sum(small)
    param, grad = (4 if case["param"] == "f32" else 2), (4 if case["grad"] == "f32" else 2)
    each = 2 * param + grad + (16 if case["state"] == 32 else 4 + 4) + (2 if case["out"] else 0)
    return {"bytes": n * each + (0 if case["state"] == 32 else 16 * (n // BLOCK)), "flops": 14 * n}


# ---------------------------------------------------------------- inputs

def _draws(seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 29)
    rand = lambda *n, **kw: torch.rand(*n, device="cuda", generator=g, **kw)  # noqa: E731
    randn = lambda *n, **kw: torch.randn(*n, device="cuda", generator=g, **kw)  # noqa: E731
    return g, rand, randn


def prepare(case, seed):
    return {"experts": _prepare_experts, "stats": _prepare_stats, "adamw": _prepare_adamw}[case["op"]](case, seed)


def _prepare_experts(case, seed):
    g, rand, randn = _draws(seed)
    rows, hidden, experts, k, kind = case["rows"], case["hidden"], case["experts"], case["k"], TYPES[case["type"]]
    s = {"case": case, "slots": _slots(case)}
    logits = randn(rows, experts) + 0.7 * randn(experts)
    values, s["topk"] = torch.topk(logits, k, dim=-1)
    s["weight"] = torch.softmax(values, dim=-1)
    s["mask"] = ((torch.arange(rows, device="cuda") * 7919 + 500) % 1000 >= case["masked"]).to(torch.uint8) if case["masked"] else None
    s["x"] = randn(rows, hidden, dtype=kind)  # the tokens, or the gradient of what they come back as
    s["y"] = randn(s["slots"], hidden, dtype=kind)  # what the experts made of their rows
    s["sorted"] = torch.zeros(s["slots"], hidden, dtype=kind, device="cuda")
    s["out"] = torch.zeros(rows, hidden, dtype=kind, device="cuda")
    if case["way"] == "forward":
        s["start"] = torch.zeros(experts + 1, dtype=torch.int64, device="cuda")
        s["count"] = torch.zeros(experts, dtype=torch.int32, device="cuda")
        s["slot"] = torch.zeros(rows, k, dtype=torch.int32, device="cuda")
        if own:
            import sharded_state_raggedshard_amd as rs
            s["work"] = torch.empty(rs.rs_expert_sort_bytes(rows, experts, k), dtype=torch.uint8, device="cuda")
    else:
        s["start"], s["count"], s["slot"] = _plain_sort(s, case)
        s["dsorted"] = randn(s["slots"], hidden, dtype=kind)  # gradient of the sorted tokens
        s["dweight"] = torch.zeros(rows, k, device="cuda")
    return s


def _prepare_stats(case, seed):
    g, rand, randn = _draws(seed)
    rows, vocab, kind, top = case["rows"], case["vocab"], TYPES[case["type"]], case["top"]
    # a bell curve with the row's token lifted to a probability between a few percent and nearly one
    s = {"case": case, "logits": randn(rows, vocab, dtype=kind).mul_(2.5)}
    scored = torch.tensor(_scored(case), device="cuda")
    target = torch.randint(0, vocab, (rows,), device="cuda", generator=g)
    if case["banned"]:
        s["logits"].masked_fill_((torch.arange(vocab, device="cuda") * 7919 + 500) % 1000 < case["banned"], -math.inf)
    lift = math.log(vocab) + 3.1 - 3.0 + 7.0 * rand(rows)
    s["logits"].scatter_(1, target[:, None], lift[:, None].to(kind))
    s["target"] = torch.where(scored, target, torch.full_like(target, -1))
    s["logp"], s["entropy"] = torch.zeros(rows, device="cuda"), torch.zeros(rows, device="cuda")
    s["top_id"] = torch.zeros(rows, top, dtype=torch.int64, device="cuda")
    s["top_logp"] = torch.zeros(rows, top, device="cuda")
    if case["way"] == "train":
        s["dlogp"] = randn(rows) / rows
        s["dentropy"] = -0.01 * rand(rows) / rows
        s["dlogits"] = torch.zeros(rows, vocab, dtype=kind, device="cuda")
    if own:
        import sharded_state_raggedshard_amd as rs
        s["work"] = torch.empty(rs.rs_token_stats_bytes(rows, vocab, top), dtype=torch.uint8, device="cuda")
        s["saved"] = torch.zeros(rows, 4, device="cuda")
    return s


def _prepare_adamw(case, seed):
    g, rand, randn = _draws(seed)
    big, small = _sizes(case)
    sizes, eight = big + small, case["state"] == 8
    starts, end = _starts(sizes, BLOCK if eight else 1)
    cut = starts[len(big)] if small else end
    s = {"case": case, "cut": cut}
    # one store for all tensors, with gaps up to the next block where moments have 8 bits
    live = None
    if eight:
        at, n = torch.tensor(starts, device="cuda"), torch.tensor(sizes, device="cuda")
        s["where"] = torch.arange(sum(sizes), device="cuda") + torch.repeat_interleave(at - (n.cumsum(0) - n), n)
        live = torch.zeros(end, device="cuda")
        live[s["where"]] = 1.0
    keep = lambda x: x if live is None else x * live  # noqa: E731
    s["param"] = keep(0.04 * rand(end) - 0.02).to(TYPES[case["param"]])
    s["grad"] = keep(1e-3 * randn(end)).to(TYPES[case["grad"]])
    m, v = keep(3e-4 * randn(end)), keep(1e-6 * (0.05 + rand(end)))
    if eight:
        s["amax_m"], s["amax_v"] = m.view(-1, BLOCK).abs().amax(1), v.view(-1, BLOCK).amax(1)
        s["m"] = torch.round(m.view(-1, BLOCK) / s["amax_m"][:, None] * 127.0).to(torch.int8).view(-1)
        s["v"] = torch.round(v.view(-1, BLOCK) / s["amax_v"][:, None] * 255.0).to(torch.uint8).view(-1)
        s["m_values"], s["v_values"] = (torch.zeros(sum(sizes), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    else:
        s["m"], s["v"] = m, v
    s["out"] = torch.zeros(end, dtype=torch.bfloat16, device="cuda") if case["out"] else None
    s["sumsq"], s["scale"] = torch.zeros(1, dtype=torch.float64, device="cuda"), torch.ones(1, device="cuda")
    if own:
        import sharded_state_raggedshard_amd as rs
        kinds = {"f32": rs.RS_F32, "bf16": rs.RS_BF16}
        state = rs.RS_STATE_INT8 if eight else rs.RS_STATE_F32
        s["adamw"] = rs.AdamW([(n, kinds[case["param"]], kinds[case["grad"]], state, BLOCK if eight else 0, 0 if i < len(big) else 1)
                               for i, n in enumerate(sizes)]).upload()
        views = lambda x: None if x is None else [x[a:a + n] for a, n in zip(starts, sizes)]  # noqa: E731
        scales = lambda x: [x[a // BLOCK:(a + n + BLOCK - 1) // BLOCK] for a, n in zip(starts, sizes)] if eight else None  # noqa: E731
        s["adamw"].bind(views(s["param"]), views(s["grad"]), views(s["m"]), views(s["v"]), scales(s.get("amax_m")), scales(s.get("amax_v")),
                        views(s["out"]))
    return s


# ------------------------------------------------------------ plain forms

def _plain_sort(s, case):
    """First slot of every expert (and the end), tokens per expert, slot of every choice (-1: not taken)."""
    experts, align = case["experts"], case["align"]
    ids = s["topk"].reshape(-1)
    if s["mask"] is not None:
        ids = torch.where(s["mask"][:, None] != 0, s["topk"], torch.full_like(s["topk"], experts)).reshape(-1)
    order = torch.sort(ids, stable=True).indices
    count = torch.zeros(experts + 1, dtype=torch.int64, device=ids.device).scatter_add_(0, ids, torch.ones_like(ids))
    padded = (count + align - 1) // align * align
    first, start = count.cumsum(0) - count, padded.cumsum(0) - padded
    here = ids[order]
    slot = torch.empty_like(ids)
    slot[order] = torch.where(here < experts, start[here] + torch.arange(ids.numel(), device=ids.device) - first[here], torch.full_like(here, -1))
    return start, count[:experts].to(torch.int32), slot.to(torch.int32).view(s["topk"].shape)


def _to_slots(rows, slot, slots):
    """rows [n, hidden] at their slots, zeros elsewhere (a last row takes what has none)."""
    to = torch.where(slot < 0, torch.full_like(slot, slots), slot).long().reshape(-1)
    return torch.zeros(slots + 1, rows.shape[1], device=rows.device).index_copy_(0, to, rows)[:slots]


def _from_slots(y, slot):
    """y's rows [rows, k, hidden] for every choice, zeros for one without a slot."""
    got = y.float()[slot.clamp(min=0).long()]
    return torch.where((slot >= 0)[..., None], got, torch.zeros_like(got))


def _plain_experts(s, case):
    kind, k = s["x"].dtype, case["k"]
    if case["way"] == "forward":
        start, count, slot = _plain_sort(s, case)
        x = s["x"].float().repeat_interleave(k, dim=0)
        out = (s["weight"][..., None] * _from_slots(s["y"], slot)).sum(1)
        return {"start": start, "count": count, "slot": slot, "sorted": _to_slots(x, slot, s["slots"]).to(kind), "out": out.to(kind)}
    slot, dout = s["slot"], s["x"].float()
    dy = _to_slots((s["weight"][..., None] * dout[:, None, :]).reshape(-1, case["hidden"]), slot, s["slots"])
    dweight = (dout[:, None, :] * _from_slots(s["y"], slot)).sum(-1)
    return {"dy": dy.to(kind), "dweight": dweight, "dx": _from_slots(s["dsorted"], slot).sum(1).to(kind)}


def _plain_stats(s, case):
    rows, vocab = s["logits"].shape
    scale, n = 1.0 / case["temperature"], case["top"]
    valid = s["target"] >= 0
    target = s["target"].clamp(min=0)[:, None]
    z = s["logits"].float()
    m = z.amax(-1, keepdim=True)
    d = (z - m) * scale
    e = torch.exp(d)
    total = e.sum(-1, dtype=torch.float64)  # long sums in 64 bits
    away = d.clamp(min=-1e4)  # what is ruled out has no part: 0 times -inf is none
    mean = (e * away).sum(-1, dtype=torch.float64) / total
    log_total = torch.log(total)
    at = d.gather(1, target)[:, 0].double()
    zero = torch.zeros_like(total)
    got = {"logp": torch.where(valid, at - log_total, zero).float(), "entropy": torch.where(valid, log_total - mean, zero).float()}
    if n:
        # one key per value: larger values first, of equal ones the lower index
        bits = z.view(torch.int32).long()
        bits = torch.where(bits < 0, -(bits & 0x7fffffff), bits)
        key = (bits << 32) - torch.arange(vocab, device=z.device)
        ids = torch.topk(key, n, dim=-1).indices
        logp = d.gather(1, ids).double() - log_total[:, None]
        lost = ~valid[:, None] | torch.isinf(logp)
        got["top_id"] = torch.where(lost, torch.full_like(ids, -1), ids)
        got["top_logp"] = torch.where(lost, torch.full_like(logp, -math.inf), logp).float()
    if case["way"] == "train":
        # d logp / dz = [i = y] - p, d entropy / dz = -p (log p + entropy), both over the temperature
        c, b = s["dlogp"].double() * scale, s["dentropy"].double() * scale
        p = e / total.float()[:, None]
        level = (c - b * mean)[:, None].float()  # log p + entropy = d - mean
        g = -p * (level + b[:, None].float() * away)
        g.scatter_add_(1, target, c[:, None].float())
        got["dlogits"] = torch.where(valid[:, None], g, torch.zeros_like(g)).to(s["logits"].dtype)
    return got


def _plain_adamw(s, case):
    cut, eight = s["cut"], case["state"] == 8
    g = s["grad"].float()
    if case["clip"]:
        s["sumsq"].copy_(g.double().square().sum())
        s["scale"].copy_(torch.clamp(MAX_NORM / (torch.sqrt(s["sumsq"]) + 1e-6), max=1.0))
        g = g * s["scale"]
    if eight:
        # dividing by a tensor: a division by a plain number is turned into a product
        levels_m, levels_v = torch.full((1,), 127.0, device=g.device), torch.full((1,), 255.0, device=g.device)
        m = ((s["m"].float() / levels_m).view(-1, BLOCK) * s["amax_m"][:, None]).view(-1)
        v = ((s["v"].float() / levels_v).view(-1, BLOCK) * s["amax_v"][:, None]).view(-1)
    else:
        m, v = s["m"], s["v"]
    m = m * BETA1 + g * (1.0 - BETA1)
    v = v * BETA2 + (g * g) * (1.0 - BETA2)
    kappa, size = 1.0 / math.sqrt(1.0 - BETA2 ** STEP), LR / (1.0 - BETA1 ** STEP)
    p = s["param"].float()
    p = torch.cat([p[:cut] * (1.0 - LR * DECAY), p[cut:]]) - (m / (torch.sqrt(v) * kappa + EPS)) * size
    s["param"].copy_(p)
    got = {"param": s["param"]}
    if case["out"]:
        s["out"].copy_(p)
        got["out"] = s["out"]
    if case["clip"]:
        got["sumsq"], got["scale"] = s["sumsq"], s["scale"]
    if not eight:
        s["m"].copy_(m)
        s["v"].copy_(v)
        return {**got, "m": s["m"], "v": s["v"]}
    m, v = m.view(-1, BLOCK), v.view(-1, BLOCK)
    s["amax_m"].copy_(m.abs().amax(1))
    s["amax_v"].copy_(v.amax(1))
    some = lambda a: torch.where(a > 0, a, torch.ones_like(a))[:, None]  # noqa: E731
    s["m"].copy_(torch.round(m / some(s["amax_m"]) * 127.0).view(-1))
    s["v"].copy_(torch.round(v / some(s["amax_v"]) * 255.0).view(-1))
    m = (s["m"].float() / levels_m).view(-1, BLOCK) * s["amax_m"][:, None]
    v = (s["v"].float() / levels_v).view(-1, BLOCK) * s["amax_v"][:, None]
    return {**got, "m": m.view(-1)[s["where"]].bfloat16(), "v": v.view(-1)[s["where"]].bfloat16(), "amax_m": s["amax_m"], "amax_v": s["amax_v"]}


# ------------------------------------------------------------- one pass

def _own_experts(s, case):
    import sharded_state_raggedshard_amd as rs
    kind = rs.RS_F32 if case["type"] == "f32" else rs.RS_BF16
    rows, hidden, experts, k, slots = case["rows"], case["hidden"], case["experts"], case["k"], s["slots"]
    if case["way"] == "forward":
        rs.rs_expert_sort(s["topk"], rows, experts, k, k, s["mask"], case["align"], s["start"], s["count"], s["slot"], s["work"], s["work"].numel())
        rs.rs_expert_dispatch(s["x"], kind, rows, hidden, hidden, s["slot"], k, None, 0, experts, s["start"], s["count"], s["sorted"], slots, hidden)
        rs.rs_expert_combine(s["y"], kind, slots, hidden, hidden, s["slot"], rows, k, s["weight"], k, None, 0, s["out"], hidden)
        return {"start": s["start"], "count": s["count"], "slot": s["slot"], "sorted": s["sorted"], "out": s["out"]}
    rs.rs_expert_combine_grad(s["x"], kind, rows, hidden, hidden, s["y"], slots, hidden, s["slot"], k, s["weight"], k, experts, s["start"], s["count"],
                              s["sorted"], hidden, s["dweight"], k)
    rs.rs_expert_combine(s["dsorted"], kind, slots, hidden, hidden, s["slot"], rows, k, None, 0, None, 0, s["out"], hidden)
    return {"dy": s["sorted"], "dweight": s["dweight"], "dx": s["out"]}


def _own_stats(s, case):
    import sharded_state_raggedshard_amd as rs
    kind = rs.RS_F32 if case["type"] == "f32" else rs.RS_BF16
    rows, vocab = s["logits"].shape
    train, n = case["way"] == "train", case["top"]
    rs.rs_token_stats(s["logits"], kind, rows, vocab, vocab, s["target"], s["logp"], s["entropy"], n, s["top_id"] if n else None,
                      s["top_logp"] if n else None, s["saved"] if train else None, s["work"], s["work"].numel(), temperature=case["temperature"])
    got = {"logp": s["logp"], "entropy": s["entropy"]}
    if n:
        got["top_id"], got["top_logp"] = s["top_id"], s["top_logp"]
    if train:
        rs.rs_token_stats_grad(s["logits"], kind, rows, vocab, vocab, s["target"], s["saved"], s["dlogp"], s["dentropy"], s["dlogits"], vocab,
                               temperature=case["temperature"])
        got["dlogits"] = s["dlogits"]
    return got


def _own_adamw(s, case):
    import sharded_state_raggedshard_amd as rs
    h = s["adamw"]
    if case["clip"]:
        h.l2norm_clip(MAX_NORM, s["sumsq"], s["scale"])
    h.step([dict(lr=LR, beta1=BETA1, beta2=BETA2, eps=EPS, weight_decay=decay, step=STEP) for decay in (DECAY, 0.0)],
           grad_scale=s["scale"] if case["clip"] else None)
    got = {"param": s["param"]}
    if case["out"]:
        got["out"] = s["out"]
    if case["clip"]:
        got["sumsq"], got["scale"] = s["sumsq"], s["scale"]
    if case["state"] == 32:
        return {**got, "m": s["m"], "v": s["v"]}
    h.moments(s["m_values"], s["v_values"], rs.RS_BF16)
    return {**got, "m": s["m_values"], "v": s["v_values"], "amax_m": s["amax_m"], "amax_v": s["amax_v"]}


def run(state):
    case = state["case"]
    if own:
        return {"experts": _own_experts, "stats": _own_stats, "adamw": _own_adamw}[case["op"]](state, case)
    return {"experts": _plain_experts, "stats": _plain_stats, "adamw": _plain_adamw}[case["op"]](state, case)


# ---------------------------------------------------- 64-bit definitions

def exact(case, seed):
    s = prepare(case, seed)
    return {"experts": _exact_experts, "stats": _exact_stats, "adamw": _exact_adamw}[case["op"]](s, case)


def _exact_experts(s, case):
    """Choice by choice: the lists of every expert in the order of the tokens."""
    rows, hidden, experts, k, slots = case["rows"], case["hidden"], case["experts"], case["k"], s["slots"]
    live = [True] * rows if s["mask"] is None else [bool(x) for x in s["mask"].tolist()]
    lists = [[] for _ in range(experts)]
    for t, ids in enumerate(s["topk"].tolist()):
        if live[t]:
            for j, e in enumerate(ids):
                lists[e].append(t * k + j)
    start, choice, at = [0], [], []
    for one in lists:
        choice += one
        at += range(start[-1], start[-1] + len(one))
        start.append(start[-1] + -(-len(one) // case["align"]) * case["align"])
    choice, at = torch.tensor(choice, device="cuda"), torch.tensor(at, device="cuda")
    token, w = choice // k, s["weight"].reshape(-1).double()
    got = {}
    some = max(1, (1 << 28) // hidden)  # rows at a time
    if case["way"] == "forward":
        got["start"], got["count"] = torch.tensor(start, device="cuda"), torch.tensor([len(one) for one in lists], dtype=torch.int32, device="cuda")
        slot = torch.full((rows * k,), -1, dtype=torch.int32, device="cuda")
        slot[choice] = at.int()
        got["slot"] = slot.view(rows, k)
        got["sorted"], got["out"] = s["x"].new_zeros(slots, hidden, dtype=torch.float64), s["x"].new_zeros(rows, hidden, dtype=torch.float64)
        for a in range(0, len(choice), some):
            t, i, c = token[a:a + some], at[a:a + some], choice[a:a + some]
            got["sorted"][i] = s["x"][t].double()
            got["out"].index_add_(0, t, s["y"][i].double() * w[c, None])
        return got
    got["dy"], got["dx"] = s["x"].new_zeros(slots, hidden, dtype=torch.float64), s["x"].new_zeros(rows, hidden, dtype=torch.float64)
    dweight = torch.zeros(rows * k, dtype=torch.float64, device="cuda")
    for a in range(0, len(choice), some):
        t, i, c = token[a:a + some], at[a:a + some], choice[a:a + some]
        dout = s["x"][t].double()
        got["dy"][i] = dout * w[c, None]
        dweight[c] = (dout * s["y"][i].double()).sum(1)
        got["dx"].index_add_(0, t, s["dsorted"][i].double())
    return {**got, "dweight": dweight.view(rows, k)}


def _exact_stats(s, case):
    """log softmax some rows at a time; the gradient by the chain rule of autograd."""
    rows, vocab = s["logits"].shape
    n, train = case["top"], case["way"] == "train"
    some = max(1, (1 << 26) // vocab)
    parts = []
    for a in range(0, rows, some):
        here = slice(a, a + some)
        t = s["target"][here]
        live = t >= 0
        z = s["logits"][here].double().requires_grad_(train)
        ls = torch.log_softmax(z / case["temperature"], dim=-1)
        logp = ls.gather(1, t.clamp(min=0)[:, None])[:, 0] * live
        p = torch.exp(ls)
        entropy = -torch.where(p > 0, p * ls.masked_fill(p == 0, 0.0), torch.zeros_like(p)).sum(-1) * live
        got = {"logp": logp.detach(), "entropy": entropy.detach()}
        if n:
            # a stable sort keeps equal values in the order of their indexes
            best = torch.sort(ls.detach(), dim=-1, descending=True, stable=True)
            values, ids = best.values[:, :n], best.indices[:, :n]
            lost = ~live[:, None] | torch.isinf(values)
            got["top_id"], got["top_logp"] = ids.masked_fill(lost, -1), values.masked_fill(lost, -math.inf)
        if train:
            loss = (s["dlogp"][here].double() * logp).sum() + (s["dentropy"][here].double() * entropy).sum()
            (got["dlogits"],) = torch.autograd.grad(loss, z)
        parts.append(got)
    return {name: torch.cat([x[name] for x in parts]) for name in parts[0]}


def _exact_adamw(s, case):
    """The definition of the step, every quantity in 64 bits, tensor stores as prepared."""
    eight, cut = case["state"] == 8, s["cut"]
    grad, theta = s["grad"].double(), s["param"].double()
    blocks = lambda x: x.view(-1, BLOCK)  # noqa: E731
    got = {}
    if case["clip"]:
        norm = torch.linalg.vector_norm(grad)
        got["sumsq"] = (norm ** 2).view(1)
        got["scale"] = torch.minimum(torch.ones_like(norm), MAX_NORM / (norm + 1e-6)).view(1)
        grad = grad * got["scale"]
    if eight:
        m0 = (blocks(s["m"].double()) * s["amax_m"].double()[:, None] / 127).view(-1)
        v0 = (blocks(s["v"].double()) * s["amax_v"].double()[:, None] / 255).view(-1)
    else:
        m0, v0 = s["m"].double(), s["v"].double()
    m, v = torch.lerp(grad, m0, BETA1), torch.lerp(grad.square(), v0, BETA2)
    hat_m, hat_v = m / (1 - BETA1 ** STEP), v / (1 - BETA2 ** STEP)
    theta[:cut] -= LR * DECAY * theta[:cut]
    theta -= LR * hat_m / (hat_v.sqrt() + EPS)
    got["param"] = theta
    if case["out"]:
        got["out"] = theta
    if not eight:
        return {**got, "m": m, "v": v}
    got["amax_m"], got["amax_v"] = blocks(m).abs().amax(1), blocks(v).amax(1)
    for name, x, levels in (("m", m, 127), ("v", v, 255)):
        step = (got["amax_" + name] / levels)[:, None]
        got[name] = torch.nan_to_num(torch.round(blocks(x) / step) * step).view(-1)[s["where"]]
    return got
