"""One rank's training-state update with the library, end to end.

    python -m sharded_state_raggedshard_amd.example

Plans three tensors over m = 4 ranks: the output head of a tiny model and a
router in one bucket (matrices in 128 x 128 tiles), the head's bias in
another (a vector in 32-element blocks); neither bucket needs padding.
Copies fp32 master parameters in, and runs a few steps of: the tokens of
random hidden states sorted by the router's choices, carried to the experts
(each scales its rows) and back with their weights, the losses on what comes
out with their logits' gradients (a preference loss on packed pairs in the
first step, a clipped policy loss with a KL term in the second, a weighted
log-probability with an entropy bonus from then on; the router's balance loss
in each), the way back through the experts, the parameters' gradients into
the grad DBuffer, global L2 norm with the clipping coefficient, the
blockwise-int8 AdamW step of rank `rank` (grad scale = the coefficient, bf16
copy-in of the new parameters fused), zeroing of the gradients, copy-out to
per-parameter bf16 views; and, for the experts' scales and a scale of the
hidden states, which no plan holds, an AdamW step over both tensors.  On m GPUs each rank would run the same calls on
its own slices and an AllGather / ReduceScatter would move the bf16 buffer
between them; on one GPU every rank's slice lives in the same arrays.
"""
from __future__ import annotations

import torch

import sharded_state_raggedshard_amd as rs
from synth import ROWS, TILE, TensorSpec


TOKENS, TOPK, PAIRS, ALTERNATIVES, TILE_ROWS = 96, 4, 4, 5, 2


def main(steps: int = 3, rank: int = rs.RS_ALL) -> dict:
    specs = [TensorSpec("w", (1024, 512), TILE, 128, 128, bucket=0),
             TensorSpec("router", (512, 512), TILE, 128, 128, bucket=0),
             TensorSpec("b", (1024,), ROWS, 32, bucket=1)]
    plan = rs.Plan(specs, 4, 16).upload()  # layout, then its device tables
    dev = "cuda"
    total, nblk = plan.total, plan.n_blocks
    vocab, experts = 1024, 512
    # the DBuffers: one array per state in the planned layout
    theta = torch.zeros(total, device=dev)                      # fp32 master
    grad = torch.zeros(total, dtype=torch.int16, device=dev)    # bf16 bits
    qm = torch.zeros(total, dtype=torch.int8, device=dev)       # int8 m codes
    qv = torch.zeros(total, dtype=torch.uint8, device=dev)      # uint8 v codes
    amax_m = torch.zeros(nblk, device=dev)                      # one absmax per block
    amax_v = torch.zeros(nblk, device=dev)
    gathered = torch.zeros(total, dtype=torch.int16, device=dev)  # bf16 buffer
    sumsq = torch.zeros(1, dtype=torch.float64, device=dev)
    clip = torch.zeros(1, device=dev)
    # per-parameter views: fp32 masters to copy in, bf16 weights to copy out
    masters = [torch.randn(s.numel, device=dev) * 0.02 for s in specs]
    weights = [torch.zeros(s.numel, dtype=torch.int16, device=dev) for s in specs]
    rs.rs_bind_views(plan.h, rs.RS_VIEW_F32_SRC, masters)
    rs.rs_bind_views(plan.h, rs.RS_VIEW_BF16_DST, weights)
    rs.rs_pack_shard(plan.h, rs.RS_ALL, rs.RS_ALL, gathered)  # initial bf16 copy-in
    rs.rs_unpack_full(plan.h, rs.RS_ALL, gathered)
    for i, s in enumerate(specs):  # the master in the planned layout
        theta[plan.pos[i]:plan.pos[i] + s.numel] = masters[i]
    # the objectives' outputs and one scratch area for all of them
    dlogits = torch.empty(TOKENS, vocab, device=dev)
    drouter = torch.empty(TOKENS, experts, device=dev)
    old_logp, ref_logp, logp = (torch.zeros(TOKENS, device=dev) for _ in range(3))
    seq_logp = torch.zeros(2 * PAIRS, device=dev)
    counts = torch.zeros(experts, dtype=torch.int32, device=dev)
    mean_prob = torch.zeros(experts, device=dev)
    policy_stats, pair_stats, router_stats = (torch.zeros(n, device=dev) for n in (4, 3, 2))
    entropy, saved = torch.zeros(TOKENS, device=dev), torch.zeros(TOKENS, 4, device=dev)
    top_id = torch.zeros(TOKENS, ALTERNATIVES, dtype=torch.int64, device=dev)
    top_logp = torch.zeros(TOKENS, ALTERNATIVES, device=dev)
    nbytes = max(rs.rs_objective_bytes(TOKENS, vocab, 2 * PAIRS),
                 rs.rs_router_balance_bytes(TOKENS, experts),
                 rs.rs_token_stats_bytes(TOKENS, vocab, ALTERNATIVES),
                 rs.rs_expert_sort_bytes(TOKENS, experts, TOPK))
    work = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    start = torch.arange(2 * PAIRS + 1, device=dev) * (TOKENS // (2 * PAIRS))
    weight = torch.full((TOKENS,), 1.0 / TOKENS, device=dev)
    # the sorted tokens, in tiles of rows per expert, and their gradients
    slots = rs.rs_expert_slots(TOKENS, experts, TOPK, TILE_ROWS)
    first = torch.zeros(experts + 1, dtype=torch.int64, device=dev)
    taken = torch.zeros(experts, dtype=torch.int32, device=dev)
    slot = torch.zeros(TOKENS, TOPK, dtype=torch.int32, device=dev)
    rows, drows = torch.zeros(slots, 512, device=dev), torch.zeros(slots, 512, device=dev)
    mixed, dx = torch.zeros(TOKENS, 512, device=dev), torch.zeros(TOKENS, 512, device=dev)
    dgate = torch.zeros(TOKENS, TOPK, device=dev)
    # parameters of no plan: the experts' scales with 8-bit moments, a scale of
    # the hidden states with binary32 ones and no weight decay
    scales = [torch.ones(experts, 512, device=dev), torch.ones(512, device=dev)]
    dscales = [torch.zeros_like(p) for p in scales]
    adamw = rs.AdamW([(experts * 512, rs.RS_F32, rs.RS_F32, rs.RS_STATE_INT8_ROOT, 256, 0),
                      (512, rs.RS_F32, rs.RS_F32, rs.RS_STATE_F32, 0, 1)]).upload()
    adamw.bind(scales, dscales,
               [torch.zeros(experts * 512, dtype=torch.int8, device=dev), torch.zeros(512, device=dev)],
               [torch.zeros(experts * 512, dtype=torch.uint8, device=dev), torch.zeros(512, device=dev)],
               [torch.zeros(experts * 2, device=dev), None], [torch.zeros(experts * 2, device=dev), None])
    other_sumsq, other_clip = torch.zeros(1, dtype=torch.float64, device=dev), torch.zeros(1, device=dev)
    for t in range(1, steps + 1):
        # forward pass of the tiny model on random hidden states
        w, router, b = (v.view(torch.bfloat16).float() for v in weights)
        w, router = w.view(vocab, 512), router.view(experts, 512)
        hidden = torch.randn(TOKENS, 512, device=dev)
        x = hidden * scales[1]
        scores = x @ router.T
        values, topk = scores.topk(TOPK)
        gate = torch.softmax(values, -1)
        rs.rs_expert_sort(topk, TOKENS, experts, TOPK, TOPK, None, TILE_ROWS, first, taken, slot, work, nbytes)
        rs.rs_expert_dispatch(x, rs.RS_F32, TOKENS, 512, 512, slot, TOPK, None, 0, experts, first, taken, rows, slots,
                              512)
        of = torch.searchsorted(first[1:], torch.arange(slots, device=dev), right=True).clamp(max=experts - 1)
        made = rows * scales[0][of]  # the experts: a row of each one's tile times its scales
        rs.rs_expert_combine(made, rs.RS_F32, slots, 512, 512, slot, TOKENS, TOPK, gate, TOPK, x, 512, mixed, 512)
        logits = mixed @ w.T + b
        target = torch.randint(0, vocab, (TOKENS,), device=dev)
        if t == 1:
            rs.rs_preference_loss(logits, rs.RS_F32, TOKENS, vocab, vocab, target, start, PAIRS,
                                  None, None, dlogits, vocab, seq_logp, pair_stats, work, nbytes)
        elif t == 2:
            rs.rs_token_logp(logits, rs.RS_F32, TOKENS, vocab, vocab, target, old_logp, work,
                             nbytes)
            ref_logp.copy_(old_logp).add_(0.1 * torch.randn(TOKENS, device=dev))
            advantage = torch.randn(TOKENS, device=dev)
            rs.rs_policy_loss(logits, rs.RS_F32, TOKENS, vocab, vocab, target, old_logp, ref_logp,
                              advantage, weight, dlogits, vocab, logp, policy_stats, work, nbytes,
                              kl_coef=0.05)
        else:
            rs.rs_token_stats(logits, rs.RS_F32, TOKENS, vocab, vocab, target, logp, entropy, ALTERNATIVES, top_id,
                              top_logp, saved, work, nbytes)
            # loss = -sum weight (advantage logp + 0.01 entropy)
            rs.rs_token_stats_grad(logits, rs.RS_F32, TOKENS, vocab, vocab, target, saved,
                                   -weight * torch.randn(TOKENS, device=dev), -0.01 * weight, dlogits, vocab)
        rs.rs_router_balance(scores, rs.RS_F32, TOKENS, experts, experts, topk, TOPK, TOPK, None,
                             None, 1, drouter, experts, counts, mean_prob, router_stats, work,
                             nbytes)
        # backward pass: through the head and the experts to the hidden states,
        # the parameters' gradients accumulating into the grad DBuffer
        dmixed = dlogits @ w
        rs.rs_expert_combine_grad(dmixed, rs.RS_F32, TOKENS, 512, 512, made, slots, 512, slot, TOPK, gate, TOPK,
                                  experts, first, taken, drows, 512, dgate, TOPK)
        live = torch.arange(slots, device=dev) < first[-1]
        dscales[0].zero_().index_add_(0, of[live], (drows * rows)[live])
        drows *= scales[0][of]
        rs.rs_expert_combine(drows, rs.RS_F32, slots, 512, 512, slot, TOKENS, TOPK, None, 0, dmixed, 512, dx, 512)
        dvalues = gate * (dgate - (gate * dgate).sum(-1, keepdim=True))
        drouter.scatter_add_(1, topk, dvalues)
        dx += drouter @ router
        torch.sum(dx * hidden, 0, out=dscales[1])
        for i, g in enumerate((dlogits.T @ mixed, drouter.T @ x, dlogits.sum(0))):
            n = specs[i].numel
            grad[plan.pos[i]:plan.pos[i] + n] = g.to(torch.bfloat16).reshape(-1).view(torch.int16)
        rs.rs_group_l2norm_clip(plan.h, rs.RS_ALL, rank, grad, rs.RS_BF16, 1.0, sumsq, clip)
        rs.rs_adam8_step(plan.h, rs.RS_ALL, rank, theta, grad, qm, qv, amax_m, amax_v,
                         lr=1e-3, step=t, grad_scale=clip, bf16_out=gathered)
        adamw.l2norm_clip(1.0, other_sumsq, other_clip)
        adamw.step([dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=decay, step=t) for decay in (0.01, 0.0)],
                   grad_scale=other_clip)
        rs.rs_group_zero(plan.h, rs.RS_ALL, rank, grad, rs.RS_BF16)
        rs.rs_unpack_full(plan.h, rs.RS_ALL, gathered)
    rs.rs_plan_check_device(plan.h)  # no cross-workgroup wait gave up
    torch.cuda.synchronize()
    out = {"S": plan.S, "padding": plan.padding, "grad_norm": sumsq.sqrt().item(),
           "clip": clip.item(), "weights": [w.view(torch.bfloat16).float() for w in weights],
           "theta": theta, "plan": plan, "preference": pair_stats, "policy": policy_stats,
           "router": router_stats, "counts": counts,
           "taken": taken, "entropy": entropy, "top_id": top_id, "top_logp": top_logp, "scales": scales,
           "scales_norm": other_sumsq.sqrt().item()}
    return out


if __name__ == "__main__":
    r = main()
    print(f"S per bucket {r['S']}, padding {r['padding']}, last grad norm {r['grad_norm']:.4g}, "
          f"clip {r['clip']:.4g}")
    r["plan"].free()
