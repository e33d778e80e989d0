"""One rank's training-state update with the library, end to end.

    python -m sharded_state_raggedshard_amd.example

Plans three tensors over m = 4 ranks: the output head of a tiny model and a
router in one bucket (matrices in 128 x 128 tiles), the head's bias in
another (a vector in 32-element blocks); neither bucket needs padding.
Copies fp32 master parameters in, and runs a few steps of: the losses on
random hidden states with their logits' gradients (a preference loss on
packed pairs in the first step, a clipped policy loss with a KL term after
it; the router's balance loss in each), the parameters' gradients into the
grad DBuffer, global L2 norm with the clipping coefficient, the
blockwise-int8 AdamW step of rank `rank` (grad scale = the coefficient, bf16
copy-in of the new parameters fused), zeroing of the gradients, copy-out to
per-parameter bf16 views.  On m GPUs each rank would run the same calls on
its own slices and an AllGather / ReduceScatter would move the bf16 buffer
between them; on one GPU every rank's slice lives in the same arrays.
"""
from __future__ import annotations

import torch

import sharded_state_raggedshard_amd as rs
from synth import ROWS, TILE, TensorSpec


TOKENS, TOPK, PAIRS = 96, 4, 4


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
    nbytes = max(rs.rs_objective_bytes(TOKENS, vocab, 2 * PAIRS),
                 rs.rs_router_balance_bytes(TOKENS, experts))
    work = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    start = torch.arange(2 * PAIRS + 1, device=dev) * (TOKENS // (2 * PAIRS))
    weight = torch.full((TOKENS,), 1.0 / TOKENS, device=dev)
    for t in range(1, steps + 1):
        # forward pass of the tiny model on random hidden states
        w, router, b = (v.view(torch.bfloat16).float() for v in weights)
        w, router = w.view(vocab, 512), router.view(experts, 512)
        x = torch.randn(TOKENS, 512, device=dev)
        logits, scores = x @ w.T + b, x @ router.T
        target = torch.randint(0, vocab, (TOKENS,), device=dev)
        if t == 1:
            rs.rs_preference_loss(logits, rs.RS_F32, TOKENS, vocab, vocab, target, start, PAIRS,
                                  None, None, dlogits, vocab, seq_logp, pair_stats, work, nbytes)
        else:
            rs.rs_token_logp(logits, rs.RS_F32, TOKENS, vocab, vocab, target, old_logp, work,
                             nbytes)
            ref_logp.copy_(old_logp).add_(0.1 * torch.randn(TOKENS, device=dev))
            advantage = torch.randn(TOKENS, device=dev)
            rs.rs_policy_loss(logits, rs.RS_F32, TOKENS, vocab, vocab, target, old_logp, ref_logp,
                              advantage, weight, dlogits, vocab, logp, policy_stats, work, nbytes,
                              kl_coef=0.05)
        topk = scores.topk(TOPK).indices
        rs.rs_router_balance(scores, rs.RS_F32, TOKENS, experts, experts, topk, TOPK, TOPK, None,
                             None, 1, drouter, experts, counts, mean_prob, router_stats, work,
                             nbytes)
        # backward pass accumulating into the grad DBuffer
        for i, g in enumerate((dlogits.T @ x, drouter.T @ x, dlogits.sum(0))):
            n = specs[i].numel
            grad[plan.pos[i]:plan.pos[i] + n] = g.to(torch.bfloat16).reshape(-1).view(torch.int16)
        rs.rs_group_l2norm_clip(plan.h, rs.RS_ALL, rank, grad, rs.RS_BF16, 1.0, sumsq, clip)
        rs.rs_adam8_step(plan.h, rs.RS_ALL, rank, theta, grad, qm, qv, amax_m, amax_v,
                         lr=1e-3, step=t, grad_scale=clip, bf16_out=gathered)
        rs.rs_group_zero(plan.h, rs.RS_ALL, rank, grad, rs.RS_BF16)
        rs.rs_unpack_full(plan.h, rs.RS_ALL, gathered)
    rs.rs_plan_check_device(plan.h)  # no cross-workgroup wait gave up
    torch.cuda.synchronize()
    out = {"S": plan.S, "padding": plan.padding, "grad_norm": sumsq.sqrt().item(),
           "clip": clip.item(), "weights": [w.view(torch.bfloat16).float() for w in weights],
           "theta": theta, "plan": plan, "preference": pair_stats, "policy": policy_stats,
           "router": router_stats, "counts": counts}
    return out


if __name__ == "__main__":
    r = main()
    print(f"S per bucket {r['S']}, padding {r['padding']}, last grad norm {r['grad_norm']:.4g}, "
          f"clip {r['clip']:.4g}")
    r["plan"].free()
