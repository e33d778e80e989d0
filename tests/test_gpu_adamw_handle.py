"""The AdamW class of the binding on the device: what a refused call leaves."""
import pytest
import torch

import sharded_state_raggedshard_amd as rs
from gpu_harness import log

pytestmark = pytest.mark.gpu

F32 = rs.RS_F32
HP = dict(lr=1e-2, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, step=1)


def made(n=5000):
    h = rs.AdamW([(n, F32, F32, rs.RS_STATE_F32, 0, 0)]).upload()
    a = dict(params=[torch.ones(n, device="cuda")], grads=[torch.ones(n, device="cuda")],
             m=[torch.zeros(n, device="cuda")], v=[torch.zeros(n, device="cuda")])
    return h.bind(**a), a


def test_a_refused_upload_leaves_a_working_plan():
    log("adamw refused upload")
    h, a = made()
    before = h.workspace
    with pytest.raises(rs.RaggedShardError):
        h.upload(device="cpu")
    assert h.workspace is before
    torch.full((before.numel(),), 0xFF, dtype=torch.uint8, device="cuda")  # what was let go of would be here
    h.step([HP])
    # m / sqrt(v) of a first step is 1: (1 - lr) within its roundings
    assert ((a["params"][0] - 0.99).abs() <= 1e-6).all()
    h.free()


def test_a_refused_binding_writes_nothing_and_keeps_the_old_one():
    log("adamw refused binding")
    h, a = made()
    other = {k: [x[0].clone().int() if k == "params" else x[0].clone()] for k, x in a.items()}
    with pytest.raises(rs.RaggedShardError):
        h.bind(**other)
    h.step([HP])
    assert (other["params"][0] == 1).all() and ((a["params"][0] - 0.99).abs() <= 1e-6).all()
    h.free()


def test_a_norm_that_gave_up_shows_until_the_next_upload():
    """The mark that a bounded wait leaves, set from the host: the last 64 words
    of the workspace begin with the number of the last call, then the mark."""
    log("adamw norm behind a mark")
    h, a = made(3 * 4096 + 5)
    sumsq, scale = torch.zeros(1, dtype=torch.float64, device="cuda"), torch.zeros(1, device="cuda")
    n = a["grads"][0].numel()
    for turn in range(2):
        words = h.workspace.view(torch.int32)[-64:]
        for call in (1, 2):
            h.l2norm_clip(1.0, sumsq, scale)
            assert sumsq.item() == n and abs(scale.item() * n ** 0.5 - 1) < 1e-5
            assert words[:3].tolist() == [call, 0, 0]
        words[1] = 1
        for call in (3, 4):
            sumsq.zero_()
            scale.zero_()
            h.l2norm_clip(1.0, sumsq, scale)
            assert torch.isnan(sumsq).all() and torch.isnan(scale).all()
        h.upload().bind(**a)
    h.free()
