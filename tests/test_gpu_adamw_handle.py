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
