"""The AdamW class of the binding: what it refuses before the library is
called, on tensors of the host (a call that gets past its checks is refused for
the device that they are on)."""
import pytest
import torch

import sharded_state_raggedshard_amd as rs

F32, BF16 = rs.RS_F32, rs.RS_BF16
N, BLOCK = 600, 256


def lists(**other):
    """Arrays of a binary32 tensor with 8-bit moments and of a bf16 one with binary32 moments."""
    a = dict(params=[torch.zeros(N), torch.zeros(N, dtype=torch.bfloat16)],
             grads=[torch.zeros(N, dtype=torch.bfloat16), torch.zeros(N)],
             m=[torch.zeros(N, dtype=torch.int8), torch.zeros(N)], v=[torch.zeros(N, dtype=torch.uint8), torch.zeros(N)],
             amax_m=[torch.zeros(3), None], amax_v=[torch.zeros(3), None],
             bf16_out=[torch.zeros(N, dtype=torch.bfloat16), None])
    for name, (i, dtype) in other.items():
        a[name][i] = a[name][i].to(dtype)
    return a


@pytest.fixture
def adamw():
    h = rs.AdamW([(N, F32, BF16, rs.RS_STATE_INT8, BLOCK, 0), (N, BF16, F32, rs.RS_STATE_F32, 0, 0)])
    yield h
    h.free()


@pytest.mark.parametrize("other", [{}, dict(grads=(0, torch.int16), bf16_out=(0, torch.uint16)), dict(params=(1, torch.int16))])
def test_types_of_the_plan_pass(adamw, other):
    """bf16 also as its bits."""
    with pytest.raises(rs.RaggedShardError, match="not on the current device"):
        adamw.bind(**lists(**other))


WRONG = [("params", 0, torch.int32), ("params", 1, torch.float16), ("grads", 0, torch.float16), ("grads", 1, torch.int32),
         ("m", 0, torch.uint8), ("v", 0, torch.int8), ("m", 1, torch.int32), ("v", 1, torch.int32), ("amax_m", 0, torch.int32),
         ("amax_v", 0, torch.int32), ("bf16_out", 0, torch.float16)]


@pytest.mark.parametrize("name,i,dtype", WRONG)
def test_other_types_of_the_same_width_are_refused(adamw, name, i, dtype):
    with pytest.raises(rs.RaggedShardError, match=f"tensor {i}: .*{dtype}") as e:
        adamw.bind(**lists(**{name: (i, dtype)}))
    assert e.value.status == rs.RS_EINVAL
    assert adamw.arrays is None


def test_an_empty_tensor_of_another_type_is_not_looked_at():
    h = rs.AdamW([(0, F32, F32, rs.RS_STATE_F32, 0, 0), (N, F32, F32, rs.RS_STATE_F32, 0, 0)])
    empty, full = torch.zeros(0, dtype=torch.float16), torch.zeros(N)
    with pytest.raises(rs.RaggedShardError, match="not on the current device"):
        h.bind(*[[empty, full] for _ in range(4)])
    h.free()


def test_a_refused_upload_leaves_what_was_there(adamw):
    """The plan still points into the old workspace, so somebody has to hold it."""
    workspace, arrays = object(), [object()]
    adamw.workspace, adamw.arrays = workspace, arrays
    with pytest.raises(rs.RaggedShardError, match="not on the current device"):
        adamw.upload(device="cpu")
    assert adamw.workspace is workspace and adamw.arrays is arrays


def test_an_upload_lets_go_of_what_was_bound(adamw, monkeypatch):
    monkeypatch.setattr(rs, "rs_adamw_upload", lambda *a: None)
    adamw.arrays = [object()]
    assert adamw.upload(device="cpu") is adamw
    assert adamw.workspace.numel() == rs.rs_adamw_device_bytes(adamw.h) and adamw.arrays is None


def test_what_is_bound_does_not_follow_the_callers_lists(adamw, monkeypatch):
    """The plan points to the tensors that were bound: they live on when the
    caller's lists let go of them, as where gradients are set to None."""
    monkeypatch.setattr(rs, "rs_adamw_bind", lambda *a, **k: None)
    a = lists()
    bound = [list(x) for x in a.values()]
    adamw.bind(**a)
    for x in a.values():
        x[0] = None
        x.clear()
    assert all(held is not None and len(held) == len(was) and all(x is y for x, y in zip(held, was))
               for held, was in zip(adamw.arrays, bound))
