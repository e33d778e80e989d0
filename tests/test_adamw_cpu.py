"""AdamW over many tensors: what the entry points refuse, on the host and
before any launch.  Arrays are addresses that nothing reads; calls that pass
every check of their arguments end with RS_ESTATE, as nothing is uploaded."""
import random

import pytest
import torch

import sharded_state_raggedshard_amd as rs

F32, BF16 = rs.RS_F32, rs.RS_BF16
OK = (1000, F32, BF16, rs.RS_STATE_F32, 0, 0)
EIGHT = (1000, F32, BF16, rs.RS_STATE_INT8, 256, 0)
AT = 1 << 40


def status(call, *args, **kw):
    with pytest.raises(rs.RaggedShardError) as e:
        call(*args, **kw)
    return e.value.status


@pytest.fixture
def handles():
    made = []

    def make(*tensors):
        made.append(rs.rs_adamw_plan(tensors))
        return made[-1]
    yield make
    for h in made:
        rs.rs_adamw_free(h)


@pytest.mark.parametrize("at,value", [(0, -1), (1, 2), (2, -1), (3, 3), (3, -1), (4, 64), (5, -1), (5, 16)])
def test_bad_tensors(at, value):
    t = list(OK)
    t[at] = value
    assert status(rs.rs_adamw_plan, [OK, t]) == rs.RS_EINVAL


@pytest.mark.parametrize("block", [0, 1, 32, 63, 96, 4095, 8192, -256])
def test_bad_blocks(block):
    for state in (rs.RS_STATE_INT8, rs.RS_STATE_INT8_ROOT):
        assert status(rs.rs_adamw_plan, [(1000, F32, F32, state, block, 0)]) == rs.RS_EINVAL


def test_sizes():
    assert status(rs.rs_adamw_plan, []) == rs.RS_EINVAL
    assert status(rs.rs_adamw_plan, [((1 << 42) + 1, *OK[1:])]) == rs.RS_EOVERFLOW
    assert status(rs.rs_adamw_plan, [(1 << 42, *OK[1:])] * 3) == rs.RS_EOVERFLOW
    assert status(rs.rs_adamw_device_bytes, None) == rs.RS_EINVAL
    rs.rs_adamw_free(None)


def test_workspace_grows_with_the_tensors(handles):
    sizes = [rs.rs_adamw_device_bytes(handles(*[(n, *OK[1:])] * 3)) for n in (0, 1, 4096, 4097, 1 << 24)]
    assert sizes == sorted(sizes) and sizes[0] > 0 and sizes[-1] > sizes[0]


def test_upload_refusals(handles):
    h = handles(OK)
    n = rs.rs_adamw_device_bytes(h)
    assert status(rs.rs_adamw_upload, h, None, n, stream=0) == rs.RS_EINVAL
    assert status(rs.rs_adamw_upload, h, AT + 16, n, stream=0) == rs.RS_EINVAL
    assert status(rs.rs_adamw_upload, h, AT, n - 1, stream=0) == rs.RS_ENOMEM
    assert status(rs.rs_adamw_upload, None, AT, n, stream=0) == rs.RS_EINVAL


def lists(n=2, eight=False, out=False):
    """Apart arrays for n tensors of 1000 elements."""
    at = lambda i: [AT + (8 * j + i) * 8192 for j in range(n)]  # noqa: E731
    return dict(params=at(0), grads=at(1), m=at(2), v=at(3), amax_m=at(4) if eight else None,
                amax_v=at(5) if eight else None, bf16_out=at(6) if out else None)


def test_bind_takes_arrays_that_are_apart(handles):
    for eight in (False, True):
        h = handles(*[EIGHT if eight else OK] * 2)
        for out in (False, True):
            assert status(rs.rs_adamw_bind, h, **lists(eight=eight, out=out), stream=0) == rs.RS_ESTATE
    # adjacent arrays; shared gradients; nothing bound of an empty tensor
    h = handles(OK, OK)
    a = lists()
    a["params"][1] = a["params"][0] + 4000
    a["grads"][1] = a["grads"][0] + 500
    assert status(rs.rs_adamw_bind, h, **a, stream=0) == rs.RS_ESTATE
    h = handles(OK, (0, *EIGHT[1:]))
    a = lists(eight=True)
    for x in a.values():
        if x:
            x[1] = None
    assert status(rs.rs_adamw_bind, h, **a, stream=0) == rs.RS_ESTATE


@pytest.mark.parametrize("name,off", [("params", 2), ("grads", 1), ("m", 2), ("v", 1), ("amax_m", 2), ("amax_v", 1),
                                      ("bf16_out", 1), ("params", None), ("grads", None), ("m", None), ("v", None),
                                      ("amax_m", None)])
def test_bind_refuses_misaligned_and_missing(handles, name, off):
    h = handles(OK, EIGHT)
    a = lists(eight=True, out=True)
    at = 0 if name in ("m", "v") and off else 1  # codes need no alignment, binary32 moments do
    a[name][at] = None if off is None else a[name][at] + off
    assert status(rs.rs_adamw_bind, h, **a, stream=0) == rs.RS_EINVAL


def test_bind_refuses_missing_lists_and_a_copy_of_bf16(handles):
    h = handles(EIGHT, OK)
    for name in ("grads", "m", "v", "amax_m", "amax_v"):
        assert status(rs.rs_adamw_bind, h, **{**lists(eight=True), name: None}, stream=0) == rs.RS_EINVAL
    h = handles((1000, BF16, BF16, rs.RS_STATE_F32, 0, 0), OK)
    assert status(rs.rs_adamw_bind, h, **lists(out=True), stream=0) == rs.RS_EINVAL
    a = lists(out=True)
    a["bf16_out"][0] = None
    assert status(rs.rs_adamw_bind, h, **a, stream=0) == rs.RS_ESTATE


def test_bind_refuses_exactly_what_overlaps(handles):
    """Random places against the sets of bytes."""
    rng = random.Random(7)
    kinds = [0, 0]
    for _ in range(1500):
        n = rng.randrange(1, 4)
        tensors = []
        for _ in range(n):
            eight = rng.random() < 0.5
            tensors.append((rng.randrange(0, 130), rng.choice([F32, BF16]), rng.choice([F32, BF16]),
                            rs.RS_STATE_INT8 if eight else rs.RS_STATE_F32, 64 if eight else 0, 0))
        h = handles(*tensors)
        place = lambda: AT + 4 * rng.randrange(0, 1500)  # noqa: E731
        a = {name: [place() for _ in range(n)] for name in ("params", "grads", "m", "v", "amax_m", "amax_v")}
        written, read, shared = set(), set(), False
        for i, (numel, p, g, state, block, _) in enumerate(tensors):
            s = 1 if state == rs.RS_STATE_INT8 else 4
            blocks = -(-numel // block) if block else 0
            for name, size in (("params", numel * (4 if p == F32 else 2)), ("m", numel * s), ("v", numel * s),
                               ("amax_m", 4 * blocks), ("amax_v", 4 * blocks)):
                got = set(range(a[name][i], a[name][i] + size))
                shared = shared or bool(written & got)
                written |= got
            read |= set(range(a["grads"][i], a["grads"][i] + numel * (4 if g == F32 else 2)))
        shared = shared or bool(written & read)
        assert status(rs.rs_adamw_bind, h, **a, stream=0) == (rs.RS_EINVAL if shared else rs.RS_ESTATE)
        kinds[shared] += 1
    assert min(kinds) > 100, kinds


HP = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01, step=1)


@pytest.mark.parametrize("field,value", [("lr", float("nan")), ("beta1", 1.0), ("beta1", -0.1), ("beta2", 1.0),
                                         ("beta2", float("nan")), ("eps", float("inf")),
                                         ("weight_decay", float("-inf")), ("step", 0)])
def test_hyper_parameters(handles, field, value):
    h = handles(OK, (1000, F32, F32, rs.RS_STATE_F32, 0, 2))
    assert status(rs.rs_adamw_step, h, [HP] * 3, stream=0) == rs.RS_ESTATE
    assert status(rs.rs_adamw_step, h, [HP, HP, {**HP, field: value}], stream=0) == rs.RS_EINVAL


def test_step_norm_and_moments(handles):
    h = handles(OK, (1000, F32, F32, rs.RS_STATE_F32, 0, 2))
    assert status(rs.rs_adamw_step, h, [HP] * 2, stream=0) == rs.RS_EINVAL
    assert status(rs.rs_adamw_step, h, [HP] * 17, stream=0) == rs.RS_EINVAL
    assert status(rs.rs_adamw_step, h, [HP] * 3, grad_scale=AT + 2, stream=0) == rs.RS_EINVAL
    assert status(rs.rs_adamw_step, None, [HP] * 3, stream=0) == rs.RS_EINVAL
    norm = lambda *a: status(rs.rs_adamw_l2norm_clip, h, *a, stream=0)  # noqa: E731
    assert norm(1.0, AT, AT + 8) == norm(0.0, AT) == rs.RS_ESTATE
    for bad in ((1.0, None, AT), (1.0, AT + 4, AT), (1.0, AT, AT + 10), (0.0, AT, AT + 8), (float("inf"), AT, AT + 8),
                (float("nan"), AT, AT + 8), (1.0, AT, AT + 4)):
        assert norm(*bad) == rs.RS_EINVAL, bad
    moments = lambda *a: status(rs.rs_adamw_moments, h, *a, stream=0)  # noqa: E731
    assert moments(AT, AT + 8000, F32) == moments(AT, AT + 4000, BF16) == moments(AT, None, F32) == rs.RS_ESTATE
    for bad in ((AT, AT + 7996, F32), (AT, AT + 3998, BF16), (AT + 2, None, F32), (None, AT + 1, BF16), (AT, None, 2)):
        assert moments(*bad) == rs.RS_EINVAL, bad


def test_tensors_of_the_host_are_refused(handles):
    h = handles(OK)
    x = torch.zeros(1000)
    with pytest.raises(rs.RaggedShardError, match="not on the current device"):
        rs.rs_adamw_bind(h, [x], [x], [x], [x], stream=0)
