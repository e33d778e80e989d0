"""Tokens to experts and back: what the entry points refuse, on the host and
before any launch.  Arrays are addresses that nothing reads; without a GPU a
call that passes every check fails at its launch with RS_EHIP."""
import pytest
import torch

import sharded_state_raggedshard_amd as rs

MB = 1 << 20
AT = {name: (i + 1) << 33 for i, name in enumerate((
    "topk", "mask", "start", "count", "slot", "work", "x", "y", "weight", "add", "out", "dy", "dweight"))}
ROWS, HIDDEN, EXPERTS, K, LD, SLOTS = 6, 100, 8, 3, 120, 40


def sort(**kw):
    a = dict(topk=AT["topk"], rows=ROWS, experts=EXPERTS, k=K, ldk=5, mask=AT["mask"], align=4, start=AT["start"],
             count=AT["count"], slot=AT["slot"], work=AT["work"], nbytes=MB, stream=0)
    rs.rs_expert_sort(**{**a, **kw})


def dispatch(**kw):
    a = dict(x=AT["x"], dtype=rs.RS_F32, rows=ROWS, hidden=HIDDEN, ldx=LD, slot=AT["slot"], k=K, weight=AT["weight"], ldw=4,
             experts=EXPERTS, start=AT["start"], count=AT["count"], y=AT["y"], slots=SLOTS, ldy=LD, stream=0)
    rs.rs_expert_dispatch(**{**a, **kw})


def combine(**kw):
    a = dict(y=AT["y"], dtype=rs.RS_F32, slots=SLOTS, hidden=HIDDEN, ldy=LD, slot=AT["slot"], rows=ROWS, k=K, weight=AT["weight"],
             ldw=4, add=AT["add"], lda=LD, out=AT["out"], ldo=LD, stream=0)
    rs.rs_expert_combine(**{**a, **kw})


def gradient(**kw):
    a = dict(dout=AT["x"], dtype=rs.RS_F32, rows=ROWS, hidden=HIDDEN, ldo=LD, y=AT["y"], slots=SLOTS, ldy=LD, slot=AT["slot"], k=K,
             weight=AT["weight"], ldw=4, experts=EXPERTS, start=AT["start"], count=AT["count"], dy=AT["dy"], lddy=LD,
             dweight=AT["dweight"], lddw=7, stream=0)
    rs.rs_expert_combine_grad(**{**a, **kw})


def status(call, **kw):
    with pytest.raises(rs.RaggedShardError) as e:
        call(**kw)
    return e.value.status


def passes(call, **kw):
    if torch.cuda.is_available():
        pytest.skip("the accepted calls would launch")
    assert status(call, **kw) == rs.RS_EHIP


BAD = {
    sort: [dict(topk=None), dict(start=None), dict(count=None), dict(slot=None), dict(work=None), dict(topk=AT["topk"] + 4),
           dict(start=AT["start"] + 4), dict(count=AT["count"] + 2), dict(slot=AT["slot"] + 1), dict(work=AT["work"] + 8),
           dict(rows=-1), dict(experts=0), dict(experts=1025), dict(k=0), dict(k=EXPERTS + 1), dict(ldk=K - 1), dict(align=0),
           dict(align=(1 << 16) + 1)],
    dispatch: [dict(dtype=2), dict(rows=-1), dict(slots=-1), dict(hidden=0), dict(hidden=(1 << 24) + 1), dict(k=0), dict(k=1025),
               dict(ldx=HIDDEN - 1), dict(ldy=HIDDEN - 1), dict(ldw=K - 1), dict(x=None), dict(y=None), dict(slot=None),
               dict(start=None), dict(count=None), dict(experts=0), dict(experts=1025), dict(x=AT["x"] + 2), dict(y=AT["y"] + 1),
               dict(slot=AT["slot"] + 2), dict(weight=AT["weight"] + 2), dict(start=AT["start"] + 4), dict(count=AT["count"] + 2)],
    combine: [dict(dtype=-1), dict(rows=-1), dict(slots=-1), dict(hidden=0), dict(k=0), dict(ldy=HIDDEN - 1), dict(lda=HIDDEN - 1),
              dict(ldo=HIDDEN - 1), dict(ldw=K - 1), dict(y=None), dict(out=None), dict(slot=None), dict(add=AT["add"] + 2),
              dict(out=AT["out"] + 2), dict(dtype=rs.RS_BF16, add=AT["add"] + 1)],
    gradient: [dict(dtype=5), dict(rows=-1), dict(slots=-1), dict(hidden=0), dict(k=0), dict(ldo=HIDDEN - 1), dict(ldy=HIDDEN - 1),
               dict(lddy=HIDDEN - 1), dict(lddw=K - 1), dict(ldw=K - 1), dict(dout=None), dict(y=None), dict(slot=None),
               dict(dweight=None), dict(start=None), dict(count=None), dict(experts=0), dict(dweight=AT["dweight"] + 2),
               dict(dy=AT["dy"] + 2)],
}


@pytest.mark.parametrize("call,kw", [(c, kw) for c, many in BAD.items() for kw in many])
def test_bad_arguments(call, kw):
    assert status(call, **kw) == rs.RS_EINVAL


@pytest.mark.parametrize("call,kw", [
    (sort, dict(rows=1 << 30)), (sort, dict(rows=715_800_000, k=3, align=1 << 16)), (sort, dict(ldk=1 << 49)),
    (dispatch, dict(rows=1 << 30)), (dispatch, dict(slots=1 << 31)), (dispatch, dict(ldx=1 << 49)), (dispatch, dict(ldy=1 << 48)),
    (combine, dict(rows=1 << 30)), (combine, dict(lda=1 << 49)), (gradient, dict(lddy=1 << 48))])
def test_sizes_beyond_the_tables(call, kw):
    assert status(call, **kw) == rs.RS_EOVERFLOW


def test_scratch_and_slots():
    n = rs.rs_expert_sort_bytes(ROWS, EXPERTS, K)
    assert status(sort, nbytes=n - 1) == rs.RS_ENOMEM
    passes(sort, nbytes=n)
    last = 0
    for rows in (0, 1, 100, 3000, 20_000, 100_000, 1 << 27):
        got = rs.rs_expert_sort_bytes(rows, 256, 8)
        assert got >= last and got > 0
        last = got
    assert rs.rs_expert_slots(6, 8, 3, 4) == 18 + 8 * 3
    assert rs.rs_expert_slots(1, 256, 2, 128) == 2 + 2 * 127
    assert rs.rs_expert_slots(0, 256, 2, 128) == 0
    for bad in ((-1, 8, 2, 1), (6, 0, 1, 1), (6, 1025, 1, 1), (6, 8, 9, 1), (6, 8, 2, 0), (1 << 30, 8, 2, 1)):
        with pytest.raises(rs.RaggedShardError):
            rs.rs_expert_slots(*bad)
    for bad in ((-1, 8, 2), (6, 0, 1), (6, 1025, 1), (6, 8, 9), (1 << 31, 8, 2)):
        with pytest.raises(rs.RaggedShardError):
            rs.rs_expert_sort_bytes(*bad)


@pytest.mark.parametrize("call", [sort, dispatch, combine, gradient])
def test_arrays_that_are_apart_pass(call):
    passes(call)


@pytest.mark.parametrize("call,kw", [
    (sort, dict(mask=None)), (sort, dict(rows=0, topk=None, slot=None)),
    (dispatch, dict(weight=None, ldw=0)), (dispatch, dict(start=None, count=None, experts=0)), (dispatch, dict(rows=0, x=None, slot=None)),
    (combine, dict(weight=None, ldw=0)), (combine, dict(add=None, lda=0)), (combine, dict(out=AT["add"])),
    (combine, dict(out=AT["y"] + 4 * HIDDEN, ldy=240, ldo=240, lda=240)), (combine, dict(slots=0, y=None)),
    (gradient, dict(dy=None, lddy=0)), (gradient, dict(dy=AT["y"])), (gradient, dict(dweight=AT["x"] + 4 * HIDDEN, lddw=LD)),
    (gradient, dict(weight=None, ldw=0, start=None, count=None))])
def test_what_is_allowed_passes(call, kw):
    passes(call, **kw)


SPAN = {"topk": 8 * (5 * 5 + 3), "mask": 6, "start": 72, "count": 32, "slot": 72, "work": 256, "x": 4 * (5 * LD + 100),
        "y": 4 * (39 * LD + 100), "weight": 4 * (5 * 4 + 3), "add": 4 * (5 * LD + 100), "out": 4 * (5 * LD + 100),
        "dy": 4 * (39 * LD + 100), "dweight": 4 * (5 * 7 + 3)}
WRITES = {sort: ["start", "count", "slot", "work"], dispatch: ["y"], combine: ["out"], gradient: ["dy", "dweight"]}
TAKES = {sort: ["topk", "mask"], dispatch: ["x", "slot", "weight", "start", "count"], combine: ["y", "slot", "weight", "add"],
         gradient: ["x", "y", "slot", "weight", "start", "count"]}


@pytest.mark.parametrize("call", [sort, dispatch, combine, gradient])
def test_overlaps_are_refused(call):
    key = lambda name: "dout" if call is gradient and name == "x" else name  # noqa: E731
    for out in WRITES[call]:
        for other in WRITES[call] + TAKES[call]:
            if other == out:
                continue
            step = 16 if out == "work" else 8
            for at in (AT[other], AT[other] - SPAN[out] + step, AT[other] + (SPAN[other] - 1) // step * step):
                if at % step == 0 and not (call is combine and at == AT["add"]) and not (call is gradient and out == "dy" and at == AT["y"]):
                    assert status(call, **{key(out): at}) == rs.RS_EINVAL, (out, other, at - AT[other])
    # in place only with the same stride
    if call is combine:
        assert status(call, out=AT["add"], ldo=LD + 1) == rs.RS_EINVAL
    if call is gradient:
        assert status(call, dy=AT["y"], lddy=LD + 1) == rs.RS_EINVAL


def test_tensors_of_the_host_are_refused():
    with pytest.raises(rs.RaggedShardError, match="not on the current device"):
        combine(y=torch.zeros(40, 120))
