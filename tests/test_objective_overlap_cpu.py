"""Overlapping arrays of the objectives are refused on the host, before any
launch: outputs and scratch against each other, against every input and
against the logits and their gradient; arrays in the columns behind a row's
values are apart from it.  No GPU is needed: without one, a call that passes
every check fails at its launch with RS_EHIP."""
import random

import pytest
import torch

import sharded_state_raggedshard_amd as rs

MB = 1 << 20
AT = {name: (i + 1) << 32 for i, name in enumerate((
    "logits", "dlogits", "target", "old_logp", "ref_logp", "advantage", "weight", "logp", "lse", "seq_logp",
    "stats", "start", "topk", "mask", "counts", "mean_prob", "work"))}
ROWS, WIDTH, LD, LDD = 4, 100, 120, 130


def logp(**kw):
    a = dict(logits=AT["logits"], dtype=rs.RS_F32, rows=ROWS, vocab=WIDTH, ld=LD, target=AT["target"],
             logp=AT["logp"], work=AT["work"], nbytes=MB, lse=AT["lse"], stream=0)
    rs.rs_token_logp(**{**a, **kw})


def policy(**kw):
    a = dict(logits=AT["logits"], dtype=rs.RS_F32, rows=ROWS, vocab=WIDTH, ld=LD, target=AT["target"],
             old_logp=AT["old_logp"], ref_logp=AT["ref_logp"], advantage=AT["advantage"], weight=AT["weight"],
             dlogits=AT["dlogits"], ldd=LDD, logp=AT["logp"], stats=AT["stats"], work=AT["work"], nbytes=MB, stream=0)
    rs.rs_policy_loss(**{**a, **kw})


def preference(**kw):
    a = dict(logits=AT["logits"], dtype=rs.RS_F32, rows=ROWS, vocab=WIDTH, ld=LD, target=AT["target"],
             start=AT["start"], n_pairs=2, ref_logp=AT["ref_logp"], weight=AT["weight"], dlogits=AT["dlogits"],
             ldd=LDD, seq_logp=AT["seq_logp"], stats=AT["stats"], work=AT["work"], nbytes=MB, stream=0)
    rs.rs_preference_loss(**{**a, **kw})


def balance(**kw):
    a = dict(logits=AT["logits"], dtype=rs.RS_F32, rows=ROWS, experts=WIDTH, ld=LD, topk=AT["topk"], k=2, ldk=5,
             mask=AT["mask"], start=AT["start"], n_seq=3, dlogits=AT["dlogits"], ldd=LDD, counts=AT["counts"],
             mean_prob=AT["mean_prob"], stats=AT["stats"], work=AT["work"], nbytes=MB, stream=0)
    rs.rs_router_balance(**{**a, **kw})


ROW = 4 * WIDTH
LAST = 4 * ((ROWS - 1) * LD + WIDTH)     # bytes from the first logit to behind the last
LASTD = 4 * ((ROWS - 1) * LDD + WIDTH)
# bytes of each small array, per call
SIZES = {
    logp: dict(target=32, logp=16, lse=16),
    policy: dict(target=32, old_logp=16, ref_logp=16, advantage=16, weight=16, logp=16, stats=16),
    preference: dict(target=32, start=40, ref_logp=16, weight=8, seq_logp=16, stats=12),
    balance: dict(topk=8 * (3 * 5 + 2), mask=4, start=32, counts=1200, mean_prob=1200, stats=8),
}
OUTPUTS = {logp: ("logp", "lse"), policy: ("logp", "stats"), preference: ("seq_logp", "stats"),
           balance: ("counts", "mean_prob", "stats")}


def work_bytes(call):
    return {logp: rs.rs_objective_bytes(ROWS, WIDTH), policy: rs.rs_objective_bytes(ROWS, WIDTH),
            preference: rs.rs_objective_bytes(ROWS, WIDTH, 4),
            balance: rs.rs_router_balance_bytes(ROWS, WIDTH, 3)}[call]


def refused(call, **kw):
    with pytest.raises(rs.RaggedShardError, match="overlaps") as e:
        call(**kw)
    assert e.value.status == rs.RS_EINVAL


def passes_the_checks(call, **kw):
    """The overlaps are the last check: behind it there is no device."""
    with pytest.raises(rs.RaggedShardError) as e:
        call(**kw)
    assert e.value.status == rs.RS_EHIP, e.value


CALLS = [logp, policy, preference, balance]


@pytest.mark.parametrize("call", CALLS)
def test_outputs_against_small_arrays(call):
    for out in OUTPUTS[call]:
        n = SIZES[call][out]
        for name, size in SIZES[call].items():
            if name == out:
                continue
            step = {"target": 8, "start": 8, "topk": 8, "mask": 4}.get(name, 4)
            refused(call, **{out: AT[name]})
            refused(call, **{out: AT[name] + (size - 1) // step * step // 4 * 4})  # its last word
            refused(call, **{out: AT[name] - (n - 4)})                             # the output's own last word


@pytest.mark.parametrize("call", CALLS)
def test_outputs_against_logits_and_gradient(call):
    for out in OUTPUTS[call]:
        n = SIZES[call][out]
        rows = [("logits", LD, LAST)] + ([("dlogits", LDD, LASTD)] if call is not logp else [])
        for name, ld, last in rows:
            for off in (0, ROW - 4, 4 * ld, 4 * ld + ROW - 4, last - 4, -(n - 4), 4 * ld - (n - 4)):
                refused(call, **{out: AT[name] + off})


@pytest.mark.parametrize("call", CALLS)
def test_scratch_against_everything(call):
    n = work_bytes(call)
    for name, size in SIZES[call].items():
        at = (AT[name] + size - 1) & ~15
        refused(call, work=at if at >= AT[name] else AT[name])
        refused(call, work=(AT[name] - n + 16) & ~15)
    refused(call, work=AT["logits"])
    refused(call, work=AT["logits"] - n + 16)
    if call is not logp:
        refused(call, work=AT["dlogits"] + 2 * 4 * LDD)


@pytest.mark.parametrize("call", [policy, preference, balance])
def test_gradient_against_small_arrays(call):
    for name, size in SIZES[call].items():
        if name in OUTPUTS[call]:
            continue
        refused(call, dlogits=AT[name])
        refused(call, dlogits=AT[name] - LASTD + 4)
        refused(call, dlogits=AT[name] - 4 * LDD - ROW + 4)


@pytest.mark.parametrize("call", CALLS)
def test_arrays_that_are_apart_pass(call):
    """Adjacent arrays, and arrays in the columns behind a row's values."""
    if torch.cuda.is_available():
        pytest.skip("the accepted calls would launch")
    passes_the_checks(call)
    for out in OUTPUTS[call]:
        n = SIZES[call][out]
        for name, size in SIZES[call].items():
            if name != out:
                passes_the_checks(call, **{out: AT[name] + (size + 3) // 4 * 4})
                passes_the_checks(call, **{out: AT[name] - n})
        if n <= 4 * (LD - WIDTH):
            passes_the_checks(call, **{out: AT["logits"] + ROW})
            passes_the_checks(call, **{out: AT["logits"] + 4 * 2 * LD + ROW})
            passes_the_checks(call, **{out: AT["logits"] + 4 * LD - n})
        passes_the_checks(call, **{out: AT["logits"] + LAST})
    if call is not logp:
        passes_the_checks(call, dlogits=None)
        passes_the_checks(call, dlogits=None, ldd=1 << 62)
        passes_the_checks(call, dlogits=AT["logits"], ldd=LD)
        passes_the_checks(call, ld=210, ldd=210, dlogits=AT["logits"] + 4 * 105)


def test_random_places_against_a_set_of_words():
    """rs_policy_loss refuses exactly the places that share a 4-byte word."""
    if torch.cuda.is_available():
        pytest.skip("the accepted calls would launch")
    rng = random.Random(3)
    base = AT["logits"] // 4
    kinds = [0, 0]
    for _ in range(3000):
        rows, width = rng.randrange(1, 5), rng.randrange(1, 9)
        ld = width + rng.randrange(0, 9)
        ldd = rng.choice([ld, ld, width + rng.randrange(0, 9)])
        z = {base + t * ld + i for t in range(rows) for i in range(width)}
        d0 = base + rng.randrange(-40, 40)
        d = {d0 + t * ldd + i for t in range(rows) for i in range(width)}
        l0, s0 = base + rng.randrange(-50, 60), base + rng.randrange(-50, 60)
        l, s = set(range(l0, l0 + rows)), set(range(s0, s0 + 4))
        in_place = d0 == base and ld == ldd
        shared = l & s or l & z or s & z or l & d or s & d or (z & d and not in_place)
        # two arrays of different strides, one inside the other's gaps, are refused as well
        unequal = rows > 1 and ld != ldd and min(d) <= max(z) and min(z) <= max(d)
        kw = dict(rows=rows, vocab=width, ld=ld, ldd=ldd, dlogits=4 * d0, logp=4 * l0, stats=4 * s0)
        (refused if shared or unequal else passes_the_checks)(policy, **kw)
        kinds[bool(shared or unequal)] += 1
    assert min(kinds) > 300, kinds
