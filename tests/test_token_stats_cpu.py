"""Token statistics: what the entry points refuse, on the host and before any
launch.  Without a GPU a call that passes every check fails at its launch."""
import pytest
import torch

import sharded_state_raggedshard_amd as rs

MB = 1 << 20
AT = {name: (i + 1) << 32 for i, name in enumerate((
    "logits", "target", "logp", "entropy", "top_id", "top_logp", "saved", "work", "dlogp", "dentropy", "dlogits"))}
ROWS, VOCAB, LD, TOP = 4, 100, 120, 3


def stats(**kw):
    a = dict(logits=AT["logits"], dtype=rs.RS_F32, rows=ROWS, vocab=VOCAB, ld=LD, target=AT["target"], logp=AT["logp"],
             entropy=AT["entropy"], top=TOP, top_id=AT["top_id"], top_logp=AT["top_logp"], saved=AT["saved"], work=AT["work"],
             nbytes=MB, stream=0)
    rs.rs_token_stats(**{**a, **kw})


def gradient(**kw):
    a = dict(logits=AT["logits"], dtype=rs.RS_F32, rows=ROWS, vocab=VOCAB, ld=LD, target=AT["target"], saved=AT["saved"],
             dlogp=AT["dlogp"], dentropy=AT["dentropy"], dlogits=AT["dlogits"], ldd=LD + 4, stream=0)
    rs.rs_token_stats_grad(**{**a, **kw})


def status(call, **kw):
    with pytest.raises(rs.RaggedShardError) as e:
        call(**kw)
    return e.value.status


def passes(call, **kw):
    if torch.cuda.is_available():
        pytest.skip("the accepted calls would launch")
    assert status(call, **kw) == rs.RS_EHIP


COMMON = [dict(dtype=2), dict(rows=-1), dict(vocab=0), dict(vocab=(1 << 24) + 1, ld=1 << 25), dict(ld=VOCAB - 1), dict(logits=None),
          dict(logits=AT["logits"] + 2), dict(dtype=rs.RS_BF16, logits=AT["logits"] + 1), dict(target=AT["target"] + 4),
          dict(temperature=0.0), dict(temperature=float("nan")), dict(temperature=2.0 ** 21), dict(temperature=-1.0)]


@pytest.mark.parametrize("kw", COMMON + [
    dict(top=-1), dict(top=33), dict(top_id=None), dict(top_logp=None), dict(work=None), dict(work=AT["work"] + 8),
    dict(target=None), dict(logp=AT["logp"] + 2), dict(entropy=AT["entropy"] + 1), dict(top_id=AT["top_id"] + 4),
    dict(top_logp=AT["top_logp"] + 2), dict(saved=AT["saved"] + 2)])
def test_bad_arguments_of_the_statistics(kw):
    assert status(stats, **kw) == rs.RS_EINVAL


@pytest.mark.parametrize("kw", COMMON + [
    dict(saved=None), dict(dlogits=None), dict(target=None), dict(saved=AT["saved"] + 2), dict(dlogp=AT["dlogp"] + 2),
    dict(dentropy=AT["dentropy"] + 2), dict(dlogits=AT["dlogits"] + 2), dict(ldd=VOCAB - 1)])
def test_bad_arguments_of_the_gradient(kw):
    assert status(gradient, **kw) == rs.RS_EINVAL


def test_sizes():
    assert status(stats, rows=1 << 44) == status(gradient, rows=1 << 44) == rs.RS_EOVERFLOW
    assert status(gradient, ldd=1 << 49) == rs.RS_EOVERFLOW
    n = rs.rs_token_stats_bytes(ROWS, VOCAB, TOP)
    assert status(stats, nbytes=n - 1) == rs.RS_ENOMEM
    passes(stats, nbytes=n)
    for bad in ((-1, 10, 1), (1, 0, 1), (1, (1 << 24) + 1, 1), (1, 10, 33), (1, 10, -1), (1 << 45, 1 << 10, 0)):
        with pytest.raises(rs.RaggedShardError):
            rs.rs_token_stats_bytes(*bad)
    last = 0
    for rows, vocab, top in ((0, 1, 0), (1, 10, 0), (1, 1 << 20, 8), (16, 1 << 20, 20), (513, 1 << 20, 20), (10_000, 1 << 20, 32)):
        got = rs.rs_token_stats_bytes(rows, vocab, top)
        assert got >= last > -1 and got > 0
        last = got


@pytest.mark.parametrize("call,kw", [
    (stats, {}), (gradient, {}), (stats, dict(target=None, logp=None)), (stats, dict(logp=None, entropy=None, saved=None)),
    (stats, dict(top=0, top_id=None, top_logp=None)),
    (gradient, dict(dlogp=None)), (gradient, dict(dentropy=None)), (gradient, dict(target=None, dlogp=None)),
    (gradient, dict(dlogits=AT["logits"], ldd=LD)), (stats, dict(logp=AT["logits"] + 4 * VOCAB)),
    (stats, dict(entropy=AT["logp"] + 4 * ROWS))])
def test_what_is_allowed_passes(call, kw):
    passes(call, **kw)


def test_no_rows():
    stats(rows=0, logits=None, target=None, logp=None, entropy=None, top_id=None, top_logp=None, saved=None)
    gradient(rows=0, logits=None, target=None, saved=None, dlogp=None, dentropy=None, dlogits=None)


SPAN = {"logits": 4 * (3 * LD + VOCAB), "target": 32, "logp": 16, "entropy": 16, "top_id": 96, "top_logp": 48, "saved": 64,
        "work": 256, "dlogp": 16, "dentropy": 16, "dlogits": 4 * (3 * (LD + 4) + VOCAB)}


def test_overlaps_are_refused():
    outs = ["logp", "entropy", "top_id", "top_logp", "saved", "work"]
    for out in outs:
        for other in outs + ["logits", "target"]:
            if out != other:
                step = 16 if out == "work" else 8
                for at in (AT[other], AT[other] - SPAN[out] + step, AT[other] + (SPAN[other] - 1) // step * step):
                    assert status(stats, **{out: at}) == rs.RS_EINVAL, (out, other)
    for other in ("target", "saved", "dlogp", "dentropy"):
        assert status(gradient, dlogits=AT[other]) == rs.RS_EINVAL
        assert status(gradient, dlogits=AT[other] - SPAN["dlogits"] + 4) == rs.RS_EINVAL
    assert status(gradient, dlogits=AT["logits"]) == rs.RS_EINVAL  # another stride
    assert status(gradient, dlogits=AT["logits"] + 4, ldd=LD) == rs.RS_EINVAL


def test_tensors_of_the_host_are_refused():
    with pytest.raises(rs.RaggedShardError, match="not on the current device"):
        stats(logits=torch.zeros(4, 120))
