"""Refusals of the training objectives: every argument check answers with
its status on the host, before any launch (no GPU is needed)."""
import ctypes as C

import pytest

import sharded_state_raggedshard_amd as rs

P = 1 << 20      # a device address that nothing may touch
WORK = 1 << 30


def _expect(status, f, **kw):
    with pytest.raises(rs.RaggedShardError) as e:
        f(**kw)
    assert e.value.status == status, e.value


def _logp(**kw):
    a = dict(logits=P, dtype=rs.RS_BF16, rows=4, vocab=100, ld=100, target=P, logp=P, work=P,
             nbytes=WORK, lse=None, temperature=1.0, stream=0)
    a.update(kw)
    rs.rs_token_logp(**a)


def _policy(**kw):
    a = dict(logits=P, dtype=rs.RS_F32, rows=4, vocab=100, ld=100, target=P, old_logp=P, ref_logp=P,
             advantage=P, weight=P, dlogits=P + (1 << 16), ldd=100, logp=None, stats=P, work=P,
             nbytes=WORK, stream=0)
    a.update(kw)
    rs.rs_policy_loss(**a)


def _pref(**kw):
    a = dict(logits=P, dtype=rs.RS_F32, rows=4, vocab=100, ld=100, target=P, start=P, n_pairs=2,
             ref_logp=P, weight=P, dlogits=P + (1 << 16), ldd=100, seq_logp=P, stats=P, work=P,
             nbytes=WORK, stream=0)
    a.update(kw)
    rs.rs_preference_loss(**a)


@pytest.mark.parametrize("call", [_logp, _policy, _pref])
def test_logits_arguments_are_checked(call):
    _expect(rs.RS_EINVAL, call, dtype=7)
    _expect(rs.RS_EINVAL, call, rows=-1)
    _expect(rs.RS_EINVAL, call, vocab=0)
    _expect(rs.RS_EINVAL, call, vocab=(1 << 24) + 1, ld=1 << 25)
    _expect(rs.RS_EINVAL, call, ld=99)
    _expect(rs.RS_EINVAL, call, ld=-5)
    _expect(rs.RS_EOVERFLOW, call, rows=1 << 40, ld=1 << 20)
    _expect(rs.RS_EOVERFLOW, call, rows=(1 << 62), ld=1 << 62)
    _expect(rs.RS_EINVAL, call, logits=None)
    _expect(rs.RS_EINVAL, call, logits=P + 1)
    _expect(rs.RS_EINVAL, call, target=None)
    _expect(rs.RS_EINVAL, call, target=P + 4)
    _expect(rs.RS_EINVAL, call, work=None)
    _expect(rs.RS_EINVAL, call, work=P + 8)
    _expect(rs.RS_ENOMEM, call, nbytes=16)
    for t in (0.0, -1.0, float("nan"), float("inf"), 1e-12, 1e12):
        _expect(rs.RS_EINVAL, call, temperature=t)


def test_token_logp_outputs_are_checked():
    _expect(rs.RS_EINVAL, _logp, logp=None)
    _expect(rs.RS_EINVAL, _logp, logp=P + 2)
    _expect(rs.RS_EINVAL, _logp, lse=P + 2)


@pytest.mark.parametrize("call", [_policy, _pref])
def test_gradient_arguments_are_checked(call):
    _expect(rs.RS_EINVAL, call, stats=None)
    _expect(rs.RS_EINVAL, call, stats=P + 1)
    _expect(rs.RS_EINVAL, call, ldd=99)
    _expect(rs.RS_EINVAL, call, dlogits=P + (1 << 16) + 2)
    _expect(rs.RS_EOVERFLOW, call, rows=1 << 20, ldd=1 << 40, dlogits=1 << 50)
    # overlaps: shifted, the last row's last value, another stride
    _expect(rs.RS_EINVAL, call, dlogits=P + 4)
    _expect(rs.RS_EINVAL, call, dlogits=P + 4 * (4 * 100 - 1))
    _expect(rs.RS_EINVAL, call, dlogits=P, ldd=101)
    _expect(rs.RS_EINVAL, call, ld=210, ldd=210, dlogits=P + 4 * 111)
    _expect(rs.RS_EINVAL, call, ld=210, ldd=210, dlogits=P - 4 * 111)
    # the same places are left to the next check when they do not overlap
    for ok in (dict(dlogits=P), dict(dlogits=None), dict(dlogits=P + 1600),
               dict(ld=210, ldd=210, dlogits=P + 4 * 100),
               dict(ld=210, ldd=210, dlogits=P + 4 * 110),
               dict(ld=210, ldd=210, dlogits=P - 4 * 110)):
        _expect(rs.RS_EINVAL, call, weight=P + 1, **ok)
        with pytest.raises(rs.RaggedShardError, match="misaligned"):
            call(weight=P + 1, **ok)


def test_policy_arguments_are_checked():
    for name in ("old_logp", "advantage", "weight"):
        _expect(rs.RS_EINVAL, _policy, **{name: None})
        _expect(rs.RS_EINVAL, _policy, **{name: P + 2})
    _expect(rs.RS_EINVAL, _policy, ref_logp=None, kl_coef=0.1)
    _expect(rs.RS_EINVAL, _policy, ref_logp=P + 1)
    _expect(rs.RS_EINVAL, _policy, logp=P + 1)
    for kw in (dict(clip_low=-0.1), dict(clip_low=1.5), dict(clip_high=-0.1), dict(kl_coef=-1.0),
               dict(clip_low=float("nan")), dict(clip_high=float("inf")), dict(kl_coef=float("nan"))):
        _expect(rs.RS_EINVAL, _policy, **kw)
    assert rs.lib().rs_policy_loss(P, 0, 4, 100, 100, P, P, P, P, P, None, None, 100, None, P, P,
                                   C.c_size_t(WORK), None) == rs.RS_EINVAL


def test_preference_arguments_are_checked():
    _expect(rs.RS_EINVAL, _pref, start=None)
    _expect(rs.RS_EINVAL, _pref, start=P + 4)
    _expect(rs.RS_EINVAL, _pref, n_pairs=0)
    _expect(rs.RS_EINVAL, _pref, n_pairs=(1 << 23) + 1)
    for name in ("ref_logp", "weight", "seq_logp"):
        _expect(rs.RS_EINVAL, _pref, **{name: P + 1})
    for kw in (dict(beta=0.0), dict(beta=float("inf")), dict(label_smoothing=0.5),
               dict(label_smoothing=-0.1), dict(margin=float("nan")), dict(kind=3),
               dict(kind=rs.RS_PREF_IPO, margin=0.1), dict(kind=rs.RS_PREF_IPO, label_smoothing=0.1),
               dict(kind=rs.RS_PREF_HINGE, label_smoothing=0.1)):
        _expect(rs.RS_EINVAL, _pref, **kw)


def test_outputs_that_overlap_other_arrays_are_refused():
    def refused(call, **kw):
        with pytest.raises(rs.RaggedShardError, match="overlaps another array") as e:
            call(**kw)
        assert e.value.status == rs.RS_EINVAL

    far = [P + (i << 20) for i in range(1, 8)]
    refused(_logp, logp=far[0], lse=far[0])
    refused(_logp, logp=far[0], lse=far[0] + 4 * 3)  # the last of four rows
    policy = dict(old_logp=far[0], ref_logp=far[1], advantage=far[2], weight=far[3], logp=far[4],
                  stats=far[5])
    for name in ("old_logp", "ref_logp", "advantage", "weight"):
        for out in ("logp", "stats"):
            refused(_policy, **{**policy, out: policy[name]})
            refused(_policy, **{**policy, out: policy[name] + 4 * 3})
            refused(_policy, **{**policy, out: policy[name] - 4 * 3})
    refused(_policy, **{**policy, "stats": policy["logp"]})
    pref = dict(ref_logp=far[0], weight=far[1], seq_logp=far[2], stats=far[3])
    for name, n in (("ref_logp", 4), ("weight", 2)):
        for out in ("seq_logp", "stats"):
            refused(_pref, **{**pref, out: pref[name]})
            refused(_pref, **{**pref, out: pref[name] + 4 * (n - 1)})
    refused(_pref, **{**pref, "stats": pref["seq_logp"]})


def test_scratch_sizes():
    assert rs.rs_objective_bytes(0, 1, 0) > 0
    a, b = rs.rs_objective_bytes(1000, 32000), rs.rs_objective_bytes(1000, 32000, 8)
    assert 8 * 1000 <= a < b < 1 << 20
    for bad in ((-1, 10, 0), (10, 0, 0), (10, (1 << 24) + 1, 0), (1 << 60, 8, 0), (10, 10, -2)):
        with pytest.raises(rs.RaggedShardError):
            rs.rs_objective_bytes(*bad)


def _balance(**kw):
    a = dict(logits=P, dtype=rs.RS_F32, rows=4, experts=100, ld=100, topk=P, k=2, ldk=2, mask=P,
             start=P, n_seq=3, dlogits=P + (1 << 16), ldd=100, counts=P, mean_prob=P, stats=P, work=P,
             nbytes=WORK, stream=0)
    a.update(kw)
    rs.rs_router_balance(**a)


def test_router_balance_arguments_are_checked():
    for name in ("logits", "topk", "counts", "mean_prob", "stats", "work", "start"):
        _expect(rs.RS_EINVAL, _balance, **{name: None})
    for name in ("logits", "topk", "counts", "mean_prob", "stats", "work", "start", "dlogits"):
        _expect(rs.RS_EINVAL, _balance, **{name: P + (1 << 16) + 1})
    for kw in (dict(dtype=2), dict(rows=-1), dict(experts=0, ld=100), dict(experts=1025, ld=2000, ldd=2000),
               dict(ld=99), dict(ldd=99), dict(k=0), dict(k=101, ldk=101), dict(ldk=1), dict(n_seq=0),
               dict(n_seq=(1 << 16) + 1), dict(balance_coef=float("nan")), dict(balance_coef=-1.0),
               dict(z_coef=float("inf")), dict(z_coef=-1.0), dict(score=2),
               dict(score=rs.RS_SCORE_SIGMOID, z_coef=0.1), dict(dlogits=P + 4), dict(dlogits=P, ldd=101)):
        _expect(rs.RS_EINVAL, _balance, **kw)
    _expect(rs.RS_EOVERFLOW, _balance, rows=1 << 30, k=4, ldk=4, dlogits=None)
    _expect(rs.RS_EOVERFLOW, _balance, rows=1 << 44, dlogits=None)
    _expect(rs.RS_EOVERFLOW, _balance, ldk=1 << 50, dlogits=None)
    _expect(rs.RS_ENOMEM, _balance, nbytes=255)
    hp = rs.rs_balance_hparams(0.1, 0.0, 0, 1)
    assert rs.lib().rs_router_balance(P, 0, 4, 100, 100, P, 2, 2, P, P, 3, C.byref(hp), None, 100, P, P, P,
                                      P, C.c_size_t(WORK), None) == rs.RS_EINVAL
    assert rs.rs_router_balance_bytes(0, 1, 1) > 0
    for bad in ((-1, 8, 1), (1, 0, 1), (1, 1025, 1), (1, 8, 0), (1, 8, 1 << 17)):
        with pytest.raises(rs.RaggedShardError):
            rs.rs_router_balance_bytes(*bad)
