"""Post-training operators without a GPU: structure layouts, refusals before any work, and the oracle itself."""
import ctypes
import math

import numpy as np
import pytest
import torch

import oracle.post_training_oracle as ref_ops
from linear_cross_entropy_tiled_gb300 import (
    AdamW, _lib, adamw_plan, policy_loss, policy_loss_and_grad, preference_loss_and_grad)

FAKE = 1 << 20   # an aligned address that is never read: every call below is refused first
OK, INVALID, ALIGNMENT, WORKSPACE = 0, 1, 3, 4


@pytest.fixture(scope="module", autouse=True)
def lib():
    import os
    if not os.path.exists(_lib.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return _lib.load()


def test_structures_have_the_c_layout():
    assert ctypes.sizeof(_lib.FlceTokens) == 64
    assert ctypes.sizeof(_lib.FlcePolicyArgs) == _lib.POLICY_ARGS.size == 248
    assert ctypes.sizeof(_lib.FlcePreferenceArgs) == _lib.PREFERENCE_ARGS.size == 192
    assert ctypes.sizeof(_lib.FlceAdamWTensor) == 64
    assert ctypes.sizeof(_lib.FlceAdamWArgs) == 88


def test_packed_bytes_are_the_structure():
    """struct.pack puts every argument where the ctypes mirror has it."""
    a = _lib.FlcePolicyArgs.from_buffer_copy(_lib.POLICY_ARGS.pack(*range(1, 10), *range(10, 20), 20,
                                                                   *range(21, 26), .5, .25, 3., .1,
                                                                   *range(30, 36)))
    assert (a.tokens.sequences, a.tokens.ignore_index, a.tokens.mask_kind) == (1, 7, 9)
    assert (a.log_probs, a.workspace, a.ws_bytes, a.ld_log_probs, a.ld_grad) == (10, 19, 20, 21, 25)
    assert (a.clip_low, a.kl_coef, a.dtype, a.negated, a.reserved) == (.5, .1, 30, 34, 35)
    b = _lib.FlcePreferenceArgs.from_buffer_copy(_lib.PREFERENCE_ARGS.pack(
        *range(1, 10), *range(10, 17), 17, 18, 19, 20, .1, .2, .3, 21, 22, 23, 24))
    assert (b.log_probs, b.workspace, b.ws_bytes, b.ld_grad) == (10, 16, 17, 20)
    assert (b.beta, b.margin, b.dtype, b.average, b.negated) == (.1, .3, 21, 23, 24)


def policy_args(**kw):
    a = _lib.FlcePolicyArgs()
    t = a.tokens
    t.sequences, t.cols = 4, 100
    for k in ("log_probs", "old_log_probs", "ref_log_probs", "advantages", "loss", "grad", "num_tokens",
              "num_clipped", "kl_sum", "workspace"):
        setattr(a, k, FAKE)
    a.ws_bytes = 1 << 30
    for k in ("ld_log_probs", "ld_old", "ld_ref", "ld_advantages", "ld_grad"):
        setattr(a, k, 100)
    a.clip_low, a.clip_high, a.kl_coef = 0.2, 0.2, 0.1
    for k, v in kw.items():
        setattr(t if hasattr(t, k) else a, k, v)
    return a


@pytest.mark.parametrize("bad,code", [
    (dict(dtype=3), INVALID), (dict(dtype=-1), INVALID), (dict(reduction=2), INVALID),
    (dict(kl_estimator=3), INVALID), (dict(clip_low=1.0), INVALID), (dict(clip_low=-0.1), INVALID),
    (dict(clip_high=math.inf), INVALID), (dict(clip_high=math.nan), INVALID),
    (dict(dual_clip=1.0), INVALID), (dict(dual_clip=-3.0), INVALID), (dict(kl_coef=math.nan), INVALID),
    (dict(advantage_per_token=2), INVALID), (dict(negated=2), INVALID), (dict(reserved=1), INVALID),
    (dict(sequences=-1), INVALID), (dict(cols=-1), INVALID), (dict(cols=1 << 31), INVALID),
    (dict(sequences=1 << 20, cols=1 << 20), INVALID), (dict(packed=2), INVALID),
    (dict(packed=1), INVALID),                                     # no cu_seqlens
    (dict(cu_seqlens=FAKE), INVALID),                              # cu_seqlens without packed
    (dict(packed=1, cu_seqlens=FAKE + 2), ALIGNMENT),
    (dict(packed=1, cu_seqlens=FAKE, tokens=1 << 31), INVALID),
    (dict(mask=FAKE), INVALID), (dict(mask_kind=3), INVALID), (dict(mask_kind=1), INVALID),
    (dict(mask_kind=2, mask=FAKE + 4, ld_mask=100), ALIGNMENT),
    (dict(mask_kind=1, mask=FAKE, ld_mask=99), INVALID),
    (dict(log_probs=0), INVALID), (dict(log_probs=FAKE + 2), ALIGNMENT),
    (dict(log_probs=FAKE + 1, dtype=1), ALIGNMENT), (dict(ld_log_probs=99), INVALID),
    (dict(ld_old=99), INVALID), (dict(ref_log_probs=0), INVALID), (dict(ld_grad=50), INVALID),
    (dict(grad=FAKE + 2), ALIGNMENT), (dict(advantages=0), INVALID), (dict(advantages=FAKE + 2), ALIGNMENT),
    (dict(advantage_per_token=1, ld_advantages=9), INVALID), (dict(loss=0), INVALID),
    (dict(loss=FAKE + 1), ALIGNMENT), (dict(num_tokens=FAKE + 4), ALIGNMENT),
    (dict(cols=10000, ld_log_probs=10000, ld_old=10000, ld_ref=10000, ld_grad=10000, ws_bytes=100), WORKSPACE),
    (dict(cols=10000, ld_log_probs=10000, ld_old=10000, ld_ref=10000, ld_grad=10000, workspace=0), WORKSPACE),
    (dict(cols=10000, ld_log_probs=10000, ld_old=10000, ld_ref=10000, ld_grad=10000, workspace=FAKE + 8),
     ALIGNMENT),
])
def test_policy_loss_refuses(lib, bad, code):
    a = policy_args(**bad)
    assert _lib.policy_loss_raw(a, 0) == code, _lib.last_error_detail()


def test_policy_workspace_bounds(lib):
    """None for small batches, and never more than the stated bound."""
    g = np.random.default_rng(3)
    assert _lib.policy_workspace_bytes(policy_args()) == 0
    for _ in range(300):
        S, T = int(10 ** g.uniform(0, 5)), int(10 ** g.uniform(0, 4))
        kind = int(g.integers(0, 3))
        a = policy_args(sequences=S, cols=T, reduction=int(g.choice([0, 1, 3])), mask_kind=kind,
                        mask=FAKE if kind else 0, ld_mask=T + int(g.integers(0, 3)),
                        ld_log_probs=T + int(g.integers(0, 2)), ld_old=T, ld_ref=T, ld_grad=T)
        n = _lib.policy_workspace_bytes(a)
        assert n <= 49152 + 8 * S
        if S * T <= 8192 and S <= 1024:
            assert n == 0
    assert _lib.load().flce_policy_workspace_bytes(None, None) == INVALID


def preference_args(**kw):
    a = _lib.FlcePreferenceArgs()
    a.tokens.sequences, a.tokens.cols = 4, 100
    for k in ("log_probs", "ref_log_probs", "loss", "grad", "chosen_rewards", "rejected_rewards",
              "workspace"):
        setattr(a, k, FAKE)
    a.ws_bytes, a.ld_log_probs, a.ld_ref, a.ld_grad, a.beta = 1 << 30, 100, 100, 100, 0.1
    for k, v in kw.items():
        setattr(a.tokens if hasattr(a.tokens, k) else a, k, v)
    return a


@pytest.mark.parametrize("bad,code", [
    (dict(sequences=5), INVALID), (dict(dtype=3), INVALID), (dict(loss_type=3), INVALID),
    (dict(beta=0.0), INVALID), (dict(beta=-1.0), INVALID), (dict(beta=math.inf), INVALID),
    (dict(margin=math.nan), INVALID), (dict(label_smoothing=0.6), INVALID),
    (dict(label_smoothing=-0.1), INVALID), (dict(average=2), INVALID), (dict(negated=-1), INVALID),
    (dict(log_probs=0), INVALID), (dict(ref_log_probs=FAKE + 2), ALIGNMENT), (dict(ld_ref=1), INVALID),
    (dict(loss=0), INVALID), (dict(chosen_rewards=FAKE + 2), ALIGNMENT),
    (dict(sequences=200, cols=1, ws_bytes=0), WORKSPACE),
])
def test_preference_loss_refuses(lib, bad, code):
    assert _lib.preference_loss_raw(preference_args(**bad), 0) == code, _lib.last_error_detail()


def test_preference_workspace_bounds(lib):
    assert _lib.preference_workspace_bytes(preference_args()) == 0
    for S, T in ((128, 64), (130, 1), (2, 40000), (1 << 20, 8)):
        n = _lib.preference_workspace_bytes(preference_args(sequences=S, cols=T))
        assert n <= 256 + 4 * (S // 2) and (n == 0) == (S <= 128 and S * T <= 65536)


def adamw_args(entries, **kw):
    table = (_lib.FlceAdamWTensor * max(1, len(entries)))()
    for e, given in zip(table, entries):
        for k in ("param", "grad", "exp_avg", "exp_avg_sq"):
            setattr(e, k, FAKE)
        e.numel = 1000
        for k, v in given.items():
            setattr(e, k, v)
    a = _lib.FlceAdamWArgs()
    a.tensors, a.count, a.step = ctypes.addressof(table), len(entries), 1
    a.lr, a.beta1, a.beta2, a.eps, a.weight_decay, a.state_bits = 1e-3, 0.9, 0.999, 1e-8, 0.01, 32
    for k, v in kw.items():
        setattr(a, k, v)
    return a, table


@pytest.mark.parametrize("entries,kw,code", [
    ([{}], dict(count=-1), INVALID), ([{}], dict(tensors=0), INVALID), ([{}], dict(step=0), INVALID),
    ([{}], dict(lr=-1.0), INVALID), ([{}], dict(lr=math.nan), INVALID), ([{}], dict(eps=-1.0), INVALID),
    ([{}], dict(weight_decay=math.inf), INVALID), ([{}], dict(beta1=1.0), INVALID),
    ([{}], dict(beta2=-0.1), INVALID), ([{}], dict(dtype=5), INVALID),
    ([{}], dict(dtype=1, grad_dtype=2), INVALID), ([{}], dict(grad_dtype=1), INVALID),
    ([{}], dict(state_bits=16), INVALID), ([{}], dict(grad_scale=FAKE + 2), ALIGNMENT),
    ([dict(numel=-1)], {}, INVALID), ([dict(numel=1 << 39)], {}, INVALID), ([dict(param=0)], {}, INVALID),
    ([dict(grad=0)], {}, INVALID), ([dict(exp_avg=0)], {}, INVALID), ([dict(exp_avg_sq=0)], {}, INVALID),
    ([{}], dict(state_bits=8), INVALID),                                       # no scales
    ([dict(exp_avg_scale=FAKE)], {}, INVALID),                                 # scales with 32 bits
    ([dict(master=FAKE)], {}, INVALID),                                        # master of fp32
    ([dict(master=FAKE), {}], dict(dtype=1, grad_dtype=1), INVALID),           # one master of two
    ([dict(param=FAKE + 2)], {}, ALIGNMENT), ([dict(exp_avg=FAKE + 1)], {}, ALIGNMENT),
    ([dict(param=FAKE + 1)], dict(dtype=1, grad_dtype=1), ALIGNMENT),
    ([], {}, OK),                                                              # nothing to do
])
def test_adamw_refuses(lib, entries, kw, code):
    a, keep = adamw_args(entries, **kw)
    assert _lib.adamw_raw(a, 0) == code, _lib.last_error_detail()


def test_an_empty_tensor_has_no_say_in_the_master_copies(lib):
    """A tensor of no elements has address 0 for everything; the others' masters are still accepted,
    so that it is the next check, the alignment, that refuses."""
    a, keep = adamw_args([dict(numel=0, param=0, grad=0, exp_avg=0, exp_avg_sq=0),
                          dict(master=FAKE, param=FAKE + 1)], dtype=1, grad_dtype=1)
    assert _lib.adamw_raw(a, 0) == ALIGNMENT


def test_null_arguments(lib):
    assert lib.flce_policy_loss(None, None) == INVALID
    assert lib.flce_preference_loss(None, None) == INVALID
    assert lib.flce_adamw(None, None) == INVALID


def test_python_refuses_cpu_tensors():
    x = torch.zeros(2, 3)
    with pytest.raises(ValueError, match="no CPU path"):
        policy_loss_and_grad(x, x, torch.ones(2))
    with pytest.raises(ValueError, match="no CPU path"):
        policy_loss(x.requires_grad_(True), x, torch.ones(2))
    with pytest.raises(ValueError, match="no CPU path"):
        preference_loss_and_grad(x.detach())
    with pytest.raises(ValueError, match="no CPU path"):
        adamw_plan([x], [x], [x])


def test_plan_and_optimizer_refuse():
    x = torch.zeros(4)
    with pytest.raises(ValueError, match="one tensor for each"):
        adamw_plan([x, x], [x], [x, x])
    p = torch.nn.Parameter(torch.zeros(4))
    for kw in (dict(state_bits=4), dict(lr=-1.0), dict(eps=math.nan), dict(betas=(0.9, 1.0)),
               dict(weight_decay=math.inf)):
        with pytest.raises(ValueError):
            AdamW([p], **kw)
    adamw_plan([], [], []).step([], step=1, lr=1e-3)     # nothing to do


# ------------------------------------------------------------- the oracle
def test_oracle_policy_gradient_against_differences():
    g = np.random.default_rng(0)
    for dual in (0.0, 2.0):
        for kl in ("k1", "k2", "k3"):
            for red in ("sum", "mean", "sequence_mean"):
                lp, old, ref, adv = (g.normal(size=12) for _ in range(4))
                cut = [np.array([0, 1, 3]), np.array([], int), np.array([5, 6, 7, 8, 11])]

                def f(x):
                    return ref_ops.policy(cut, x, old, ref, adv, 0.2, 0.3, dual, 0.1, kl, red)
                grad = f(lp)[1]
                for i in range(12):
                    d = np.zeros(12)
                    d[i] = 1e-6
                    assert (f(lp + d)[0] - f(lp - d)[0]) / 2e-6 == pytest.approx(grad[i], abs=1e-7)


def test_oracle_preference_gradient_against_differences():
    g = np.random.default_rng(1)
    for kind, e in (("sigmoid", 0.0), ("sigmoid", 0.2), ("hinge", 0.0), ("ipo", 0.0)):
        for average in (False, True):
            lp, ref = g.normal(size=10), g.normal(size=10)
            cut = [np.array([0, 1]), np.array([2]), np.array([4, 5, 6]), np.array([], int)]

            def f(x):
                return ref_ops.preference(cut, x, ref, 0.3, 0.1, kind, e, average)
            grad = f(lp)[1]
            for i in range(10):
                d = np.zeros(10)
                d[i] = 1e-6
                assert (f(lp + d)[0] - f(lp - d)[0]) / 2e-6 == pytest.approx(grad[i], abs=1e-7)


def test_oracle_e4m3_is_torchs():
    v = torch.arange(0x7F, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(ref_ops.e4m3_values(), v)


def test_random_bits_are_even_and_unrelated():
    """Every bit set half of the time, in every step; neighbours, steps and seeds uncorrelated."""
    n = 1 << 16
    a = ref_ops.pair_bits(n, 0, 1, 1)
    for seed, step in ((1, 1), (1, 2), (2, 1), (0, 1000)):
        b = ref_ops.pair_bits(n, 0, seed, step)
        for bit in range(16):    # 6 sigma of a fair coin: 3 / sqrt(n)
            assert abs((b >> bit & 1).mean() - 0.5) < 3 / math.sqrt(n)
        if (seed, step) != (1, 1):
            assert abs(np.corrcoef(a, b)[0, 1]) < 6 / math.sqrt(n)
        for lag in (1, 2, 256):
            assert abs(np.corrcoef(b[lag:], b[:-lag])[0, 1]) < 6 / math.sqrt(n)
    np.testing.assert_array_equal(ref_ops.pair_bits(512, 3, 7, 9), ref_ops.pair_bits(2048, 0, 7, 9)[768:1280])


def test_stochastic_code_matches_its_probability():
    x = np.full(1 << 16, 20.5)              # between 20 and 22: a quarter of the way
    c = ref_ops.stochastic_code(x, np.arange(1 << 16))
    v = ref_ops.e4m3_values()[c]
    assert set(v) == {20.0, 22.0} and v.mean() == pytest.approx(20.5, abs=1e-4)
    assert (ref_ops.stochastic_code(np.array([0.0, 1e-9, 448.0]), np.array([65535, 0, 65535])) ==
            [0, 1, 0x7E]).all()
