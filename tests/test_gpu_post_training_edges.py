"""Corners of the post-training operators: many sequences with few tokens, NaN in tokens that count, copies of
the optimizer. Tolerances as in test_gpu_post_training.py."""
import copy
import io

import numpy as np
import pytest
import torch

import oracle.post_training_oracle as ref_ops
from linear_cross_entropy_tiled_gb300 import AdamW, policy_loss_and_grad, preference_loss_and_grad

pytestmark = pytest.mark.gpu

TOL = 4e-6


@pytest.mark.parametrize("lengths", [[0] * 3000, [0] * 2999 + [5], [3] + [0] * 1500 + [1] * 700 + [40],
                                     [1, 0] * 2000])
@pytest.mark.parametrize("red", ["sum", "mean", "sequence_mean"])
def test_many_sequences_few_tokens(lengths, red):
    """More sequences than one cluster counts, with tokens for a fraction of a block."""
    g = torch.Generator(device="cuda").manual_seed(0)
    cu = np.concatenate([[0], np.cumsum(lengths)])
    n = int(cu[-1])
    lp = -torch.rand(n, device="cuda", generator=g)
    mask = torch.rand(n, device="cuda", generator=g) < 0.8
    adv = torch.randn(len(lengths), device="cuda", generator=g)
    keep = mask.cpu().numpy()
    cut = [np.arange(a, b)[keep[a:b]] for a, b in zip(cu, cu[1:])]
    row = np.repeat(np.arange(len(lengths)), lengths)
    cu_t = torch.tensor(cu, dtype=torch.int32, device="cuda")
    loss, grad, m = policy_loss_and_grad(lp, None, adv, mask=mask, cu_seqlens=cu_t, reduction=red,
                                         return_metrics=True)
    x = lp.double().cpu().numpy()
    want, wgrad, tokens, _, _, total, size, _ = ref_ops.policy(
        cut, x, None, None, adv.double().cpu().numpy()[row], 0.2, 0.2, 0.0, 0.0, "k3", red)
    if np.isnan(want):
        assert loss.isnan()
    else:
        assert abs(loss.item() - want) <= TOL * total + 1e-30
    assert (np.abs(grad.double().cpu().numpy() - wgrad) <= TOL * size).all()
    assert int(m["num_tokens"]) == tokens
    loss, grad, chosen, rejected = preference_loss_and_grad(lp, mask=mask, cu_seqlens=cu_t)
    want, wgrad, wc, wr, slack = ref_ops.preference(cut, x, None, 0.1, 0.0, "sigmoid", 0.0, False)
    assert loss.item() == pytest.approx(want, abs=TOL * (1 + slack.max()))
    assert np.abs(grad.double().cpu().numpy() - wgrad).max(initial=0) <= TOL * (1 + slack.max())
    np.testing.assert_allclose(chosen.double().cpu().numpy(), wc, atol=TOL * (1 + slack.max()))


@pytest.mark.parametrize("shape", [(3000, 0), (3000, 2), (5000, 3)])
def test_many_short_rows(shape):
    lp = -torch.rand(shape, device="cuda")
    mask = torch.rand(shape, device="cuda") < 0.5
    adv = torch.ones(shape[0], device="cuda")
    loss, grad = policy_loss_and_grad(lp, None, adv, mask=mask, reduction="sequence_mean")
    n = mask.sum(1, keepdim=True)
    want = torch.where(mask, -1.0 / (shape[0] * n.clamp(min=1)), 0.0)
    assert torch.allclose(grad, want, rtol=1e-6, atol=0)
    assert loss.item() == pytest.approx(-(n > 0).float().mean().item() if shape[1] else 0.0, rel=1e-5)


@pytest.mark.parametrize("kind", ["sigmoid", "hinge", "ipo"])
def test_nan_that_counts_shows(kind):
    """A NaN log prob of a token that counts: NaN loss, NaN gradients of its pair, and of no other."""
    lp = -torch.rand(8, 50, device="cuda")
    lp[1, 7] = float("nan")
    loss, grad, chosen, rejected = preference_loss_and_grad(lp, loss_type=kind)
    assert loss.isnan() and chosen[1].isnan() and chosen.isnan().sum() == 1 and not rejected.isnan().any()
    assert grad[1].isnan().all() and grad[5].isnan().all()
    assert grad[[0, 2, 3, 4, 6, 7]].isfinite().all()
    lp[1, 7] = float("inf")
    loss, grad, chosen, _ = preference_loss_and_grad(lp, loss_type=kind)
    assert chosen[1] == float("inf")


def test_optimizer_copies():
    """deepcopy and torch.save keep the kind of states, and the copies step alike."""
    p = torch.nn.Parameter(torch.ones(700, device="cuda", dtype=torch.bfloat16))
    opt = AdamW([p], lr=0.01, state_bits=8, master_weights=True, seed=3)
    p.grad = torch.randn_like(p)
    opt.step()
    q, qopt = copy.deepcopy((p, opt))
    assert qopt.param_groups[0]["params"][0] is q and qopt.param_groups[0]["state_bits"] == 8
    file = io.BytesIO()
    torch.save((p, opt), file)
    file.seek(0)
    r, ropt = torch.load(file, weights_only=False)
    for x, o in ((p, opt), (q, qopt), (r, ropt)):
        x.grad = torch.full_like(x, 0.5)
        o.step()
    for x, o in ((q, qopt), (r, ropt)):
        assert torch.equal(p, x) and o.state[x]["exp_avg"].dtype == torch.float8_e4m3fn
        assert torch.equal(opt.state[p]["exp_avg_sq"].view(torch.uint8),
                           o.state[x]["exp_avg_sq"].view(torch.uint8))


def test_groups_of_different_states():
    a, b = (torch.nn.Parameter(torch.ones(300, device="cuda")) for _ in range(2))
    opt = AdamW([{"params": [a], "state_bits": 8}, {"params": [b]}], lr=0.1)
    for p in (a, b):
        p.grad = torch.ones_like(p)
    opt.step()
    assert opt.state[a]["exp_avg"].dtype == torch.float8_e4m3fn
    assert opt.state[b]["exp_avg"].dtype == torch.float32
    assert torch.equal(a, b)     # the update uses the unrounded moments
