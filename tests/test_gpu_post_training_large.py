"""Batches and parameters of more than 2^31 elements: every token and element is reached, once."""
import math

import pytest
import torch

from linear_cross_entropy_tiled_gb300 import adamw_plan, policy_loss_and_grad, preference_loss_and_grad

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def room():
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 64 << 30:
        pytest.skip("needs 64 GB")
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("reduction", ["mean", "sequence_mean"])
@pytest.mark.parametrize("pad", [0, 5])
def test_policy(reduction, pad):
    """Three rows, ratio 1, five masked tokens a row. Each sum of equal terms keeps 20 bits or more.

    ``pad`` puts the rows further apart, which is the strided kernel.
    """
    S, C, off = 3, 800_000_003, 5
    lp = torch.full((S, C + pad), -0.25, dtype=torch.bfloat16, device="cuda")[:, :C]
    mask = torch.ones(S, C, dtype=torch.bool, device="cuda")
    mask[:, C // 2:C // 2 + off] = False
    adv = torch.tensor([1.0, -2.0, 3.0], device="cuda")
    loss, grad, m = policy_loss_and_grad(lp, None, adv, mask=mask, reduction=reduction, return_metrics=True)
    n = S * (C - off)
    assert int(m["num_tokens"]) == n and int(m["num_clipped"]) == 0
    assert loss.item() == pytest.approx(-2 / 3, rel=2.0 ** -20)
    for s in range(S):
        assert grad[s, 0].item() == pytest.approx(-adv[s].item() / n, rel=2.0 ** -21)
        assert (grad[s, :C // 2] == grad[s, 0]).all() and (grad[s, C // 2 + off:] == grad[s, 0]).all()
        assert (grad[s, C // 2:C // 2 + off] == 0).all()


def test_preference():
    C = 1_200_000_001
    lp = torch.full((2, C), -0.5, dtype=torch.bfloat16, device="cuda")
    lp[1] = -0.25
    loss, grad, chosen, rejected = preference_loss_and_grad(lp, beta=0.5, average=True)
    assert chosen.item() == pytest.approx(-0.25, rel=2.0 ** -20)
    assert rejected.item() == pytest.approx(-0.125, rel=2.0 ** -20)
    assert loss.item() == pytest.approx(math.log1p(math.exp(0.125)), rel=2.0 ** -19)
    want = 0.5 / (1 + math.exp(-0.125)) / C
    for s, sign in ((0, -1), (1, 1)):
        assert grad[s, 0].item() == pytest.approx(sign * want, rel=2.0 ** -19)
        assert (grad[s] == grad[s, 0]).all()


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw(bits):
    """The first step moves every element by lr, against its gradient's sign, and leaves equal states."""
    n = (1 << 31) + 256 + 7
    dt = torch.bfloat16
    p = torch.ones(n, dtype=dt, device="cuda")
    g = torch.ones(n, dtype=dt, device="cuda")
    state = torch.float8_e4m3fn if bits == 8 else torch.float32
    m, v = (torch.zeros(n, dtype=torch.uint8, device="cuda").view(state) if bits == 8 else
            torch.zeros(n, device="cuda") for _ in range(2))
    scales = [torch.zeros(-(-n // 256), device="cuda") for _ in range(2)] if bits == 8 else [None] * 2
    plan = adamw_plan([p], [m], [v], **({} if bits == 32 else dict(
        exp_avg_scales=[scales[0]], exp_avg_sq_scales=[scales[1]])))
    plan.step([g], step=1, lr=0.25, eps=0.0, weight_decay=0.0)
    assert (p == 0.75).all()
    for t in (m, v):
        raw = t.view(torch.uint8) if bits == 8 else t
        assert (raw == raw[0]).all() and raw[0] != 0
    for s in scales:
        assert s is None or ((s == s[0]).all() and s[0] > 0)
