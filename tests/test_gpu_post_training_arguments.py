"""The losses' tensors, one by one: what is refused, and layouts that give what contiguous ones give."""
import pytest
import torch

from linear_cross_entropy_tiled_gb300 import policy_loss_and_grad, preference_loss_and_grad

pytestmark = pytest.mark.gpu


def tensors(packed=False, seed=0, S=6, C=50):
    g = torch.Generator(device="cuda").manual_seed(seed)
    shape = (S * C,) if packed else (S, C)
    t = {k: -torch.rand(shape, device="cuda", generator=g) for k in ("log_probs", "old", "ref")}
    t["mask"] = torch.rand(shape, device="cuda", generator=g) < 0.7
    t["advantages"] = torch.randn(shape, device="cuda", generator=g)
    t["cu"] = torch.tensor([0, 3, 3, 80, 200, 299, 300], device="cuda", dtype=torch.int32) if packed else None
    return t


def policy(t):
    loss, grad, m = policy_loss_and_grad(t["log_probs"], t["old"], t["advantages"], ref_log_probs=t["ref"],
                                         mask=t["mask"], cu_seqlens=t["cu"], kl_coef=0.1,
                                         reduction="sequence_mean", return_metrics=True)
    return (loss, grad, *(m[k] for k in ("num_tokens", "num_clipped", "kl_sum")))


def preference(t):
    return preference_loss_and_grad(t["log_probs"], t["ref"], mask=t["mask"], cu_seqlens=t["cu"])


USES = {policy: ("log_probs", "old", "ref", "mask", "advantages"), preference: ("log_probs", "ref", "mask")}
ALL = [(op, k) for op, names in USES.items() for k in names]


@pytest.mark.parametrize("op,name", ALL)
def test_wrong_tensors_are_refused(op, name):
    good = tensors()
    x = good[name]
    for bad in (x.cpu(), x.double(), x[:, :-1].contiguous(), x[:-1], x[None], x.to_sparse()):
        with pytest.raises((ValueError, TypeError, RuntimeError)):
            op({**good, name: bad})
    if name != "mask":
        with pytest.raises((TypeError, ValueError)):
            op({**good, name: x.half()})       # the others stay float32
    op(good)


@pytest.mark.parametrize("op", [policy, preference])
def test_wrong_cu_seqlens_are_refused(op):
    good = tensors(packed=True)
    cu = good["cu"]
    for bad in (None, cu.cpu(), cu.float(), cu[:0], cu[None], cu.to(torch.int16)):
        with pytest.raises((ValueError, TypeError)):
            op({**good, "cu": bad})
    with pytest.raises(ValueError):
        op({**tensors(), "cu": cu})
    op(good)


@pytest.mark.parametrize("op,name", ALL)
def test_layouts(op, name):
    """Rows further apart, columns first, every second element, expanded rows.

    What is copied gives the bits of the contiguous tensor. Rows further apart
    are read where they lie, in groups of another size, so sums may round
    otherwise: each by 2^-20 of its terms' magnitudes at most (16 roundings).
    Those add up to less than 11 for the policy loss (advantages below 4,
    ratios below e), to less than 50 for a sequence of the preference loss
    (times beta = 0.1, and a sigmoid's slope is at most 1); the KL terms are
    all positive.
    """
    t = tensors()
    want = op(t)
    x = t[name]
    wide = torch.zeros(6, 77, dtype=x.dtype, device="cuda")
    wide[:, :50] = x
    assert not wide[:, :50].is_contiguous()
    for a, b in zip(op({**t, name: wide[:, :50]}), want):
        assert torch.allclose(a, b, rtol=2.0 ** -20, atol=11 * 2.0 ** -20 if a.is_floating_point() else 0)
    for y in (x.t().contiguous().t(), torch.stack([x, x], dim=-1)[..., 0]):
        assert not y.is_contiguous()
        for a, b in zip(op({**t, name: y}), want):
            assert torch.equal(a, b)
    same = {**t, name: x[:1].expand(6, 50)}
    for a, b in zip(op(same), op({**t, name: x[:1].repeat(6, 1)})):
        assert torch.equal(a, b)


@pytest.mark.parametrize("op", [policy, preference])
def test_cu_seqlens_of_other_kinds(op):
    t = tensors(packed=True)
    want = op(t)
    for cu in (t["cu"].long(), torch.stack([t["cu"]] * 2, dim=-1)[:, 0]):
        for a, b in zip(op({**t, "cu": cu}), want):
            assert torch.equal(a, b)


def test_advantages_as_a_column_and_by_stride():
    t = tensors()
    adv = torch.randn(6, device="cuda")
    want = policy({**t, "advantages": adv})
    for a in (adv[:, None], torch.stack([adv] * 3, dim=-1)[:, 1]):
        for x, y in zip(policy({**t, "advantages": a}), want):
            assert torch.equal(x, y)
    for bad in (adv[:5], adv[None], adv.double(), adv.cpu()):
        with pytest.raises((ValueError, TypeError)):
            policy({**t, "advantages": bad})


def test_numbers_of_the_wrong_kind():
    t = tensors()
    for kw in (dict(clip_low="x"), dict(clip_high=None), dict(dual_clip="y"), dict(kl_coef="z")):
        with pytest.raises((TypeError, ValueError)):
            policy_loss_and_grad(t["log_probs"], t["old"], t["advantages"], **kw)
    for kw in (dict(beta="x"), dict(label_smoothing=None), dict(margin=[])):
        with pytest.raises((TypeError, ValueError)):
            preference_loss_and_grad(t["log_probs"], **kw)


def test_outputs_are_new_each_time_and_inputs_may_require_gradients():
    t = tensors()
    t["log_probs"].requires_grad_(True)
    first = policy(t)
    copies = [x.clone() for x in first]
    second = policy({**t, "old": t["old"] - 1})
    assert all(torch.equal(a, b) for a, b in zip(first, copies))
    assert not any(a.data_ptr() == b.data_ptr() for a, b in zip(first, second))
    assert not any(a.requires_grad for a in first)
    with torch.inference_mode():
        assert all(torch.equal(a, b) for a, b in zip(policy(t), copies))
