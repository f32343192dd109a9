"""AdamW's checks of its tensors: gradients that disagree, other orders, and parameters given other views."""
import pytest
import torch

from linear_cross_entropy_tiled_gb300 import AdamW, adamw_plan

pytestmark = pytest.mark.gpu

SHAPES = [(3, 5), (), (300,), (0, 4), (7, 2, 9)]


def made(seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    params = [torch.randn(s, device="cuda", generator=g) for s in SHAPES]
    grads = [torch.randn(s, device="cuda", generator=g) for s in SHAPES]
    return params, grads, adamw_plan(params, [torch.zeros_like(p) for p in params],
                                     [torch.zeros_like(p) for p in params])


@pytest.mark.parametrize("at", [0, 1, 4])
def test_a_gradient_that_disagrees_is_refused_and_nothing_changes(at):
    params, grads, plan = made()
    before = [p.clone() for p in params]
    p = params[at]
    for bad, error in ((grads[at].half(), TypeError), (grads[at].cpu(), TypeError),
                       (grads[at].reshape(*p.shape, 1), ValueError),
                       (torch.zeros(*p.shape, 2, device="cuda"), ValueError)):
        if at == 0 and bad.dtype == torch.half:
            continue    # the first gradient's dtype is the one the others are held to
        with pytest.raises(error):
            plan.step([*grads[:at], bad, *grads[at + 1:]], step=1, lr=0.1)
    with pytest.raises(ValueError, match="gradients for"):
        plan.step(grads[:-1], step=1, lr=0.1)
    assert all(torch.equal(x, y) for x, y in zip(params, before))


def test_gradients_of_other_orders_and_sequences():
    """Strided, expanded and transposed gradients, in a tuple: as their contiguous copies in a list."""
    a, grads, plan_a = made()
    b, _, plan_b = made()
    odd = [grads[0].t().contiguous().t(), grads[1], grads[2][:1].expand(300), grads[3],
           torch.stack([grads[4]] * 2, dim=-1)[..., 1]]
    plan_a.step(tuple(odd), step=1, lr=0.1)
    plan_b.step([g.contiguous() for g in odd], step=1, lr=0.1)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_a_parameter_given_another_view_of_its_memory():
    """Its states have another order by then: refused, and the step before it stays what it was."""
    p = torch.nn.Parameter(torch.arange(16., device="cuda").view(4, 4))
    opt = AdamW([p], lr=0.1)
    p.grad = torch.ones_like(p)
    opt.step()
    p.data, p.grad = p.data.t(), None
    p.grad = torch.ones_like(p)
    before = p.detach().clone()
    with pytest.raises(ValueError, match="shape and strides"):
        opt.step()
    assert torch.equal(p, before)
    assert opt.state[p]["step"] == 1
