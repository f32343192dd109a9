"""Post-training of a small language-model head, with the pieces that a trainer would use:

    python -m linear_cross_entropy_tiled_gb300.examples.post_training [--loss policy|preference]
        [--steps 30] [--state-bits 8|32] [--vocab 2000] [--hidden 256]

The model maps a state (one of 64 random feature vectors) through one hidden
layer and a vocabulary projection to the next token. Policy training draws a
group of responses a prompt, rewards tokens of even id, and takes clipped
policy steps with a KL term to the starting model; preference training gets
pairs of a mostly even and a mostly odd response. Per step:

    hidden states -> fused_linear_policy_loss / fused_linear_preference_loss
    -> backward (no logits stored) -> AdamW with 8-bit or 32-bit states.

The old and reference log probabilities are the per-token losses of
``fused_linear_cross_entropy(reduction="none")`` with the sign turned.
"""
from __future__ import annotations

import argparse

import torch

from linear_cross_entropy_tiled_gb300 import (
    AdamW, fused_linear_cross_entropy, fused_linear_policy_loss, fused_linear_preference_loss)

STATES = 64


class Model(torch.nn.Module):
    def __init__(self, vocab: int, hidden: int, gen: torch.Generator):
        super().__init__()
        def randn(*shape):
            return torch.randn(*shape, device="cuda", generator=gen)
        self.register_buffer("features", randn(STATES, hidden).bfloat16())
        self.layer = torch.nn.Parameter((randn(hidden, hidden) / hidden ** 0.5).bfloat16())
        self.head = torch.nn.Parameter((randn(vocab, hidden) / hidden ** 0.5).bfloat16())

    def hidden(self, states: torch.Tensor) -> torch.Tensor:
        return torch.tanh(self.features[states] @ self.layer.T)


@torch.no_grad()
def log_probs(model: Model, states: torch.Tensor, targets: torch.Tensor) -> torch.Tensor:
    return -fused_linear_cross_entropy(model.hidden(states), model.head, targets, reduction="none")


@torch.no_grad()
def sample(model: Model, states: torch.Tensor, lengths: torch.Tensor, gen: torch.Generator):
    """A token for each state; the ones past a response's length are ignored (-100)."""
    p = torch.softmax(model.hidden(states).float() @ model.head.float().T, -1)
    t = torch.multinomial(p.view(-1, p.shape[-1]), 1, generator=gen).view(states.shape)
    return t.masked_fill(torch.arange(states.shape[1], device="cuda") >= lengths[:, None], -100)


def even_share(targets: torch.Tensor) -> torch.Tensor:
    """Share of a response's tokens whose id is even: its reward."""
    valid = targets >= 0
    return ((targets % 2 == 0) & valid).sum(1) / valid.sum(1).clamp(min=1)


def policy_step(model, start, opt, gen, prompts=8, group=16, length=48):
    B = prompts * group
    states = torch.randint(0, STATES, (prompts, length), device="cuda", generator=gen)
    states = states.repeat_interleave(group, 0)
    lengths = torch.randint(1, length + 1, (B,), device="cuda", generator=gen)
    targets = sample(model, states, lengths, gen)
    reward = even_share(targets)
    by_prompt = reward.view(prompts, group)
    adv = ((by_prompt - by_prompt.mean(1, keepdim=True)) / (by_prompt.std(1, keepdim=True) + 1e-4)).view(B)
    old, ref = log_probs(model, states, targets), log_probs(start, states, targets)
    for _ in range(2):      # two steps on a batch: the second one is off its policy
        loss, m = fused_linear_policy_loss(
            model.hidden(states), model.head, targets, old, adv, ref_log_probs=ref, clip_low=0.2,
            clip_high=0.28, kl_coef=0.02, reduction="sequence_mean", return_metrics=True)
        opt.zero_grad()
        loss.backward()
        opt.step()
    return reward.mean(), loss.detach(), m["kl_sum"] / m["num_tokens"]


def preference_step(model, start, opt, gen, pairs=64, length=48):
    states = torch.randint(0, STATES, (2 * pairs, length), device="cuda", generator=gen)
    lengths = torch.randint(1, length + 1, (2 * pairs,), device="cuda", generator=gen)
    targets = sample(start, states, lengths, gen)
    # the chosen half has even ids and the rejected half odd ones, but for one token in ten
    flip = torch.rand(targets.shape, device="cuda", generator=gen) < 0.9
    want = (torch.arange(2 * pairs, device="cuda") >= pairs).long()[:, None]
    targets = torch.where(flip & (targets >= 0), targets // 2 * 2 + want, targets)
    targets = targets.clamp(max=model.head.shape[0] - 1)
    ref = log_probs(start, states, targets)
    loss, chosen, rejected = fused_linear_preference_loss(
        model.hidden(states), model.head, targets, ref, beta=0.1)
    opt.zero_grad()
    loss.backward()
    opt.step()
    return (chosen > rejected).float().mean(), loss.detach(), (chosen - rejected).mean()


def main(argv=None) -> list:
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--loss", choices=("policy", "preference"), default="policy")
    ap.add_argument("--steps", type=int, default=30)
    ap.add_argument("--state-bits", type=int, choices=(8, 32), default=8)
    ap.add_argument("--vocab", type=int, default=2000)
    ap.add_argument("--hidden", type=int, default=256)
    ap.add_argument("--seed", type=int, default=0)
    a = ap.parse_args(argv)
    gen = torch.Generator(device="cuda").manual_seed(a.seed)
    model = Model(a.vocab, a.hidden, gen)
    start = Model(a.vocab, a.hidden, gen)
    start.load_state_dict(model.state_dict())
    opt = AdamW(model.parameters(), lr=3e-3, weight_decay=0.0, betas=(0.9, 0.99),
                state_bits=a.state_bits, master_weights=True, seed=a.seed)
    step, names = {"policy": (policy_step, ("reward", "loss", "kl")),
                   "preference": (preference_step, ("accuracy", "loss", "margin"))}[a.loss]
    history = []
    for i in range(a.steps):
        history.append([float(x) for x in step(model, start, opt, gen)])
        if i % 5 == 0 or i == a.steps - 1:
            print(f"step {i:3d}  " + "  ".join(f"{n} {x:.4f}" for n, x in zip(names, history[-1])))
    return history


if __name__ == "__main__":
    main()
