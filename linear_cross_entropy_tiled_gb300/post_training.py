"""Losses of post-training on per-token log probabilities: the clipped policy loss and the preference loss.

Both come in three forms. ``*_loss_and_grad`` takes log probabilities and
returns the loss with its gradient in them, in one call of the library.
``policy_loss`` / ``preference_loss`` are the same as differentiable functions
of the log probabilities. ``fused_linear_*`` start from the hidden states and
the vocabulary projection: the log probabilities come from ``flce_forward``
(the logits are never stored) and the gradient goes on to ``flce_backward``.

A batch is padded, ``[sequences, cols]`` tensors whose rows may be strided, or
packed, ``[tokens]`` tensors with ``cu_seqlens`` (int32 ``[sequences + 1]``,
from 0 to tokens). ``mask`` says which tokens count; what the tensors hold
elsewhere is not used, and a sequence may have no token that counts.
include/flce.h gives the formulas.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import _lib
from .functional import (_DTYPES, _maybe_check, _params, _prepare, _ptr, _stream, flce_backward,
                         flce_forward)


def _laid_out(t: Optional[torch.Tensor], shape, dtype, device, name: str):
    """(tensor, row stride) of a token tensor; anything but adjacent tokens in a row is copied."""
    if t is None:
        return None, 0
    if t.shape != shape:
        raise ValueError(f"{name} must have the shape of the log probabilities, {tuple(shape)}, "
                         f"got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}")
    if t.dim() == 1:
        return t.contiguous(), 0
    if t.shape[1] > 1 and t.stride(1) != 1 or t.stride(0) < t.shape[1]:
        t = t.contiguous()
    return t, max(t.stride(0), t.shape[1])


def _token_fields(x: torch.Tensor, mask, cu_seqlens, name: str):
    """flce_tokens of the batch, the number of sequences, and the tensors it points to."""
    if not x.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (there is no CPU path)")
    if x.dtype not in _DTYPES:
        raise TypeError(f"{name} must be float32, bfloat16 or float16, got {x.dtype}")
    t = _lib.FlceTokens()
    cu = None
    if cu_seqlens is None:
        if x.dim() != 2:
            raise ValueError(f"{name} must be [sequences, cols], or [tokens] with cu_seqlens; "
                             f"got {tuple(x.shape)}")
        t.sequences, t.cols = x.shape
    else:
        if x.dim() != 1:
            raise ValueError(f"{name} must be [tokens] with cu_seqlens, got {tuple(x.shape)}")
        if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1 or cu_seqlens.device != x.device:
            raise ValueError(f"cu_seqlens must be [sequences + 1] on {x.device}")
        if cu_seqlens.dtype not in (torch.int32, torch.int64):
            raise TypeError(f"cu_seqlens must be int32 or int64, got {cu_seqlens.dtype}")
        cu = cu_seqlens.to(torch.int32).contiguous()
        t.packed, t.sequences, t.tokens, t.cu_seqlens = 1, cu.shape[0] - 1, x.shape[0], cu.data_ptr()
    if mask is not None:
        if mask.dtype not in (torch.bool, torch.uint8):
            raise TypeError(f"mask must be bool or uint8, got {mask.dtype}")
        mask, t.ld_mask = _laid_out(mask, x.shape, mask.dtype, x.device, "mask")
        t.mask, t.mask_kind = _ptr(mask), _lib.FLCE_MASK_BYTES
    return t, int(t.sequences), (cu, mask)


def _option(table: dict, value: str, name: str) -> int:
    if value not in table:
        raise ValueError(f"{name} must be one of {tuple(table)}, got {value!r}")
    return table[value]


def _run_policy(a: _lib.FlcePolicyArgs, dev: torch.device, return_metrics: bool):
    out = torch.empty(2, dtype=torch.float32, device=dev)
    a.loss = out.data_ptr()
    metrics = None
    if return_metrics:
        n = torch.empty(2, dtype=torch.int64, device=dev)
        a.num_tokens, a.num_clipped, a.kl_sum = n.data_ptr(), n.data_ptr() + 8, out.data_ptr() + 4
        metrics = {"num_tokens": n[0], "num_clipped": n[1], "kl_sum": out[1]}
    ws = torch.empty(_lib.policy_workspace_bytes(a), dtype=torch.uint8, device=dev)
    a.workspace, a.ws_bytes = ws.data_ptr(), ws.numel()
    _lib.check(_lib.policy_loss_raw(a, _stream(dev)), "flce_policy_loss")
    return out[0], metrics


def _policy_args(tokens, log_probs, ld, old, advantages, ref, clip_low, clip_high, dual_clip,
                 kl_coef, kl_estimator, reduction, grad):
    """FlcePolicyArgs without its outputs but ``grad``, and the tensors it points to."""
    shape, dtype, dev = log_probs.shape, log_probs.dtype, log_probs.device
    a = _lib.FlcePolicyArgs()
    a.tokens = tokens
    a.kl_estimator = _option(_lib.KL_ESTIMATORS, kl_estimator, "kl_estimator")
    a.reduction = _option(_lib.TOKEN_REDUCTIONS, reduction, "reduction")
    if kl_coef and ref is None:
        raise ValueError("kl_coef needs ref_log_probs")
    if advantages.dtype != torch.float32 or advantages.device != dev:
        raise TypeError(f"advantages must be float32 on {dev}")
    S = tokens.sequences
    if advantages.shape == (S,) and not (tokens.packed and shape == (S,)) \
            or advantages.shape == (S, 1) and shape[-1] != 1:
        advantages, ld_adv = advantages.reshape(S).contiguous(), 0
    else:
        advantages, ld_adv = _laid_out(advantages, shape, torch.float32, dev,
                                       "advantages, unless it is one per sequence,")
        a.advantage_per_token = 1
    old, a.ld_old = _laid_out(old, shape, dtype, dev, "old_log_probs")
    ref, a.ld_ref = _laid_out(ref, shape, dtype, dev, "ref_log_probs")
    a.log_probs, a.ld_log_probs = _ptr(log_probs), ld
    a.old_log_probs, a.ref_log_probs, a.advantages = _ptr(old), _ptr(ref), _ptr(advantages)
    a.ld_advantages = ld_adv
    a.grad, a.ld_grad = _ptr(grad), shape[-1]
    a.clip_low, a.clip_high, a.dual_clip = clip_low, clip_high, dual_clip or 0.0
    a.kl_coef, a.dtype = kl_coef, _DTYPES[dtype]
    return a, (old, ref, advantages)


def policy_loss_and_grad(log_probs: torch.Tensor, old_log_probs: Optional[torch.Tensor],
                         advantages: torch.Tensor, *,
                         ref_log_probs: Optional[torch.Tensor] = None,
                         mask: Optional[torch.Tensor] = None,
                         cu_seqlens: Optional[torch.Tensor] = None, clip_low: float = 0.2,
                         clip_high: float = 0.2, dual_clip: Optional[float] = None,
                         kl_coef: float = 0.0, kl_estimator: str = "k3", reduction: str = "mean",
                         return_metrics: bool = False):
    """The clipped policy loss with a KL term, and its gradient in ``log_probs``.

    ``old_log_probs`` (None: the policy drew the tokens itself) and
    ``ref_log_probs`` have the shape and dtype of ``log_probs``;
    ``advantages`` is float32, one per sequence or one per token. (A packed
    batch of as many sequences as tokens reads it as one per token; the two
    are the same there unless a sequence is empty.)
    ``reduction``: "sum", "mean" over the tokens that count, or
    "sequence_mean", the mean over sequences of each one's mean.

    Returns ``(loss, grad)``, both float32, or ``(loss, grad, metrics)`` with
    the device scalars num_tokens, num_clipped (int64) and kl_sum.
    """
    tokens, _, keep = _token_fields(log_probs, mask, cu_seqlens, "log_probs")
    log_probs, ld = _laid_out(log_probs, log_probs.shape, log_probs.dtype, log_probs.device,
                              "log_probs")
    grad = torch.empty(log_probs.shape, dtype=torch.float32, device=log_probs.device)
    a, keep2 = _policy_args(tokens, log_probs, ld, old_log_probs, advantages, ref_log_probs,
                            clip_low, clip_high, dual_clip, kl_coef, kl_estimator, reduction, grad)
    loss, metrics = _run_policy(a, log_probs.device, return_metrics)
    return (loss, grad, metrics) if return_metrics else (loss, grad)


def _run_preference(a: _lib.FlcePreferenceArgs, dev: torch.device, pairs: int):
    out = torch.empty(1 + 2 * pairs, dtype=torch.float32, device=dev)
    a.loss, a.chosen_rewards = out.data_ptr(), out.data_ptr() + 4
    a.rejected_rewards = out.data_ptr() + 4 + 4 * pairs
    ws = torch.empty(_lib.preference_workspace_bytes(a), dtype=torch.uint8, device=dev)
    a.workspace, a.ws_bytes = ws.data_ptr(), ws.numel()
    _lib.check(_lib.preference_loss_raw(a, _stream(dev)), "flce_preference_loss")
    return out[0], out[1:1 + pairs], out[1 + pairs:]


def _preference_args(tokens, log_probs, ld, ref, beta, loss_type, label_smoothing, margin, average,
                     grad):
    if tokens.sequences % 2:
        raise ValueError("a preference batch needs an even number of sequences: the chosen ones, "
                         "then the rejected ones")
    shape = log_probs.shape
    a = _lib.FlcePreferenceArgs()
    a.tokens = tokens
    a.loss_type = _option(_lib.PREFERENCE_LOSSES, loss_type, "loss_type")
    ref, a.ld_ref = _laid_out(ref, shape, log_probs.dtype, log_probs.device, "ref_log_probs")
    a.log_probs, a.ld_log_probs, a.ref_log_probs = _ptr(log_probs), ld, _ptr(ref)
    a.grad, a.ld_grad = _ptr(grad), shape[-1]
    a.beta, a.label_smoothing, a.margin = beta, label_smoothing, margin
    a.dtype, a.average = _DTYPES[log_probs.dtype], 1 if average else 0
    return a, ref


def preference_loss_and_grad(log_probs: torch.Tensor, ref_log_probs: Optional[torch.Tensor] = None,
                             *, mask: Optional[torch.Tensor] = None,
                             cu_seqlens: Optional[torch.Tensor] = None, beta: float = 0.1,
                             loss_type: str = "sigmoid", label_smoothing: float = 0.0,
                             margin: float = 0.0, average: bool = False):
    """The preference loss of paired sequences, and its gradient in ``log_probs``.

    The first half of the sequences are the chosen ones, the second half the
    rejected ones in the same order. ``loss_type``: "sigmoid", "hinge" or
    "ipo". ``average`` takes the mean over a sequence's tokens for the sum.

    Returns ``(loss, grad, chosen_rewards, rejected_rewards)``, all float32;
    the rewards are beta times each sequence's log ratio.
    """
    tokens, sequences, keep = _token_fields(log_probs, mask, cu_seqlens, "log_probs")
    log_probs, ld = _laid_out(log_probs, log_probs.shape, log_probs.dtype, log_probs.device,
                              "log_probs")
    grad = torch.empty(log_probs.shape, dtype=torch.float32, device=log_probs.device)
    a, keep2 = _preference_args(tokens, log_probs, ld, ref_log_probs, beta, loss_type,
                                label_smoothing, margin, average, grad)
    loss, chosen, rejected = _run_preference(a, log_probs.device, sequences // 2)
    return loss, grad, chosen, rejected


def _scaled(grad: torch.Tensor, grad_loss: torch.Tensor) -> torch.Tensor:
    """grad times the upstream scalar, in a new tensor (a second backward starts from grad again)."""
    out = torch.empty_like(grad)
    g = grad_loss.to(dtype=torch.float32).reshape(1).contiguous()
    _lib.check(_lib.scale_raw(_ptr(grad), _ptr(out), grad.numel(), _lib.FLCE_F32, _ptr(g),
                              _stream(grad.device)), "flce_scale")
    return out


class _LogProbLoss(torch.autograd.Function):
    """A loss with its gradient computed in the forward; further outputs carry no gradient."""
    @staticmethod
    def forward(ctx, log_probs, fn):
        loss, grad, *more = fn(log_probs.detach())
        ctx.save_for_backward(grad)
        ctx.dtype = log_probs.dtype
        ctx.mark_non_differentiable(*more)
        return (loss, *more)

    @staticmethod
    def backward(ctx, grad_loss, *_):
        return _scaled(ctx.saved_tensors[0], grad_loss).to(ctx.dtype), None


_METRICS = ("num_tokens", "num_clipped", "kl_sum")


def policy_loss(log_probs: torch.Tensor, old_log_probs: Optional[torch.Tensor],
                advantages: torch.Tensor, **kw):
    """``policy_loss_and_grad`` as a differentiable function of ``log_probs``.

    Returns ``loss``, or ``(loss, metrics)`` with ``return_metrics``.
    """
    return_metrics = kw.pop("return_metrics", False)

    def fn(lp):
        loss, grad, m = policy_loss_and_grad(lp, old_log_probs, advantages, return_metrics=True, **kw)
        return (loss, grad, *(m[k] for k in _METRICS))
    loss, *m = _LogProbLoss.apply(log_probs, fn)
    return (loss, dict(zip(_METRICS, m))) if return_metrics else loss


def preference_loss(log_probs: torch.Tensor, ref_log_probs: Optional[torch.Tensor] = None, **kw):
    """``preference_loss_and_grad`` as a differentiable function of ``log_probs``.

    Returns ``(loss, chosen_rewards, rejected_rewards)``.
    """
    return _LogProbLoss.apply(log_probs, lambda lp: preference_loss_and_grad(lp, ref_log_probs, **kw))


class _FusedLinear(torch.autograd.Function):
    """hidden, weight, bias -> -log p of the targets -> a loss on them, and back."""
    @staticmethod
    def forward(ctx, hidden, weight, bias, targets, head, fn):
        ignore_index, logit_scale, softcap = head
        h2, w, t1, b = _prepare(hidden, weight, targets, bias)
        p = _params(h2, w, b, "none", ignore_index, logit_scale, softcap, 0.0, False)
        nll, lse, _, _, _ = flce_forward(p, h2, w, t1, b)
        loss, grad, *more = fn(nll.view(targets.shape), t1.view(targets.shape))
        ctx.save_for_backward(h2, w, t1, lse, b, grad)
        ctx.p, ctx.hidden_shape = p, hidden.shape
        ctx.mark_non_differentiable(*more)
        return (loss, *more)

    @staticmethod
    def backward(ctx, grad_loss, *_):
        h2, w, t1, lse, b, grad = ctx.saved_tensors
        need = ctx.needs_input_grad
        gh, gw, gb, _ = flce_backward(ctx.p, h2, w, t1, lse, _scaled(grad, grad_loss), b,
                                      need_hidden=need[0], need_weight=need[1], need_bias=need[2])
        return None if gh is None else gh.reshape(ctx.hidden_shape), gw, gb, None, None, None


def _label_tokens(nll, labels, ignore_index, cu_seqlens):
    tokens, sequences, keep = _token_fields(nll, None, cu_seqlens, "targets")
    tokens.mask, tokens.mask_kind = labels.data_ptr(), _lib.FLCE_MASK_LABELS
    tokens.ld_mask, tokens.ignore_index = labels.shape[-1], ignore_index
    return tokens, sequences, keep


def fused_linear_policy_loss(hidden: torch.Tensor, weight: torch.Tensor, targets: torch.Tensor,
                             old_log_probs: Optional[torch.Tensor], advantages: torch.Tensor, *,
                             bias: Optional[torch.Tensor] = None,
                             ref_log_probs: Optional[torch.Tensor] = None,
                             cu_seqlens: Optional[torch.Tensor] = None, ignore_index: int = -100,
                             logit_scale: float = 1.0, softcap: Optional[float] = None,
                             clip_low: float = 0.2, clip_high: float = 0.2,
                             dual_clip: Optional[float] = None, kl_coef: float = 0.0,
                             kl_estimator: str = "k3", reduction: str = "mean",
                             return_metrics: bool = False):
    """The clipped policy loss of ``hidden @ weight.T``'s log probabilities of ``targets``.

    ``targets`` is ``[sequences, cols]`` with ``hidden`` ``[sequences, cols, H]``,
    or ``[tokens]`` with ``hidden`` ``[tokens, H]`` and ``cu_seqlens``. Tokens
    whose target is ``ignore_index`` do not count. ``old_log_probs`` and
    ``ref_log_probs`` are float32 of the shape of targets. ``logit_scale`` is
    one over the sampling temperature. hidden, weight and bias receive
    gradients; the logits are never stored.
    """
    def fn(nll, labels):
        tokens, _, keep = _label_tokens(nll, labels, ignore_index, cu_seqlens)
        grad = torch.empty_like(nll)
        a, keep2 = _policy_args(tokens, nll, nll.shape[-1], old_log_probs, advantages, ref_log_probs,
                                clip_low, clip_high, dual_clip, kl_coef, kl_estimator, reduction,
                                grad)
        a.negated = 1
        loss, m = _run_policy(a, nll.device, True)
        return (loss, grad, *(m[k] for k in _METRICS))
    loss, *m = _FusedLinear.apply(hidden, weight, bias, targets, (ignore_index, logit_scale, softcap),
                                  fn)
    return (loss, dict(zip(_METRICS, m))) if return_metrics else loss


def fused_linear_preference_loss(hidden: torch.Tensor, weight: torch.Tensor, targets: torch.Tensor,
                                 ref_log_probs: Optional[torch.Tensor] = None, *,
                                 bias: Optional[torch.Tensor] = None,
                                 cu_seqlens: Optional[torch.Tensor] = None,
                                 ignore_index: int = -100, logit_scale: float = 1.0,
                                 softcap: Optional[float] = None, beta: float = 0.1,
                                 loss_type: str = "sigmoid", label_smoothing: float = 0.0,
                                 margin: float = 0.0, average: bool = False):
    """The preference loss of ``hidden @ weight.T``'s log probabilities of ``targets``.

    Shapes as in ``fused_linear_policy_loss``, pairs as in
    ``preference_loss_and_grad``. Returns ``(loss, chosen_rewards,
    rejected_rewards)``; hidden, weight and bias receive gradients.
    """
    def fn(nll, labels):
        tokens, sequences, keep = _label_tokens(nll, labels, ignore_index, cu_seqlens)
        grad = torch.empty_like(nll)
        a, keep2 = _preference_args(tokens, nll, nll.shape[-1], ref_log_probs, beta, loss_type,
                                    label_smoothing, margin, average, grad)
        a.negated = 1
        loss, chosen, rejected = _run_preference(a, nll.device, sequences // 2)
        return loss, grad, chosen, rejected
    return _FusedLinear.apply(hidden, weight, bias, targets, (ignore_index, logit_scale, softcap), fn)
