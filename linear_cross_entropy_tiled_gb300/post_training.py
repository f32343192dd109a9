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

from typing import Optional

import torch

from . import _lib
from .functional import (_DTYPES, _maybe_check, _params, _prepare, _ptr, _stream, flce_backward,
                         flce_forward)

# Workspace bounds of include/flce.h: none for this many tokens, else so many
# bytes and 8 (preference loss: 4) for each sequence (pair).
_SMALL = 8192
_POLICY_WORKSPACE, _PREFERENCE_WORKSPACE = 49152, 256


def _laid_out(t: torch.Tensor, shape, dtype, device, name: str):
    """(tensor, row stride) of a token tensor; anything but adjacent tokens in a row is copied."""
    if t.shape != shape:
        raise ValueError(f"{name} must have the shape of the log probabilities, {tuple(shape)}, "
                         f"got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}")
    cols = shape[-1]
    if t.is_contiguous():
        return t, cols
    if len(shape) == 1 or (cols > 1 and t.stride(1) != 1) or t.stride(0) < cols:
        return t.contiguous(), cols
    return t, t.stride(0)


def _tokens(x: torch.Tensor, mask, cu_seqlens, name: str):
    """The fields of flce_tokens, the number of sequences, and the tensors they point to."""
    if not x.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (there is no CPU path)")
    if x.dtype not in _DTYPES:
        raise TypeError(f"{name} must be float32, bfloat16 or float16, got {x.dtype}")
    shape = x.shape
    if cu_seqlens is None:
        if len(shape) != 2:
            raise ValueError(f"{name} must be [sequences, cols], or [tokens] with cu_seqlens; "
                             f"got {tuple(shape)}")
        sequences, cols = shape
        tokens = packed = cu = 0
    else:
        if len(shape) != 1:
            raise ValueError(f"{name} must be [tokens] with cu_seqlens, got {tuple(shape)}")
        if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1 or cu_seqlens.device != x.device:
            raise ValueError(f"cu_seqlens must be [sequences + 1] on {x.device}")
        if cu_seqlens.dtype not in (torch.int32, torch.int64):
            raise TypeError(f"cu_seqlens must be int32 or int64, got {cu_seqlens.dtype}")
        cu_seqlens = cu_seqlens.to(torch.int32).contiguous()
        sequences, cols, tokens, packed = cu_seqlens.shape[0] - 1, 0, shape[0], 1
        cu = cu_seqlens.data_ptr()
    where = kind = ld = 0
    if mask is not None:
        if mask.dtype is not torch.bool and mask.dtype is not torch.uint8:
            raise TypeError(f"mask must be bool or uint8, got {mask.dtype}")
        mask, ld = _laid_out(mask, shape, mask.dtype, x.device, "mask")
        where, kind = mask.data_ptr(), _lib.FLCE_MASK_BYTES
    return (sequences, cols, tokens, cu, where, ld, 0, packed, kind), sequences, (cu_seqlens, mask)


def _label_tokens(nll, labels, ignore_index, cu_seqlens):
    """``_tokens`` for log probabilities of ``labels`` (contiguous): those that are ignored do not count."""
    (sequences, cols, tokens, cu, *_, packed, _), n, keep = _tokens(nll, None, cu_seqlens, "targets")
    return (sequences, cols, tokens, cu, labels.data_ptr(), labels.shape[-1], ignore_index, packed,
            _lib.FLCE_MASK_LABELS), n, keep


def _float_like(x: torch.Tensor, shape, device) -> torch.Tensor:
    """A new contiguous float32 tensor of the log probabilities' shape."""
    if x.dtype is torch.float32 and x.is_contiguous():
        return torch.empty_like(x)
    return torch.empty(shape, dtype=torch.float32, device=device)


_templates: dict = {}


def _scalar_templates(device):
    """A float32 and an int64 scalar of the device for empty_like, the quickest way to new scalars."""
    t = _templates.get(device)
    if t is None:
        t = _templates[device] = (torch.empty((), dtype=torch.float32, device=device),
                                  torch.empty((), dtype=torch.int64, device=device))
    return t


def _option(table: dict, value: str, name: str) -> int:
    if value not in table:
        raise ValueError(f"{name} must be one of {tuple(table)}, got {value!r}")
    return table[value]


def _policy(tokens, sequences, log_probs, old, advantages, ref, clip_low, clip_high, dual_clip,
            kl_coef, kl_estimator, reduction, return_metrics, negated):
    """(loss, grad, metrics or None) of flce_policy_loss on ``tokens``."""
    shape, dtype, dev = log_probs.shape, log_probs.dtype, log_probs.device
    estimator = _option(_lib.KL_ESTIMATORS, kl_estimator, "kl_estimator")
    reduce = _option(_lib.TOKEN_REDUCTIONS, reduction, "reduction")
    log_probs, ld = _laid_out(log_probs, shape, dtype, dev, "log_probs")
    if advantages.dtype != torch.float32 or advantages.device != dev:
        raise TypeError(f"advantages must be float32 on {dev}")
    a_shape, ld_adv, per_token = advantages.shape, 0, 0
    if a_shape == shape:
        advantages, ld_adv = _laid_out(advantages, shape, torch.float32, dev, "advantages")
        per_token = 1
    elif a_shape == (sequences,) or a_shape == (sequences, 1):
        advantages = advantages.contiguous()
    else:
        raise ValueError(f"advantages must be [{sequences}], one per sequence, or {tuple(shape)}, "
                         f"one per token; got {tuple(a_shape)}")
    old_at = ref_at = ld_old = ld_ref = 0
    if old is not None:
        old, ld_old = _laid_out(old, shape, dtype, dev, "old_log_probs")
        old_at = old.data_ptr()
    if ref is not None:
        ref, ld_ref = _laid_out(ref, shape, dtype, dev, "ref_log_probs")
        ref_at = ref.data_ptr()
    elif kl_coef:
        raise ValueError("kl_coef needs ref_log_probs")
    grad = _float_like(log_probs, shape, dev)
    ws_at = ws_bytes = 0
    if grad.numel() > _SMALL or sequences > 1024:
        ws = torch.empty(_POLICY_WORKSPACE + 8 * sequences, dtype=torch.uint8, device=dev)
        ws_at, ws_bytes = ws.data_ptr(), ws.numel()
    f0, i0 = _scalar_templates(dev)
    loss, metrics, kl_at, n_at, clipped_at = torch.empty_like(f0), None, 0, 0, 0
    if return_metrics:
        kl_sum, n, clipped = torch.empty_like(f0), torch.empty_like(i0), torch.empty_like(i0)
        kl_at, n_at, clipped_at = kl_sum.data_ptr(), n.data_ptr(), clipped.data_ptr()
        metrics = {"num_tokens": n, "num_clipped": clipped, "kl_sum": kl_sum}
    args = _lib.POLICY_ARGS.pack(
        *tokens, log_probs.data_ptr(), old_at, ref_at, advantages.data_ptr(), loss.data_ptr(),
        grad.data_ptr(), n_at, clipped_at, kl_at, ws_at, ws_bytes, ld, ld_old, ld_ref, ld_adv,
        shape[-1], clip_low, clip_high, dual_clip or 0.0, kl_coef, _DTYPES[dtype], per_token,
        estimator, reduce, negated, 0)
    _lib.check(_lib.policy_loss_raw(args, _stream(dev)), "flce_policy_loss")
    return loss, grad, metrics


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
    ``advantages`` is float32, of the shape of ``log_probs`` or one per
    sequence, ``[sequences]``. (Of a packed batch of as many sequences as
    tokens it is read as one per token; unless a sequence is empty, that is
    the same.)
    ``reduction``: "sum", "mean" over the tokens that count, or
    "sequence_mean", the mean over sequences of each one's mean.

    Returns ``(loss, grad)``, both float32, or ``(loss, grad, metrics)`` with
    the device scalars num_tokens, num_clipped (int64) and kl_sum.
    """
    tokens, sequences, keep = _tokens(log_probs, mask, cu_seqlens, "log_probs")
    loss, grad, metrics = _policy(tokens, sequences, log_probs, old_log_probs, advantages,
                                  ref_log_probs, clip_low, clip_high, dual_clip, kl_coef,
                                  kl_estimator, reduction, return_metrics, 0)
    return (loss, grad, metrics) if return_metrics else (loss, grad)


def _preference(tokens, sequences, log_probs, ref, beta, loss_type, label_smoothing, margin,
                average, negated):
    """(loss, grad, chosen rewards, rejected rewards) of flce_preference_loss on ``tokens``."""
    if sequences % 2:
        raise ValueError("a preference batch needs an even number of sequences: the chosen ones, "
                         "then the rejected ones")
    shape, dtype, dev = log_probs.shape, log_probs.dtype, log_probs.device
    kind = _option(_lib.PREFERENCE_LOSSES, loss_type, "loss_type")
    log_probs, ld = _laid_out(log_probs, shape, dtype, dev, "log_probs")
    ref_at = ld_ref = 0
    if ref is not None:
        ref, ld_ref = _laid_out(ref, shape, dtype, dev, "ref_log_probs")
        ref_at = ref.data_ptr()
    pairs = sequences // 2
    grad = _float_like(log_probs, shape, dev)
    loss = torch.empty_like(_scalar_templates(dev)[0])
    chosen = torch.empty(pairs, dtype=torch.float32, device=dev)
    rejected = torch.empty_like(chosen)

    ws_at = ws_bytes = 0
    if grad.numel() > _SMALL or pairs > 64:
        ws = torch.empty(_PREFERENCE_WORKSPACE + 4 * pairs, dtype=torch.uint8, device=dev)
        ws_at, ws_bytes = ws.data_ptr(), ws.numel()
    args = _lib.PREFERENCE_ARGS.pack(
        *tokens, log_probs.data_ptr(), ref_at, loss.data_ptr(), grad.data_ptr(), chosen.data_ptr(),
        rejected.data_ptr(), ws_at, ws_bytes, ld, ld_ref, shape[-1], beta, label_smoothing, margin, _DTYPES[dtype], kind,
        1 if average else 0, negated)
    _lib.check(_lib.preference_loss_raw(args, _stream(dev)), "flce_preference_loss")
    return loss, grad, chosen, rejected


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
    tokens, sequences, keep = _tokens(log_probs, mask, cu_seqlens, "log_probs")
    return _preference(tokens, sequences, log_probs, ref_log_probs, beta, loss_type,
                       label_smoothing, margin, average, 0)


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
        tokens, sequences, keep = _label_tokens(nll, labels, ignore_index, cu_seqlens)
        loss, grad, m = _policy(tokens, sequences, nll, old_log_probs, advantages, ref_log_probs,
                                clip_low, clip_high, dual_clip, kl_coef, kl_estimator, reduction,
                                True, 1)
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
        return _preference(tokens, sequences, nll, ref_log_probs, beta, loss_type, label_smoothing,
                           margin, average, 1)
    return _FusedLinear.apply(hidden, weight, bias, targets, (ignore_index, logit_scale, softcap), fn)
