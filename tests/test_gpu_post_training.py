"""Policy and preference losses against the fp64 oracle.

Tolerances, before any run. The inputs are the same numbers on both sides. A
token's terms are a handful of fp32 operations with exp and expm1 within 2 ulp,
so each is within 16 x 2^-24 = 1e-6 of the sum of the magnitudes it is made
of; sums add at most 32 terms in fp32 before they go on in fp64, another
32 x 2^-24 = 2e-6. So 4e-6 of the sum of magnitudes bounds the loss, the KL sum
and, token by token, the gradient. The preference loss is a smooth function
of each pair's log-ratio difference h, whose error is at most 4e-6 of the
magnitudes summed: its bound is the spread of the oracle over that interval.
Counts are exact, so inputs keep the log ratios 1e-6 away from the clips.
"""
import numpy as np
import pytest
import torch

import oracle.post_training_oracle as ref_ops
from linear_cross_entropy_tiled_gb300 import (
    _lib, fused_linear_policy_loss, fused_linear_preference_loss, policy_loss, policy_loss_and_grad,
    preference_loss, preference_loss_and_grad)

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
TOL = 4e-6
CLIPS = dict(clip_low=0.2, clip_high=0.28)


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy().ravel()


class Batch:
    """A padded or packed batch with hostile values where tokens do not count."""

    def __init__(self, layout, shape, dtype="f32", seed=0, mask="lengths", stride=None, old=True,
                 ref=True, offset=0, gap=(0, 0)):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.cu = None
        if layout == "packed":
            cu = np.concatenate([[0], np.cumsum(shape)]) + gap[0]
            n = int(cu[-1]) + gap[1]
            self.cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
            full, S = (n,), len(shape)
            spans = [np.arange(a, b) for a, b in zip(cu, cu[1:])]
        else:
            full, (S, T) = shape, shape
            spans = [np.arange(s * T, (s + 1) * T) for s in range(S)]
        n = int(np.prod(full))
        keep = np.ones(n, bool)
        if mask == "lengths":
            keep = np.random.default_rng(seed).random(n) < 0.7
            for s in range(S // 2, S, 5):
                keep[spans[s]] = False          # sequences without a token that counts
        elif mask == "none_counts":
            keep[:] = False
        self.S, self.full, self.spans = S, full, spans
        self.cut = [c[keep[c]] for c in spans]
        self.row = np.zeros(n, np.int64)
        for s, c in enumerate(spans):
            self.row[c] = s
        counted = np.zeros(n, bool)
        for c in self.cut:
            counted[c] = True
        hostile = torch.tensor(~counted, device="cuda").view(full)

        def tensor(x, dt, bad):
            x = x.to(dt)
            if bad is not None:
                x = torch.where(hostile, torch.tensor(bad, dtype=dt, device="cuda"), x)
            if stride and len(full) == 2:      # rows of a wider buffer, starting off its alignment
                wide = torch.full((S, T + stride), 7, dtype=dt, device="cuda")
                wide[:, offset:offset + T] = x
                return wide[:, offset:offset + T]
            if offset:                          # a contiguous tensor off its alignment
                flat = torch.empty(n + offset, dtype=dt, device="cuda")[offset:]
                return flat.copy_(x.reshape(-1)).view(full)
            return x.contiguous()

        def randn():
            return torch.randn(full, device="cuda", generator=g)
        dt = DT[dtype]
        lp = -(randn().square() * 0.7 + 0.01)
        # the log ratios keep away from log 0.8, log 1.28 and log 3 (16-bit types: their own grid)
        d = 0.4 * randn()
        for edge in np.log([0.8, 1.28, 3.0]):
            d = torch.where((d - edge).abs() < 1e-3, d + 4e-3, d)
        self.lp = tensor(lp, dt, float("-inf"))
        self.old = tensor(lp - d, dt, float("nan")) if old else None
        self.ref = tensor(lp + 0.3 * randn(), dt, float("inf")) if ref else None
        self.adv_token = tensor(randn() + 0.3, torch.float32, float("nan"))
        self.adv_seq = torch.randn(S, device="cuda", generator=g)
        if S > 2:
            self.adv_seq[2] = 0.0
        if mask is None:
            self.mask = None
        else:
            self.mask = tensor(torch.tensor(keep, device="cuda").view(full), torch.bool, None)


LAYOUTS = [
    ("padded", (1, 1), dict(mask=None)),
    ("padded", (2, 1), {}),
    ("padded", (4, 256), {}),
    ("padded", (7, 1001), {}),
    ("padded", (6, 515), dict(stride=13, offset=3)),
    ("padded", (6, 512), dict(stride=64)),
    ("padded", (600, 3), {}),
    ("padded", (6, 301), dict(offset=1)),
    ("padded", (2, 40000), {}),
    ("padded", (4, 33), dict(mask="none_counts")),
    ("packed", [5], dict(mask=None)),
    ("packed", [0, 3, 0, 0, 1000, 1, 0, 777], dict(mask=None)),
    ("packed", [130, 1, 0, 2049, 64, 33], {}),
    ("packed", [700, 11, 30, 500], dict(gap=(3, 6))),
    ("packed", [1] * 300 + [5] * 300, {}),
    ("packed", [30001, 12345], dict(offset=1)),
    ("packed", [0, 0], dict(mask=None)),
]


def check_policy(b, got, adv, kl, est, red, dual, tokens_are=None):
    loss, grad, m = got
    r = ref_ops.policy(b.cut, f64(b.lp), f64(b.old), f64(b.ref), adv, 0.2, 0.28, dual, kl, est, red)
    want, wgrad, n, clipped, kl_sum, total, size, kl_size = r
    g = f64(grad)
    assert grad.dtype == torch.float32 and grad.shape == b.full and loss.shape == ()
    assert int(m["num_tokens"]) == n and int(m["num_clipped"]) == clipped
    if np.isnan(want):
        assert np.isnan(loss.item())
    else:
        assert abs(loss.item() - want) <= TOL * total + 1e-30, (loss.item(), want, total)
    assert (np.abs(g - wgrad) <= TOL * size).all(), np.abs(g - wgrad).max()
    assert abs(m["kl_sum"].item() - kl_sum) <= TOL * kl_size


@pytest.mark.parametrize("layout,shape,opts", LAYOUTS)
@pytest.mark.parametrize("red", ["sum", "mean", "sequence_mean"])
def test_policy_layouts(layout, shape, opts, red):
    b = Batch(layout, shape, seed=1, **opts)
    got = policy_loss_and_grad(b.lp, b.old, b.adv_seq, ref_log_probs=b.ref, mask=b.mask,
                               cu_seqlens=b.cu, kl_coef=0.05, reduction=red, return_metrics=True,
                               **CLIPS)
    adv = f64(b.adv_seq)[b.row] if b.S else np.zeros(0)
    check_policy(b, got, adv, 0.05, "k3", red, 0.0)
    b2 = policy_loss_and_grad(b.lp, b.old, b.adv_token, ref_log_probs=b.ref, mask=b.mask,
                              cu_seqlens=b.cu, kl_coef=0.05, reduction=red, return_metrics=True,
                              **CLIPS)
    check_policy(b, b2, f64(b.adv_token), 0.05, "k3", red, 0.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("est", ["k1", "k2", "k3", None])
@pytest.mark.parametrize("dual", [0.0, 3.0])
@pytest.mark.parametrize("layout,shape,opts", [("padded", (5, 777), dict(stride=5, offset=1)),
                                               ("packed", [400, 0, 1, 900], dict(offset=1))])
def test_policy_types_and_terms(dtype, est, dual, layout, shape, opts):
    b = Batch(layout, shape, dtype, seed=2, ref=est is not None, **opts)
    kl = 0.1 if est else 0.0
    got = policy_loss_and_grad(b.lp, b.old, b.adv_token, ref_log_probs=b.ref, mask=b.mask,
                               cu_seqlens=b.cu, kl_coef=kl, kl_estimator=est or "k3",
                               dual_clip=dual or None, return_metrics=True, **CLIPS)
    check_policy(b, got, f64(b.adv_token), kl, est, "mean", dual)


def test_policy_on_its_own_samples():
    """Without old log probs the ratio is 1: the gradient is -A w."""
    b = Batch("padded", (4, 100), seed=3, old=False, ref=False)
    loss, grad, m = policy_loss_and_grad(b.lp, None, b.adv_seq, mask=b.mask, return_metrics=True)
    check_policy(b, (loss, grad, m), f64(b.adv_seq)[b.row], 0.0, "k3", "mean", 0.0)
    assert int(m["num_clipped"]) == 0


def test_policy_extreme_log_ratios():
    """exp overflow: where the clip takes the term, loss and gradient stay finite; advantage 0 gives 0."""
    lp = torch.tensor([[-0.5, -0.5, -0.5, -200.0, float("-inf")]], device="cuda")
    old = torch.tensor([[-300.0, -300.0, -300.0, -0.5, -1.0]], device="cuda")
    adv = torch.tensor([[1.0, 0.0, -1.0, -1.0, -2.0]], device="cuda")
    loss, grad, m = policy_loss_and_grad(lp, old, adv, dual_clip=3.0, reduction="sum",
                                         return_metrics=True)
    # -1.2 (clipped above), 0, dual clip 3, then -(0.8 x -1) and -(0.8 x -2), clipped below
    assert loss.item() == pytest.approx(-1.2 + 3.0 + 0.8 + 1.6, rel=1e-6)
    assert (grad == 0).all() and int(m["num_clipped"]) == 4
    lp[0, 3] = float("nan")
    loss, grad = policy_loss_and_grad(lp, old, adv, reduction="sum")
    assert loss.isnan() and grad[0, 3].isnan() and (grad[0, :2] == 0).all()
    assert grad[0, 2] == float("inf")      # without the dual clip nothing bounds -A r for A < 0


@pytest.mark.parametrize("shape", [(0, 5), (3, 0), (0, 0)])
def test_empty_batches(shape):
    z = torch.empty(shape, device="cuda")
    for red, want in (("sum", 0.0), ("mean", np.nan),
                      ("sequence_mean", np.nan if shape[0] == 0 else 0.0)):
        loss, grad, m = policy_loss_and_grad(z, z, torch.ones(shape[0], device="cuda"),
                                             reduction=red, return_metrics=True)
        np.testing.assert_equal(loss.item(), want)
        assert grad.shape == shape and int(m["num_tokens"]) == 0
    if shape[0] == 0:
        loss, grad, c, r = preference_loss_and_grad(z, z)
        assert loss.isnan() and c.numel() == r.numel() == 0
    cu = torch.zeros(1, dtype=torch.int32, device="cuda")
    loss, grad = policy_loss_and_grad(torch.ones(9, device="cuda"), None, torch.ones(9, device="cuda"),
                                      cu_seqlens=cu, reduction="sum")
    assert loss.item() == 0 and (grad == 0).all()    # no sequences: no token counts


def check_preference(b, got, beta, margin, kind, smoothing, average):
    loss, grad, chosen, rejected = got
    lp, ref = f64(b.lp), f64(b.ref)
    want, wgrad, wc, wr, slack = ref_ops.preference(b.cut, lp, ref, beta, margin, kind, smoothing,
                                                    average)
    pairs = b.S // 2
    spread, gspread = np.zeros(pairs), np.zeros(pairs)
    slope = np.zeros(pairs)
    for i in range(pairs):
        h = (wc[i] - wr[i]) / beta
        at = [ref_ops.pair_loss(h + k * TOL * slack[i], beta, margin, kind, smoothing)
              for k in (-1, 0, 1)]
        spread[i] = max(abs(at[k][0] - at[1][0]) for k in (0, 2)) + TOL * abs(at[1][0])
        gspread[i] = max(abs(at[k][1] - at[1][1]) for k in (0, 2)) + TOL * (abs(at[1][1]) + beta)
        slope[i] = at[1][1]
    assert abs(loss.item() - want) <= spread.mean() + 1e-7
    np.testing.assert_array_less(np.abs(f64(chosen) - wc), beta * TOL * slack + 1e-30)
    np.testing.assert_array_less(np.abs(f64(rejected) - wr), beta * TOL * slack + 1e-30)
    g, bound = f64(grad), np.zeros(lp.size)
    for i in range(pairs):
        for c in (b.cut[i], b.cut[pairs + i]):
            bound[c] = gspread[i] / pairs / (max(1, len(c)) if average else 1)
    assert (np.abs(g - wgrad) <= bound).all()
    assert grad.shape == b.full and grad.dtype == torch.float32


PAIRED = [
    ("padded", (2, 1), dict(mask=None)),
    ("padded", (8, 256), {}),
    ("padded", (6, 515), dict(stride=13, offset=3)),
    ("padded", (10, 1024), dict(stride=64)),
    ("padded", (600, 3), {}),
    ("padded", (2, 40001), dict(offset=1)),
    ("padded", (4, 33), dict(mask="none_counts")),
    ("packed", [0, 3, 1000, 1, 0, 777], dict(mask=None)),
    ("packed", [130, 1, 0, 2049, 64, 33], {}),
    ("packed", [700, 11, 30, 500], dict(gap=(3, 6))),
    ("packed", [30001, 12345], dict(offset=1, mask=None)),
    ("packed", [3] * 700, {}),
]


@pytest.mark.parametrize("layout,shape,opts", PAIRED)
@pytest.mark.parametrize("average", [False, True])
def test_preference_layouts(layout, shape, opts, average):
    b = Batch(layout, shape, seed=4, old=False, **opts)
    got = preference_loss_and_grad(b.lp, b.ref, mask=b.mask, cu_seqlens=b.cu, beta=0.1, margin=0.2,
                                   average=average)
    check_preference(b, got, 0.1, 0.2, "sigmoid", 0.0, average)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("kind,smoothing", [("sigmoid", 0.0), ("sigmoid", 0.1), ("hinge", 0.0),
                                            ("ipo", 0.0)])
@pytest.mark.parametrize("ref", [True, False])
def test_preference_types_and_losses(dtype, kind, smoothing, ref):
    b = Batch("padded", (12, 333), dtype, seed=5, old=False, ref=ref, stride=3)
    got = preference_loss_and_grad(b.lp, b.ref, mask=b.mask, beta=0.3, loss_type=kind,
                                   label_smoothing=smoothing, margin=0.1, average=not ref)
    check_preference(b, got, 0.3, 0.1, kind, smoothing, not ref)


def test_preference_saturates():
    """Log ratios of hundreds: the loss is linear or 0, and no exponential overflows."""
    lp = torch.tensor([[-1.0], [-1e4]], device="cuda")
    for a, want, slope in ((lp, 0.0, 0.0), (lp.flip(0), 9999.0, -1.0)):
        loss, grad, _, _ = preference_loss_and_grad(a, beta=1.0)
        assert loss.item() == pytest.approx(want, rel=1e-6)
        assert grad[0, 0].item() == pytest.approx(slope, abs=1e-30)


@pytest.mark.parametrize("op", ["policy", "preference"])
def test_gradient_against_differences(op):
    """Central differences of the library's own loss, away from the kinks."""
    b = Batch("padded", (4, 6), seed=6)

    def f(lp):
        if op == "policy":
            return policy_loss_and_grad(lp, b.old, b.adv_seq, ref_log_probs=b.ref, mask=b.mask,
                                        kl_coef=0.2, reduction="sequence_mean", **CLIPS)
        return preference_loss_and_grad(lp, b.ref, mask=b.mask, beta=0.5)[:2]
    grad = f(b.lp)[1]
    # d is 1e-3 away from the clips; fp32 loss of about 1 with h = 5e-4: error 1e-7 / 5e-4 = 2e-4
    h = 5e-4
    for i in np.concatenate([c[:2] for c in b.cut]):
        lp = b.lp.clone()
        lp.view(-1)[i] += h
        up = f(lp)[0].double()
        lp.view(-1)[i] -= 2 * h
        down = f(lp)[0].double()
        assert ((up - down) / (2 * h)).item() == pytest.approx(grad.view(-1)[i].item(), abs=1e-3)


def test_autograd_forms_scale_by_the_upstream_gradient():
    b = Batch("padded", (4, 50), "bf16", seed=7)
    kw = dict(ref_log_probs=b.ref, mask=b.mask, kl_coef=0.1)
    lp = b.lp.clone().requires_grad_(True)
    loss, m = policy_loss(lp, b.old, b.adv_seq, return_metrics=True, **kw)
    (3 * loss).backward(retain_graph=True)
    want_loss, want, wm = policy_loss_and_grad(b.lp, b.old, b.adv_seq, return_metrics=True, **kw)
    assert loss.item() == want_loss.item() and int(m["num_tokens"]) == int(wm["num_tokens"])
    assert lp.grad.dtype == torch.bfloat16 and torch.equal(lp.grad, (3 * want).bfloat16())
    lp.grad = None
    loss.backward()
    assert torch.equal(lp.grad, want.bfloat16())
    lp = b.lp.clone().requires_grad_(True)
    loss, chosen, rejected = preference_loss(lp, b.ref, mask=b.mask)
    loss.backward()
    _, want, wc, _ = preference_loss_and_grad(b.lp, b.ref, mask=b.mask)
    assert torch.equal(lp.grad, want.bfloat16()) and torch.equal(chosen, wc)
    assert not chosen.requires_grad and not rejected.requires_grad


@pytest.mark.parametrize("op", ["policy", "preference"])
def test_same_bits_again_and_on_another_stream(op):
    b = Batch("padded", (64, 3001), seed=8)

    def f():
        if op == "policy":
            return policy_loss_and_grad(b.lp, b.old, b.adv_seq, ref_log_probs=b.ref, mask=b.mask,
                                        kl_coef=0.1)
        return preference_loss_and_grad(b.lp, b.ref, mask=b.mask)
    first = f()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = f()
    torch.cuda.current_stream().wait_stream(side)
    for x, y, z in zip(first, f(), other):
        assert torch.equal(x, y) and torch.equal(x, z)


def test_strides_past_32_bits():
    """Rows 2^31 + 24 elements apart: offsets pass 32 bits, in elements and in bytes."""
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    T, ld = 1000, (1 << 31) + 24
    b = Batch("padded", (4, T), "bf16", seed=9, mask="lengths")
    wide = torch.empty(3 * ld + T, dtype=torch.bfloat16, device="cuda")
    lp = wide.as_strided((4, T), (ld, 1))
    lp.copy_(b.lp)
    for f in (lambda x: policy_loss_and_grad(x, b.old, b.adv_seq, mask=b.mask),
              lambda x: preference_loss_and_grad(x, b.ref, mask=b.mask)):
        for x, y in zip(f(lp), f(b.lp)):
            assert torch.equal(x, y)


def _head(dtype, S, T, H, V, seed, bias=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DT[dtype]
    h = torch.randn(S, T, H, device="cuda", generator=g).to(dt).requires_grad_(True)
    w = (torch.randn(V, H, device="cuda", generator=g) / H ** 0.5).to(dt).requires_grad_(True)
    bb = (0.3 * torch.randn(V, device="cuda", generator=g)).to(dt).requires_grad_(True) if bias else None
    t = torch.randint(0, V, (S, T), device="cuda", generator=g)
    t[torch.rand(S, T, device="cuda", generator=g) < 0.25] = -100
    t[S // 2] = -100
    return h, w, bb, t


@pytest.mark.parametrize("op", ["policy", "preference"])
@pytest.mark.parametrize("dtype,packed", [("bf16", False), ("f16", False), ("f32", False),
                                          ("bf16", True)])
def test_fused_linear_losses(op, dtype, packed):
    """From hidden states: loss and gradients against fp64 autograd through the explicit logits.

    The log probs come from 16-bit products with fp32 accumulation, and their
    gradients are rounded as the library's cross-entropy gradients are, so the
    bars are that loss's own: 2e-2 of the largest gradient and cosine 0.9999
    (16-bit), 1e-4 and 0.999999 (fp32).
    """
    S, T, H, V = 6, 40, 64, 333
    h, w, b, t = _head(dtype, S, T, H, V, 11, bias=True)
    cu = None
    lens = [T] * S
    if packed:
        lens = [50, 0, 70, 30, 60, 30]
        cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
        h = h.detach().view(-1, H).clone().requires_grad_(True)
        t = t.view(-1)
    hd, wd, bd = (x.detach().double().requires_grad_(True) for x in (h, w, b))
    z = (hd.reshape(-1, H) @ wd.T + bd) * 0.8
    valid = t.reshape(-1) != -100
    lp = torch.log_softmax(z, 1).gather(1, t.reshape(-1, 1).clamp(min=0))[:, 0]
    g = torch.Generator(device="cuda").manual_seed(12)
    old = (lp.detach() + 0.05 * torch.randn(lp.shape, device="cuda", generator=g)).float()
    ref = (lp.detach() + 0.1 * torch.randn(lp.shape, device="cuda", generator=g)).float()
    adv = torch.randn(S, device="cuda", generator=g)
    row = torch.repeat_interleave(torch.arange(S, device="cuda"), torch.tensor(lens, device="cuda"))
    shape = t.shape
    if op == "policy":
        r, a, e = torch.exp(lp - old.double()), adv[row].double(), ref.double() - lp
        tok = -torch.minimum(r * a, r.clamp(0.8, 1.28) * a) + 0.1 * (torch.exp(e) - e - 1)
        want = (tok * valid).sum() / valid.sum()
        got, m = fused_linear_policy_loss(h, w, t, old.view(shape), adv, bias=b, logit_scale=0.8,
                                          ref_log_probs=ref.view(shape), cu_seqlens=cu, kl_coef=0.1,
                                          return_metrics=True, **CLIPS)
        assert int(m["num_tokens"]) == int(valid.sum())
    else:
        s = torch.zeros(S, dtype=torch.float64, device="cuda").index_add(
            0, row, (lp - ref.double()) * valid)
        zz = 0.5 * (s[:S // 2] - s[S // 2:])
        want = -torch.nn.functional.logsigmoid(zz).mean()
        got, chosen, rejected = fused_linear_preference_loss(h, w, t, ref.view(shape), bias=b,
                                                             logit_scale=0.8, cu_seqlens=cu, beta=0.5)
        bar = 1e-4 if dtype == "f32" else 2e-2
        assert (chosen.double() - 0.5 * s[:S // 2]).abs().max() <= bar * (1 + s.abs().max())
    (2 * got).backward()
    (2 * want).backward()
    assert got.item() == pytest.approx(want.item(), rel=1e-5 if dtype == "f32" else 2e-3, abs=1e-4)
    tol, cos = (1e-4, 0.999999) if dtype == "f32" else (2e-2, 0.9999)
    for x, y in ((h, hd), (w, wd), (b, bd)):
        x, y = x.grad.double().reshape(-1), y.grad.reshape(-1)
        assert (x - y).abs().max() <= tol * y.abs().max()
        assert torch.dot(x, y) / (x.norm() * y.norm()) >= cos
