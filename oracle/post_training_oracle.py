"""The post-training operators in fp64 numpy, from their formulas, one sequence or element block at a time.

Nothing here shares code with the library. A batch is a list of index arrays
``cut``: cut[s] holds the flat indices of sequence s's tokens that count.
"""
from __future__ import annotations

import numpy as np


def policy(cut, lp, old, ref, adv, clip_low, clip_high, dual, kl_coef, kl_estimator, reduction):
    """adv is per token (flat). Returns (loss, grad, num_tokens, num_clipped, kl_sum, and the sums of
    magnitudes behind loss, each token's gradient, and kl_sum)."""
    lp = np.asarray(lp, np.float64).ravel()
    grad, size = np.zeros(lp.size), np.zeros(lp.size)
    n = sum(len(c) for c in cut)
    loss = kl_sum = total = kl_size = 0.0
    clipped = 0
    for c in cut:
        if len(c) == 0:
            continue
        with np.errstate(divide="ignore"):
            w = {"sum": 1.0, "mean": 1.0 / n, "sequence_mean": 1.0 / (len(cut) * len(c))}[reduction]
        a = adv[c]
        r = np.exp(lp[c] - old[c]) if old is not None else np.ones(len(c))
        ratio_cut = np.clip(r, 1 - clip_low, 1 + clip_high)
        pg = -np.minimum(np.where(a == 0, 0, a * r), a * ratio_cut)
        off = ((a > 0) & (r > 1 + clip_high)) | ((a < 0) & (r < 1 - clip_low))
        if dual:
            over = (a < 0) & (r > dual)
            pg = np.where(over, -dual * a, pg)
            off = off | over
        g = np.where(off | (a == 0), 0.0, -a * r)
        big = np.abs(pg) + np.abs(g)
        if kl_coef:
            x = ref[c] - lp[c]
            if kl_estimator == "k1":
                kl, dkl = -x, np.ones_like(x)
            elif kl_estimator == "k2":
                kl, dkl = x * x / 2, -x
            else:
                kl, dkl = np.exp(x) - x - 1, 1 - np.exp(x)
            pg, g = pg + kl_coef * kl, g + kl_coef * dkl
            big = big + abs(kl_coef) * (np.abs(kl) + np.abs(dkl) + np.abs(x))
            kl_sum += kl.sum()
            kl_size += (np.abs(kl) + np.abs(x)).sum()
        loss += w * pg.sum()
        total += w * big.sum()
        grad[c], size[c] = w * g, w * big
        clipped += int(off.sum())
    if (reduction == "mean" and n == 0) or (reduction == "sequence_mean" and not cut):
        loss = np.nan
    return loss, grad, n, clipped, kl_sum, total, size, kl_size


def pair_loss(h, beta, margin, kind, smoothing):
    """(loss, d loss / d h) of one pair with log-ratio difference h."""
    z = beta * h - margin
    if kind == "sigmoid":
        return ((1 - smoothing) * np.logaddexp(0, -z) + smoothing * np.logaddexp(0, z),
                beta * (smoothing - np.exp(-np.logaddexp(0, z))))
    if kind == "hinge":
        return max(0.0, 1 - z), -beta if z < 1 else 0.0
    u = z / beta - 0.5 / beta
    return u * u, 2 * u


def preference(cut, lp, ref, beta, margin, kind, smoothing, average):
    """Returns (loss, grad, chosen, rejected, slack) with slack[b] = sum |terms| behind pair b's h."""
    lp = np.asarray(lp, np.float64).ravel()
    grad = np.zeros(lp.size)
    pairs = len(cut) // 2
    s, size, weight = np.zeros(2 * pairs), np.zeros(2 * pairs), np.ones(2 * pairs)
    for i, c in enumerate(cut):
        v = lp[c] - ref[c] if ref is not None else lp[c]
        if average:
            weight[i] = 1.0 / max(1, len(c))
        s[i], size[i] = v.sum() * weight[i], np.abs(v).sum() * weight[i]
    losses = []
    for b in range(pairs):
        loss, slope = pair_loss(s[b] - s[pairs + b], beta, margin, kind, smoothing)
        losses.append(loss)
        grad[cut[b]] = slope * weight[b] / pairs
        grad[cut[pairs + b]] = -slope * weight[pairs + b] / pairs
    loss = np.mean(losses) if pairs else np.nan
    return loss, grad, beta * s[:pairs], beta * s[pairs:], size[:pairs] + size[pairs:]


# ------------------------------------------------------------------ AdamW
def e4m3_values():
    """Value of each code 0..0x7E: 4 exponent bits (bias 7), 3 mantissa bits; 0x7F is NaN."""
    c = np.arange(0x7F)
    e, m = c >> 3, c & 7
    return np.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * 2.0 ** (e - 7.0))


def pair_bits(total, first_block, seed, step):
    """16 random bits for each of `total` elements, the first of them first in block first_block."""
    M, C1, C2 = 0xFFFFFFFF, 0x9E3779B1, 0x85A308D3
    key = (seed * C1 + step * C2) & M
    key ^= key >> 16
    key = key * C1 & M
    i = np.arange(total, dtype=np.uint64) + np.uint64(first_block * 256)
    x = ((i >> np.uint64(1)) ^ np.uint64(key)) & np.uint64(M)
    x = x * np.uint64(C1) & np.uint64(M)
    x ^= x >> np.uint64(15)
    x = x * np.uint64(C2) & np.uint64(M)
    x ^= x >> np.uint64(13)
    x = x * np.uint64(C1) & np.uint64(M)
    x ^= x >> np.uint64(16)
    return np.where(i & np.uint64(1), x >> np.uint64(16), x & np.uint64(0xFFFF)).astype(np.int64)


def block_scale(x):
    """(scale of each 256-element block, x over its block's scale)."""
    n = x.size
    y = np.zeros(-(-n // 256) * 256)
    y[:n] = x
    y = y.reshape(-1, 256)
    top = np.abs(y).max(1)
    top = np.where(top < 2.0 ** -100, 0, top)
    with np.errstate(divide="ignore", invalid="ignore"):
        z = np.where(top[:, None] > 0, y * (448 / top[:, None]), 0)
    return top / 448, z.reshape(-1)[:n]


def stochastic_code(x, bits):
    """e4m3 code of x in [0, 448]: the neighbour below, or above where the 16 random bits say so."""
    values = e4m3_values()
    below = np.clip(np.searchsorted(values, x, side="right") - 1, 0, 0x7E)
    above = np.minimum(below + 1, 0x7E)
    with np.errstate(divide="ignore", invalid="ignore"):
        part = np.where(above > below, (x - values[below]) / (values[above] - values[below]), 0)
    # the top 20 bits of the fraction plus (16 random bits, then 8) reach 2^20
    code = np.where(np.floor(part * 2 ** 20) + bits * 16 + 8 >= 2 ** 20, above, below)
    return np.where((x > 0) & (code == 0), 1, code)


def adamw(p, g, m, v, *, step, lr, beta1, beta2, eps, weight_decay, grad_scale=1.0):
    """Returns (p, m, v, update size, sum of magnitudes behind m)."""
    p, g, m, v = (np.asarray(t, np.float64).ravel() for t in (p, g, m, v))
    g = g * grad_scale
    size = beta1 * np.abs(m) + (1 - beta1) * np.abs(g)
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    denom = np.sqrt(v / (1 - beta2 ** step)) + eps
    alpha = lr / (1 - beta1 ** step)
    return p - lr * weight_decay * p - alpha * m / denom, m, v, alpha * size / denom, size
