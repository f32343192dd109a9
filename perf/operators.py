"""Cases of the post-training operators: clipped policy loss, preference loss, and the AdamW step.

Each case is one call that a training program makes once per step. `run` computes it either in its
plain form (elementary torch operations in fp32, rounded once at the end) or through the package.
The sizes follow this package's own workloads (vocabularies of 32000 and 128256, hidden 4096, bf16)
and the token batches that go with them, from a debugging batch to a full rollout.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
BLOCK = 256          # elements that share one scale of the 8-bit optimiser state
M32 = 0xFFFFFFFF
C1, C2 = 0x9E3779B1, 0x85A308D3


def listed():
    return [
        # A debugging or per-microbatch call: 8 short responses. Latency is all that counts.
        dict(name="policy_small", op="policy", layout="padded", rows=8, cols=128, dtype="f32",
             adv="sequence", reduction="mean", kl=0.0, kl_estimator="k3", dual=0.0),
        # One rollout batch of a group-relative policy step: fp32 log probs as the forward gives them.
        dict(name="policy_rollout", op="policy", layout="padded", rows=256, cols=2048, dtype="f32",
             adv="sequence", reduction="sequence_mean", kl=0.04, kl_estimator="k3", dual=0.0),
        # Packed responses of odd lengths kept in bf16 between the stages, per-token advantages.
        dict(name="policy_packed", op="policy", layout="packed", rows=97, cols=1801, dtype="bf16",
             adv="token", reduction="mean", kl=0.01, kl_estimator="k2", dual=3.0),
        # The whole batch of a long-context step on one device.
        dict(name="policy_large", op="policy", layout="padded", rows=1024, cols=8192, dtype="f32",
             adv="token", reduction="mean", kl=0.04, kl_estimator="k3", dual=0.0),
        # A microbatch of 4 pairs.
        dict(name="preference_small", op="preference", layout="padded", rows=4, cols=256,
             dtype="f32", loss="sigmoid", smoothing=0.0, average=False, ref=True),
        # An ordinary preference batch; an odd length after the shift by one token.
        dict(name="preference_batch", op="preference", layout="padded", rows=64, cols=2047,
             dtype="f32", loss="sigmoid", smoothing=0.1, average=False, ref=True),
        # Two pairs of long documents, packed, log probs in bf16.
        dict(name="preference_long", op="preference", layout="packed", rows=2, cols=65537,
             dtype="bf16", loss="ipo", smoothing=0.0, average=True, ref=True),
        # The whole batch of a long-context step on one device.
        dict(name="preference_large", op="preference", layout="padded", rows=512, cols=8192,
             dtype="f32", loss="sigmoid", smoothing=0.0, average=False, ref=True),
        # Norm weights and a small fp32 head: launch latency counts.
        dict(name="adamw_small", op="adamw", vocab=512, hidden=128, small=11, dtype="f32",
             grad="f32", bits=32, master=False),
        # Adapters: many odd-sized 16-bit tensors beside a middling head, 8-bit states.
        dict(name="adamw_many", op="adamw", vocab=8191, hidden=1001, small=160, dtype="f16",
             grad="f16", bits=8, master=False),
        # A 32000-word head in bf16 with an fp32 master copy, fp32 states and fp32 gradients.
        dict(name="adamw_head", op="adamw", vocab=32000, hidden=4096, small=8, dtype="bf16",
             grad="f32", bits=32, master=True),
        # The 128256-word head in bf16 with 8-bit states.
        dict(name="adamw_head_8bit", op="adamw", vocab=128256, hidden=4096, small=8, dtype="bf16",
             grad="bf16", bits=8, master=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["policy", "preference", "adamw"])
    if op == "adamw":
        total = _log(rng, 1 << 13, 1 << 28)
        hidden = min(_log(rng, 16, 8192), total)
        bits = rng.choice([8, 32])
        dtype = rng.choice(["f32", "bf16", "f16"])
        return dict(op=op, vocab=max(1, total // hidden), hidden=hidden, small=rng.randint(0, 200),
                    dtype=dtype, grad=rng.choice([dtype, "f32"]), bits=bits,
                    master=dtype != "f32" and rng.random() < 0.5)
    tokens = _log(rng, 1 << 9, 1 << 23)
    cols = min(_log(rng, max(1, tokens >> 13), 1 << 16), tokens)
    layout = rng.choice(["padded", "packed"])
    dtype = rng.choice(["f32", "bf16", "f16"])
    if op == "policy":
        return dict(op=op, layout=layout, rows=max(1, tokens // cols), cols=cols, dtype=dtype,
                    adv=rng.choice(["sequence", "token"]),
                    reduction=rng.choice(["mean", "sequence_mean", "sum"]),
                    kl=rng.choice([0.0, round(rng.uniform(0.001, 0.1), 4)]),
                    kl_estimator=rng.choice(["k1", "k2", "k3"]), dual=rng.choice([0.0, 3.0]))
    ref = rng.random() < 0.7
    return dict(op=op, layout=layout, rows=max(1, tokens // (2 * cols)), cols=cols, dtype=dtype,
                loss=rng.choice(["sigmoid", "hinge", "ipo"]), smoothing=rng.choice([0.0, 0.1]),
                average=(not ref) or rng.random() < 0.5, ref=ref)


# ------------------------------------------------------------------ sizes
CLIP_LOW, CLIP_HIGH = 0.2, 0.28
BETA, MARGIN = 0.1, 0.25


def _lengths(case, seqs):
    """Lengths of packed sequences: part of the case, from 1 token (none at all for one of several)."""
    r = random.Random(seqs * 1000003 + case["cols"])
    n = [r.randint(max(1, case["cols"] // 4), case["cols"]) for _ in range(seqs)]
    if seqs >= 4:
        n[seqs // 2] = 0
    return n


def _small_sizes(case):
    r = random.Random(case["vocab"] * 31 + case["hidden"])
    return [_log(r, 1, 16 * case["hidden"]) for _ in range(case["small"])]


def _sizes(case):
    return [case["vocab"] * case["hidden"]] + _small_sizes(case)


def work(case):
    if case["op"] == "adamw":
        n = sum(_sizes(case))
        b = BYTES[case["grad"]] + BYTES[case["dtype"]] * (1 if case["master"] else 2)
        b += 8 if case["master"] else 0
        b += 16 if case["bits"] == 32 else 4 + 16 / BLOCK
        return {"bytes": n * b, "flops": 16 * n}
    e = BYTES[case["dtype"]]
    seqs = case["rows"] * (2 if case["op"] == "preference" else 1)
    if case["layout"] == "packed":
        tokens = sum(_lengths(case, seqs))
        valid = tokens
        b = tokens * 4
    else:
        tokens = seqs * case["cols"]
        valid = 0.625 * tokens          # mean length of _padded_mask
        b = tokens * (4 + 1)
    if case["op"] == "policy":
        b += valid * (e * (3 if case["kl"] else 2) + (4 if case["adv"] == "token" else 0))
        return {"bytes": b, "flops": 20 * valid}
    return {"bytes": b + valid * e * (2 if case["ref"] else 1), "flops": 3 * valid}


# ------------------------------------------------------------------ inputs
def _padded_mask(seqs, cols, gen):
    """Right-padded responses: lengths from a quarter of the row up; one row of several is empty."""
    n = ((0.25 + 0.75 * torch.rand(seqs, device=DEV, generator=gen)) * cols).ceil()
    if seqs >= 4:
        n[seqs // 2] = 0
    return torch.arange(cols, device=DEV) < n[:, None]


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed) * 2 + 1)

    def randn(*shape):
        return torch.randn(*shape, device=DEV, generator=gen)

    if case["op"] == "adamw":
        return _prepare_adamw(case, seed, randn, gen)
    dt = DT[case["dtype"]]
    seqs = case["rows"] * (2 if case["op"] == "preference" else 1)
    s = {"case": case, "mask": None, "cu": None}
    if case["layout"] == "packed":
        cu = np.concatenate([[0], np.cumsum(_lengths(case, seqs))])
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device=DEV)
        shape = (int(cu[-1]),)
    else:
        shape = (seqs, case["cols"])
        s["mask"] = _padded_mask(seqs, case["cols"], gen)
    # log probabilities of sampled tokens: mostly near 0, some unlikely; the model that drew the
    # tokens and the reference are near the one that is trained
    lp = -(randn(*shape).square() * 0.7 + 0.01)
    near = 0.15 if case["op"] == "policy" else 0.05
    old = lp + near * randn(*shape)
    ref = lp + near * randn(*shape)
    if case["op"] == "policy":
        ref -= 0.05     # a trained model gives its own samples more than the reference does
    if s["mask"] is not None:
        # what padding holds is arbitrary, and padded log probs are often -inf or NaN
        lp.masked_fill_(~s["mask"], float("-inf"))
        old.masked_fill_(~s["mask"], float("nan"))
    s["lp"], s["old"], s["ref"] = lp.to(dt), old.to(dt), ref.to(dt)
    if case["op"] == "policy":
        s["adv"] = 1 + randn(*(shape if case["adv"] == "token" else (seqs,)))
    return s


def _prepare_adamw(case, seed, randn, gen):
    sizes = _sizes(case)
    # every tensor starts on a block boundary of one flat buffer, as in a bucketed trainer
    starts = np.concatenate([[0], np.cumsum([-(-n // BLOCK) * BLOCK for n in sizes])])
    total = int(starts[-1])
    s = {"case": case, "step": 100, "seed": int(seed) & 0xFFFF, "sizes": sizes, "starts": starts}
    s["master"] = randn(total).mul_(0.02) if case["master"] else None
    p = s["master"] if case["master"] else randn(total).mul_(0.02)
    s["p"] = p.to(DT[case["dtype"]], copy=True)
    del p
    s["g"] = randn(total).mul_(5e-4).to(DT[case["grad"]])
    s["gscale"] = torch.full((1,), 0.75, device=DEV)
    if case["bits"] == 8:
        nb = total // BLOCK
        s["m"] = randn(total).mul_(80).clamp_(-448, 448).to(torch.float8_e4m3fn)
        s["v"] = randn(total).mul_(60).abs_().add_(90).clamp_(0, 448).to(torch.float8_e4m3fn)
        s["ms"] = 1e-6 * torch.exp(0.3 * randn(nb))
        s["vs"] = 3e-6 * torch.exp(0.3 * randn(nb))
    else:
        s["m"] = randn(total).mul_(1e-4)
        s["v"] = (randn(total).mul_(1.5e-4).abs_().add_(2e-4)).square_()
    flat = [k for k in ("master", "p", "g", "m", "v") if s[k] is not None]
    for n, a, b in zip(sizes, starts, starts[1:]):
        for k in flat:
            if a + n < b:
                (s[k].view(torch.uint8) if s[k].element_size() == 1 else s[k])[a + n:b] = 0
    if own:
        from linear_cross_entropy_tiled_gb300 import adamw_plan

        def views(k, scale=False):
            if s.get(k) is None:
                return None
            if scale:
                return [s[k][a // BLOCK:b // BLOCK] for a, b in zip(starts, starts[1:])]
            v = [s[k][a:a + n] for n, a in zip(sizes, starts)]
            v[0] = v[0].view(case["vocab"], case["hidden"])
            return v
        s["grads"] = views("g")
        s["plan"] = adamw_plan(views("p"), views("m"), views("v"), exp_avg_scales=views("ms", True),
                               exp_avg_sq_scales=views("vs", True), master_params=views("master"))
    return s


# -------------------------------------------------------------- the passes
def run(s):
    op = s["case"]["op"]
    if op == "policy":
        return _own_policy(s) if own else _plain_policy(s)
    if op == "preference":
        return _own_preference(s) if own else _plain_preference(s)
    s["step"] += 1
    return _own_adamw(s) if own else _plain_adamw(s)


def _own_policy(s):
    from linear_cross_entropy_tiled_gb300 import policy_loss_and_grad
    c = s["case"]
    loss, grad, metrics = policy_loss_and_grad(
        s["lp"], s["old"], s["adv"], ref_log_probs=s["ref"] if c["kl"] else None, mask=s["mask"],
        cu_seqlens=s["cu"], clip_low=CLIP_LOW, clip_high=CLIP_HIGH, dual_clip=c["dual"] or None,
        kl_coef=c["kl"], kl_estimator=c["kl_estimator"], reduction=c["reduction"],
        return_metrics=True)
    return {"loss": loss, "grad": grad, "num_tokens": metrics["num_tokens"],
            "num_clipped": metrics["num_clipped"], "kl_sum": metrics["kl_sum"]}


def _rows(s, shape):
    """Row of every token, its number of tokens per row, and the number of rows."""
    if s["cu"] is None:
        return None, None, shape[0]
    n = (s["cu"][1:] - s["cu"][:-1]).long()
    return torch.repeat_interleave(torch.arange(n.numel(), device=DEV), n, output_size=shape[0]), n, n.numel()


def _plain_policy(s):
    c = s["case"]
    lp, old, ref = s["lp"].float(), s["old"].float(), s["ref"].float()
    row, n, seqs = _rows(s, lp.shape)
    adv = s["adv"].float()
    if c["adv"] == "sequence":
        adv = adv[row] if row is not None else adv[:, None]
    valid = s["mask"] if s["mask"] is not None else torch.ones_like(lp, dtype=torch.bool)
    lo, hi = math.log(1 - CLIP_LOW), math.log(1 + CLIP_HIGH)
    d = torch.where(valid, lp - old, 0)
    ratio = torch.exp(d)
    clipped = torch.exp(d.clamp(lo, hi))
    tok = torch.maximum(-adv * ratio, -adv * clipped)
    active = ((adv > 0) & (d <= hi)) | ((adv < 0) & (d >= lo))
    if c["dual"]:
        over = (adv < 0) & (d > math.log(c["dual"]))
        tok = torch.where(over, -c["dual"] * adv, tok)
        active = active & ~over
    g = torch.where(active, -adv * ratio, 0)
    kl = torch.zeros_like(lp)
    if c["kl"]:
        e = torch.where(valid, lp - ref, 0)
        if c["kl_estimator"] == "k1":
            kl, dkl = e, torch.ones_like(e)
        elif c["kl_estimator"] == "k2":
            kl, dkl = 0.5 * e * e, e
        else:
            kl, dkl = torch.expm1(-e) + e, -torch.expm1(-e)
        tok = tok + c["kl"] * kl
        g = g + c["kl"] * dkl
    if c["reduction"] == "sum":
        w = 1.0
    elif c["reduction"] == "mean":
        w = 1.0 / valid.sum().float()
    elif row is None:
        w = 1.0 / (seqs * valid.sum(1, keepdim=True).clamp(min=1).float())
    else:
        w = (1.0 / (seqs * n.clamp(min=1).float()))[row]
    loss = torch.where(valid, tok * w, 0).sum()
    grad = torch.where(valid, g * w, 0)
    out_of_clip = valid & ~active & (adv != 0)
    return {"loss": loss, "grad": grad, "num_tokens": valid.sum(),
            "num_clipped": out_of_clip.sum(), "kl_sum": torch.where(valid, kl, 0).sum()}


def _own_preference(s):
    from linear_cross_entropy_tiled_gb300 import preference_loss_and_grad
    c = s["case"]
    loss, grad, chosen, rejected = preference_loss_and_grad(
        s["lp"], s["ref"] if c["ref"] else None, mask=s["mask"], cu_seqlens=s["cu"], beta=BETA,
        loss_type=c["loss"], label_smoothing=c["smoothing"], margin=MARGIN, average=c["average"])
    return {"loss": loss, "grad": grad, "chosen_rewards": chosen, "rejected_rewards": rejected}


def _plain_preference(s):
    c = s["case"]
    lp = s["lp"].float()
    e = lp - s["ref"].float() if c["ref"] else lp
    row, n, seqs = _rows(s, lp.shape)
    pairs = seqs // 2
    if row is None:
        valid = s["mask"]
        n = valid.sum(1)
        e = torch.where(valid, e, 0).sum(1)
    else:
        at = s["cu"][:-1, None].long() + torch.arange(c["cols"], device=DEV)
        inside = torch.arange(c["cols"], device=DEV) < n[:, None]
        e = torch.where(inside, e[at.clamp(max=lp.numel() - 1)], 0).sum(1)
    inv = 1.0 / n.clamp(min=1).float() if c["average"] else torch.ones(seqs, device=DEV)
    r = e * inv
    z = BETA * (r[:pairs] - r[pairs:]) - MARGIN
    if c["loss"] == "sigmoid":
        soft = torch.log1p(torch.exp(-z.abs()))
        eps = c["smoothing"]
        loss = (1 - eps) * (soft + (-z).clamp(min=0)) + eps * (soft + z.clamp(min=0))
        dz = eps - 1.0 / (1.0 + torch.exp(z))
    elif c["loss"] == "hinge":
        loss, dz = (1 - z).clamp(min=0), torch.where(z < 1, -1.0, 0.0)
    else:
        loss, dz = (z / BETA - 0.5 / BETA).square(), 2 * (z / BETA - 0.5 / BETA) / BETA
    dh = BETA * dz / pairs
    w = torch.cat([dh, -dh]) * inv
    if row is None:
        grad = torch.where(valid, w[:, None], 0)
    else:
        grad = w[row]
    # gradients are fp32 whatever the log probs are: 1 / tokens is below the range of 16 bits
    return {"loss": loss.mean(), "grad": grad, "chosen_rewards": BETA * r[:pairs],
            "rejected_rewards": BETA * r[pairs:]}


LR, B1, B2, EPS, DECAY = 3e-4, 0.9, 0.999, 1e-8, 0.1


def _own_adamw(s):
    s["plan"].step(s["grads"], step=s["step"], lr=LR, betas=(B1, B2), eps=EPS, weight_decay=DECAY,
                   grad_scale=s["gscale"], seed=s["seed"])
    return _adamw_out(s)


def _adamw_out(s):
    # an 8-bit state is its e4m3 values and the scale of each block of 256
    return {k: s[k] for k in ("p", "master", "m", "v", "ms", "vs") if s.get(k) is not None}


def _random16(total, seed, step):
    """16 random bits for each element: half of a hash of its pair's index, the seed and the step."""
    key = (seed * C1 + step * C2) & M32
    key ^= key >> 16
    key = (key * C1) & M32
    x = (torch.arange(total // 2, device=DEV) ^ key) & M32
    x = (x * C1) & M32
    x = x ^ (x >> 15)
    x = (x * C2) & M32
    x = x ^ (x >> 13)
    x = (x * C1) & M32
    x = x ^ (x >> 16)
    return torch.stack([x & 0xFFFF, x >> 16], 1).reshape(-1).int()


def _plain_adamw(s):
    c, t = s["case"], s["step"]
    p = s["master"] if c["master"] else s["p"].float()
    g = s["g"].float() * s["gscale"]
    if c["bits"] == 8:
        m = (s["m"].float().view(-1, BLOCK) * s["ms"][:, None]).view(-1)
        r = (s["v"].float().view(-1, BLOCK) * s["vs"][:, None]).view(-1)
        v = r * r
    else:
        m, v = s["m"], s["v"]
    m = B1 * m + (1 - B1) * g
    v = B2 * v + (1 - B2) * (g * g)
    r = v.sqrt()
    p = p * (1 - LR * DECAY) - (LR / (1 - B1 ** t)) * m / (r / math.sqrt(1 - B2 ** t) + EPS)
    if c["bits"] == 8:
        def scaled(x):
            x = x.view(-1, BLOCK)
            top = x.abs().amax(1)
            inv = torch.where(top >= 2.0 ** -100, 448.0 / top, 0)
            return (x * inv[:, None]).view(-1), torch.where(top >= 2.0 ** -100, top / 448.0, 0)
        x, ms = scaled(m)
        s["m"].copy_(x.to(torch.float8_e4m3fn))
        s["ms"].copy_(ms)
        x, vs = scaled(r)
        # e4m3 has 3 mantissa bits and bias 7: as the bits of x 2^-120 in fp32 without their last 20
        bits = (x * 2.0 ** -120).view(torch.int32)
        code = (bits + (_random16(x.numel(), s["seed"], t) * 16 + 8)) >> 20
        code = torch.where(x > 0, code.clamp(1, 0x7E), 0)
        s["v"].view(torch.uint8).copy_(code)
        s["vs"].copy_(vs)
    else:
        s["m"].copy_(m)
        s["v"].copy_(v)
    if c["master"]:
        s["master"].copy_(p)
    s["p"].copy_(p)
    return _adamw_out(s)


# ------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    """From the formulas, sequence by sequence (numpy) or block range by block range (AdamW)."""
    s = prepare(case, seed)
    if case["op"] == "adamw":
        return _exact_adamw(s)
    lp, old, ref = (s[k].double().cpu().numpy() for k in ("lp", "old", "ref"))
    if s["cu"] is not None:
        cu = s["cu"].cpu().numpy()
        cut = [np.arange(a, b) for a, b in zip(cu, cu[1:])]
    else:
        mask, cols = s["mask"].cpu().numpy(), case["cols"]
        cut = [i * cols + np.flatnonzero(mask[i]) for i in range(mask.shape[0])]
    shape = lp.shape
    lp, old, ref = lp.reshape(-1), old.reshape(-1), ref.reshape(-1)
    grad = np.zeros(lp.size)
    if case["op"] == "policy":
        return _exact_policy(case, cut, lp, old, ref, s["adv"].double().cpu().numpy(), grad, shape)
    pairs = len(cut) // 2
    logit = np.zeros(2 * pairs)
    for i, at in enumerate(cut):
        v = lp[at] - ref[at] if case["ref"] else lp[at]
        logit[i] = math.fsum(v) / (max(1, at.size) if case["average"] else 1)
    losses = []
    for i in range(pairs):
        z = BETA * (logit[i] - logit[pairs + i]) - MARGIN
        if case["loss"] == "sigmoid":
            eps = case["smoothing"]
            losses.append((1 - eps) * np.logaddexp(0, -z) + eps * np.logaddexp(0, z))
            slope = (eps - 1) * math.exp(-np.logaddexp(0, z)) + eps * math.exp(-np.logaddexp(0, -z))
        elif case["loss"] == "hinge":
            losses.append(max(0.0, 1 - z))
            slope = -1.0 if z < 1 else 0.0
        else:
            u = (z - 0.5) / BETA
            losses.append(u * u)
            slope = 2 * u / BETA
        for j, sign in ((i, 1.0), (pairs + i, -1.0)):
            n = max(1, cut[j].size) if case["average"] else 1
            grad[cut[j]] = sign * BETA * slope / (pairs * n)
    return {"loss": float(np.mean(losses)), "grad": grad.reshape(shape),
            "chosen_rewards": BETA * logit[:pairs], "rejected_rewards": BETA * logit[pairs:]}


def _exact_policy(case, cut, lp, old, ref, adv, grad, shape):
    tokens = sum(at.size for at in cut)
    adv = adv.reshape(-1)
    total, kl_sum, clipped = [], [], 0
    for i, at in enumerate(cut):
        if at.size == 0:
            continue
        w = {"sum": 1.0, "mean": 1.0 / tokens, "sequence_mean": 1.0 / (len(cut) * at.size)}[case["reduction"]]
        a = adv[at] if case["adv"] == "token" else np.full(at.size, adv[i])
        r = np.exp(lp[at] - old[at])
        surrogate = np.minimum(a * r, a * np.clip(r, 1 - CLIP_LOW, 1 + CLIP_HIGH))
        cut_off = np.where(a > 0, r > 1 + CLIP_HIGH, (a < 0) & (r < 1 - CLIP_LOW))
        if case["dual"]:
            worse = (a < 0) & (r > case["dual"])
            surrogate = np.where(worse, case["dual"] * a, surrogate)
            cut_off = cut_off | worse
        tok, g = -surrogate, np.where(cut_off, 0.0, -a * r)
        if case["kl"]:
            x = ref[at] - lp[at]
            kl, slope = {"k1": lambda: (-x, np.ones_like(x)), "k2": lambda: (x * x / 2, -x),
                         "k3": lambda: (np.exp(x) - x - 1, 1 - np.exp(x))}[case["kl_estimator"]]()
            tok, g = tok + case["kl"] * kl, g + case["kl"] * slope
            kl_sum.append(float(np.sum(kl)))
        total.append(w * float(np.sum(tok)))
        grad[at] = w * g
        clipped += int(cut_off.sum())
    return {"loss": math.fsum(total), "grad": grad.reshape(shape), "num_tokens": tokens,
            "num_clipped": clipped, "kl_sum": math.fsum(kl_sum)}


def _exact_adamw(s):
    """The rounding of the states to 8 bits is not applied: like that of p, it counts as error."""
    c, t = s["case"], s["step"] + 1
    names = [k for k in ("p", "master", "m", "v", "ms", "vs") if s.get(k) is not None]
    out = {k: torch.empty(s[k].shape, dtype=torch.float64, device=DEV) for k in names}
    total, piece = s["g"].numel(), 1 << 26
    for a in range(0, total, piece):
        at, blk = slice(a, min(total, a + piece)), slice(a // BLOCK, min(total, a + piece) // BLOCK)
        w = (s["master"] if c["master"] else s["p"])[at].double()
        g = s["g"][at].double() * s["gscale"].double()
        m, v = s["m"][at].double(), s["v"][at].double()
        if c["bits"] == 8:
            m = (m.view(-1, BLOCK) * s["ms"][blk, None].double()).view(-1)
            v = (v.view(-1, BLOCK) * s["vs"][blk, None].double()).view(-1).square()
        m = m + (1 - B1) * (g - m)
        v = v + (1 - B2) * (g.square() - v)
        w = w - LR * DECAY * w - LR * (m / (1 - B1 ** t)) / ((v / (1 - B2 ** t)).sqrt() + EPS)
        for k in ("p", "master"):
            if k in out:
                out[k][at] = w
        if c["bits"] == 8:
            for k, x in (("m", m), ("v", v.sqrt())):
                x = x.view(-1, BLOCK)
                top = x.abs().amax(1) / 448
                out[k + "s"][blk] = top
                out[k][at] = (x / top.clamp(min=1e-300)[:, None]).view(-1)
        else:
            out["m"][at], out["v"][at] = m, v
    return out
