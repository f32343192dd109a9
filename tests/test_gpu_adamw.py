"""AdamW over many tensors against the fp64 oracle.

Tolerances, before any run. Each new moment is three fp32 operations on the
same inputs: 4 x 2^-24 of the magnitudes it is summed from, so 5e-7. The
update adds a root, a quotient and three products: 16 x 2^-24 = 1e-6 of its
size (with the magnitudes behind m, which may cancel), and the parameter
itself one rounding of 2^-24 twice, plus half a unit of its own type. An 8-bit
m lies within half an e4m3 step of its value, an 8-bit root within one step,
on the side that the given random bits pick: other codes come only where the
value's fp32 rounding crosses a threshold, at most a few in 10^4.
"""
import numpy as np
import pytest
import torch

import oracle.post_training_oracle as ref_ops
from linear_cross_entropy_tiled_gb300 import AdamW, _lib, adamw_plan

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
ROUND = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}   # unit roundoff of 24, 8, 11 bits
HYPER = dict(lr=3e-3, betas=(0.9, 0.995), eps=1e-8, weight_decay=0.1)
SIZES = [1, 255, 256, 257, 8, 0, 1000, 4096, 33333, 7]


class Tensors:
    def __init__(self, sizes, dtype, grad, bits, master, seed=0, offset=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.sizes, self.dtype, self.bits, self.offset = sizes, dtype, bits, offset

        def make(f, dt):
            out = []
            for n in sizes:
                x = f(torch.randn(n, device="cuda", generator=g)).to(dt)
                if offset:                      # off the 16-byte alignment
                    y = torch.empty(n + offset, dtype=dt, device="cuda")[offset:]
                    (y.view(torch.uint8) if dt == torch.float8_e4m3fn else y).copy_(
                        x.view(torch.uint8) if dt == torch.float8_e4m3fn else x)
                    x = y
                out.append(x)
            return out
        self.master = make(lambda x: 0.02 * x, torch.float32) if master else None
        self.p = [m.to(DT[dtype]) for m in self.master] if master and not offset else \
            make(lambda x: 0.02 * x, DT[dtype])
        self.g = make(lambda x: 5e-4 * x, DT[grad])
        if bits == 8:
            blocks = [-(-n // 256) for n in sizes]
            self.m = make(lambda x: (90 * x).clamp(-448, 448), torch.float8_e4m3fn)
            self.v = make(lambda x: (90 + 60 * x.abs()).clamp(max=448), torch.float8_e4m3fn)
            self.ms = [1e-6 * torch.rand(n, device="cuda", generator=g) for n in blocks]
            self.vs = [3e-6 * (0.5 + torch.rand(n, device="cuda", generator=g)) for n in blocks]
        else:
            self.m = make(lambda x: 1e-4 * x, torch.float32)
            self.v = make(lambda x: (2e-4 * x) ** 2, torch.float32)
            self.ms = self.vs = None

    def plan(self):
        return adamw_plan(self.p, self.m, self.v, exp_avg_scales=self.ms, exp_avg_sq_scales=self.vs,
                          master_params=self.master)

    def host(self):
        def f(ts):
            return None if ts is None else [t.double().cpu().numpy() for t in ts]
        h = dict(p=f(self.master or self.p), g=f(self.g), m=f(self.m), v=f(self.v))
        if self.bits == 8:
            for k, s in (("m", self.ms), ("v", self.vs)):
                h[k] = [x * np.repeat(t.double().cpu().numpy(), 256)[:x.size]
                        for x, t in zip(h[k], s)]
            h["v"] = [x * x for x in h["v"]]
        return h


def codes(t):
    return t.reshape(-1).view(torch.uint8).cpu().numpy().astype(np.int64)


def check_step(x, before, step, grad_scale=1.0, seed=0):
    first_block, differ, total = 0, 0, 0
    for i, n in enumerate(x.sizes):
        b1, b2 = HYPER["betas"]
        p, m, v, size, behind = ref_ops.adamw(
            before["p"][i], before["g"][i], before["m"][i], before["v"][i], step=step, lr=HYPER["lr"],
            beta1=b1, beta2=b2, eps=HYPER["eps"], weight_decay=HYPER["weight_decay"],
            grad_scale=grad_scale)
        tol = 2 * 2.0 ** -24 * np.abs(p) + 1e-6 * size + 1e-30
        if x.master:
            assert (np.abs(x.master[i].double().cpu().numpy() - p) <= tol).all()
            assert torch.equal(x.p[i], x.master[i].to(DT[x.dtype]))
        else:
            got = x.p[i].double().cpu().numpy()
            assert (np.abs(got - p) <= tol + 1.01 * ROUND[x.dtype] * np.abs(p) + 2.0 ** -25).all()
        if x.bits == 32:
            assert (np.abs(x.m[i].double().cpu().numpy() - m) <= 5e-7 * behind).all()
            assert (np.abs(x.v[i].double().cpu().numpy() - v) <= 5e-7 * v + 1e-38).all()
            continue
        values = ref_ops.e4m3_values()
        for name, want, got, scale in (("m", m, x.m[i], x.ms[i]), ("v", np.sqrt(v), x.v[i], x.vs[i])):
            s, z = ref_ops.block_scale(want)
            c = codes(got)
            np.testing.assert_allclose(scale.double().cpu().numpy(), s, rtol=1e-6, atol=1e-36)
            y = values[c & 0x7F] * np.where(c & 0x80, -1, 1)
            spacing = 2.0 ** np.maximum(np.floor(np.log2(np.maximum(np.abs(z), 2.0 ** -6))), -6) / 8
            slack = 1e-6 * (behind / np.maximum(np.repeat(s, 256)[:n], 1e-36) if name == "m" else z)
            assert (np.abs(y - z) <= (0.5 if name == "m" else 1.0) * spacing * 1.0001 + slack).all()
            if name == "v":
                assert ((c > 0) | (z == 0)).all()
                want_c = ref_ops.stochastic_code(z, ref_ops.pair_bits(n, first_block, seed, step))
                differ += int((want_c != c).sum())
                total += n
        first_block += -(-n // 256)
    assert differ <= 5e-4 * total + 3, (differ, total)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dtype,grad,master", [("f32", "f32", False), ("bf16", "bf16", False),
                                               ("bf16", "f32", True), ("f16", "f16", True),
                                               ("f16", "f32", False)])
@pytest.mark.parametrize("offset", [0, 1])
def test_step(bits, dtype, grad, master, offset):
    x = Tensors(SIZES, dtype, grad, bits, master, seed=1, offset=offset)
    plan = x.plan()
    scale = torch.full((1,), 0.5, device="cuda")
    for step in (1, 2, 700):
        before = x.host()
        plan.step(x.g, step=step, grad_scale=scale, seed=9, **HYPER)
        check_step(x, before, step, 0.5, 9)


@pytest.mark.parametrize("bits", [32, 8])
def test_more_tensors_than_a_table(bits):
    """Several launches; the random bits go on counting through them."""
    r = np.random.default_rng(0)
    x = Tensors([int(n) for n in r.integers(1, 700, 1000)], "bf16", "bf16", bits,
                False, seed=2)
    before = x.host()
    n0 = _lib.launch_count()
    x.plan().step(x.g, step=3, **HYPER)
    assert _lib.launch_count() - n0 == 3           # tables of 448
    check_step(x, before, 3)


def test_canaries():
    """Nothing around any tensor changes, at sizes that end inside a block, off alignment."""
    for bits in (8, 32):
        for offset in (3, 64):
            n = 777
            x = Tensors([n], "bf16", "bf16", bits, True, seed=3)
            for name in ("p", "master", "m", "v", "ms", "vs"):
                ts = getattr(x, name)
                if ts is None:
                    continue
                t = ts[0]
                raw = torch.full((t.numel() * t.element_size() + 4096,), 0xA5, dtype=torch.uint8,
                                 device="cuda")
                o = 2048 + offset * t.element_size()
                y = raw[o:o + t.numel() * t.element_size()].view(t.dtype)
                y.view(torch.uint8).copy_(t.view(torch.uint8))
                ts[0] = y
                x.__dict__.setdefault("raws", []).append((raw, o, y))
            x.plan().step(x.g, step=1, **HYPER)
            for raw, o, y in x.raws:
                end = o + y.numel() * y.element_size()
                assert (raw[:o] == 0xA5).all() and (raw[end:] == 0xA5).all()


def test_nonfinite_gradients():
    """32-bit states: the element's own. 8-bit: its block of 256, and no other."""
    for bad in (float("nan"), float("inf")):
        for bits in (32, 8):
            x = Tensors([1000], "f32", "f32", bits, False, seed=4)
            x.g[0][300] = bad
            x.plan().step(x.g, step=1, **HYPER)
            assert x.p[0].isfinite().sum() == 999
            if bits == 8:
                m = x.m[0].float() * x.ms[0].repeat_interleave(256)[:1000]
                v = x.v[0].float() * x.vs[0].repeat_interleave(256)[:1000]
                for t in (m, v):
                    assert t[:256].isfinite().all() and t[512:].isfinite().all()
                    assert not t[300].isfinite()


def test_zero_blocks_and_tiny_values():
    """Blocks of zeros stay zeros; magnitudes below 2^-100 are held as zeros; a tiny root keeps a code."""
    x = Tensors([768], "f32", "f32", 8, False, seed=5)
    for t in (x.m[0], x.v[0]):
        t.view(torch.uint8).zero_()
    x.g[0].zero_()
    x.g[0][256] = 1e-37          # alone in its block: m = 1e-38 < 2^-100
    x.g[0][512] = 1.0
    x.g[0][513] = 1e-9           # its root is far below the block's smallest code
    x.plan().step(x.g, step=1, **HYPER)
    assert (codes(x.m[0])[:512] == 0).all() and (x.ms[0][:2] == 0).all() and (x.vs[0][:2] == 0).all()
    assert codes(x.v[0])[513] == 1 and codes(x.m[0])[513] == 0 and x.p[0].isfinite().all()


def test_stochastic_rounding_is_unbiased():
    """Constant second moment: its stored root averages to the true one over seeds."""
    n, seeds = 4096, 200
    total = torch.zeros(n, dtype=torch.float64, device="cuda")
    for seed in range(seeds):
        x = Tensors([n], "f32", "f32", 8, False, seed=6)
        x.plan().step(x.g, step=5, seed=seed, **HYPER)
        total += x.v[0].double() * x.vs[0].double().repeat_interleave(256)
    x = Tensors([n], "f32", "f32", 8, False, seed=6)
    h = x.host()
    _, _, v, _, _ = ref_ops.adamw(h["p"][0], h["g"][0], h["m"][0], h["v"][0], step=5, lr=0, beta1=0.9,
                                  beta2=HYPER["betas"][1], eps=1e-8, weight_decay=0)
    rel = total.cpu().numpy() / seeds / np.sqrt(v) - 1
    # one rounding is off by at most 1/8 of the value, 1/16 in the root mean square at most; the
    # mean over n x seeds draws by 1/16 / sqrt(819200) = 7e-5 (5 sigma: 3.5e-4), and one element's
    # mean by 1/16 / sqrt(200) = 4.4e-3 (6 sigma: 2.7e-2)
    assert abs(rel.mean()) < 3.5e-4 and np.abs(rel).max() < 2.7e-2


def test_a_decaying_second_moment_decays():
    """With gradients gone, v falls by beta2 a step although each step is below one code."""
    n = 4096
    x = Tensors([n], "f32", "f32", 8, False, seed=7)
    x.g[0].zero_()
    x.g[0][::256] = 1e-3                      # keeps every block's scale up
    r0 = (x.v[0].double() * x.vs[0].double().repeat_interleave(256)).cpu().numpy()
    plan = x.plan()
    for step in range(1, 201):
        plan.step(x.g, step=step, seed=1, **HYPER)
    r = (x.v[0].double() * x.vs[0].double().repeat_interleave(256)).cpu().numpy()
    rest = np.arange(n) % 256 != 0
    want = HYPER["betas"][1] ** 100           # of the root after 200 steps
    assert r[rest].sum() / r0[rest].sum() == pytest.approx(want, rel=0.05)


def test_layouts_of_dimensions():
    """A transposed parameter is stepped in its own order; a gradient in another order is copied."""
    p = torch.randn(40, 30, device="cuda").t()
    g = torch.randn(30, 40, device="cuda")
    m, v = torch.zeros_like(p), torch.zeros_like(p)
    assert m.stride() == p.stride()
    q = p.clone(memory_format=torch.contiguous_format)
    mq, vq = torch.zeros_like(q), torch.zeros_like(q)
    adamw_plan([p], [m], [v]).step([g], step=1, **HYPER)
    adamw_plan([q], [mq], [vq]).step([g], step=1, **HYPER)
    assert torch.equal(p, q) and torch.equal(m, mq) and torch.equal(v, vq)


@pytest.mark.parametrize("bits,master", [(32, False), (32, True), (8, True), (8, False)])
def test_optimizer(bits, master):
    """Groups, parameters without gradients, a saved and restored state: the same bits as one run."""
    def model():
        g = torch.Generator(device="cuda").manual_seed(3)
        ps = [torch.nn.Parameter(torch.randn(s, device="cuda", generator=g).to(dt))
              for s, dt in (((64, 33), torch.bfloat16), ((129,), torch.bfloat16),
                            ((5,), torch.float32), ((7,), torch.bfloat16))]
        opt = AdamW([{"params": ps[:2]}, {"params": ps[2:], "weight_decay": 0.0, "lr": 1e-2}],
                    lr=1e-3, state_bits=bits, master_weights=master, seed=4)
        return ps, opt

    def grads(ps, t):
        g = torch.Generator(device="cuda").manual_seed(100 + t)
        for i, p in enumerate(ps):
            p.grad = None if i == 3 and t < 3 else torch.randn(p.shape, device="cuda",
                                                               generator=g).to(p.dtype)
    a, opt_a = model()
    for t in range(6):
        grads(a, t)
        opt_a.step(grad_scale=torch.full((1,), 0.5, device="cuda"))
    b, opt_b = model()
    for t in range(3):
        grads(b, t)
        opt_b.step(grad_scale=torch.full((1,), 0.5, device="cuda"))
    assert 3 not in [i for i, p in enumerate(b) if p in opt_b.state and i == 3]
    c, opt_c = model()
    for x, y in zip(c, b):
        x.data.copy_(y.data)
    opt_c.load_state_dict(opt_b.state_dict())
    for t in range(3, 6):
        grads(c, t)
        opt_c.step(grad_scale=torch.full((1,), 0.5, device="cuda"))
    for x, y in zip(a, c):
        assert torch.equal(x, y)
        for k, v in opt_a.state[x].items():
            w = opt_c.state[y][k]
            if isinstance(v, torch.Tensor):
                assert v.dtype == w.dtype and torch.equal(v.view(torch.uint8), w.view(torch.uint8))
            else:
                assert v == w
    s = opt_a.state[a[0]]
    assert s["exp_avg"].dtype == (torch.float8_e4m3fn if bits == 8 else torch.float32)
    assert ("master" in s) == master and "master" not in opt_a.state[a[2]]


def test_optimizer_follows_reassigned_storage():
    p = torch.nn.Parameter(torch.ones(300, device="cuda"))
    opt = AdamW([p], lr=0.1, weight_decay=0.0)
    p.grad = torch.ones_like(p)
    opt.step()
    old = p.data
    p.data = p.data.clone()
    opt.step()
    assert (p < old).all() and (old - 0.9).abs().max() < 1e-5


def test_optimizer_trains_alike_with_8_and_32_bits():
    """A least-squares fit: 300 steps of 8-bit states end within a tenth of the loss drop of 32-bit ones."""
    end = {}
    for bits in (8, 32):
        g = torch.Generator(device="cuda").manual_seed(8)
        x = torch.randn(512, 64, device="cuda", generator=g)
        y = x @ torch.randn(64, 16, device="cuda", generator=g)
        w = torch.nn.Parameter(torch.zeros(64, 16, device="cuda"))
        opt = AdamW([w], lr=2e-2, weight_decay=0.0, state_bits=bits, betas=(0.9, 0.999))
        for _ in range(300):
            opt.zero_grad()
            loss = (x @ w - y).square().mean()
            loss.backward()
            opt.step()
        end[bits] = loss.item()
    assert end[8] < 6.4 and abs(end[8] - end[32]) < 6.4      # from about 64
