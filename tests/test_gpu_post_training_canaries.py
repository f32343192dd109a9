"""Post-training losses: no byte outside the outputs and the stated workspace changes, kernels per call, CUDA
graphs, and the small suites again under the build that checks every store."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from linear_cross_entropy_tiled_gb300 import (_lib, adamw_plan, policy_loss_and_grad,
                                              preference_loss_and_grad)

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
GUARD = 4096


class Guarded:
    def __init__(self, nbytes, offset=0):
        self.raw = torch.full((nbytes + 2 * GUARD,), 0xA5, dtype=torch.uint8, device="cuda")
        self.lo, self.hi = GUARD + offset, GUARD + offset + nbytes

    @property
    def ptr(self):
        return self.raw.data_ptr() + self.lo

    def check(self):
        assert (self.raw[:self.lo] == 0xA5).all() and (self.raw[self.hi:] == 0xA5).all()


@pytest.mark.parametrize("op", ["policy", "preference"])
@pytest.mark.parametrize("S,T,ld,offset", [(4, 33, 33, 0), (4, 33, 40, 4), (6, 7001, 7001, 0), (6, 7001, 7008, 0),
                                           (6, 7001, 7001, 12), (2, 90001, 90001, 0)])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("reduction", [1, 3])
def test_nothing_outside_changes(op, S, T, ld, offset, packed, reduction):
    if packed and ld != T:
        pytest.skip("packed tokens have no row stride")
    g = np.random.default_rng(0)
    lp = -torch.rand(S * ld + 8, device="cuda")
    mask = (torch.rand(S * T, device="cuda") < 0.6).to(torch.uint8)
    adv = torch.randn(S, device="cuda")
    cu = torch.tensor(np.concatenate([[0], np.sort(g.integers(0, S * T, S - 1)), [S * T]]), dtype=torch.int32,
                      device="cuda")
    grad = Guarded(((S - 1) * ld + T) * 4, offset)
    scalars = [Guarded(8) for _ in range(4)]
    rewards = [Guarded(S // 2 * 4) for _ in range(2)]
    a = _lib.FlcePolicyArgs() if op == "policy" else _lib.FlcePreferenceArgs()
    t = a.tokens
    t.sequences, t.mask, t.ld_mask, t.mask_kind = S, mask.data_ptr(), T, _lib.FLCE_MASK_BYTES
    if packed:
        t.packed, t.tokens, t.cu_seqlens = 1, S * T, cu.data_ptr()
    else:
        t.cols = T
    a.log_probs, a.ref_log_probs, a.ld_log_probs, a.ld_ref = lp.data_ptr(), lp.data_ptr() + 32, ld, ld
    a.grad, a.ld_grad, a.loss = grad.ptr, ld, scalars[0].ptr
    if op == "policy":
        a.advantages, a.num_tokens, a.num_clipped, a.kl_sum = (adv.data_ptr(), *(s.ptr for s in scalars[1:]))
        a.clip_low, a.clip_high, a.kl_coef, a.reduction = 0.2, 0.2, 0.1, reduction
        need, run = _lib.policy_workspace_bytes(a), _lib.policy_loss_raw
    else:
        a.chosen_rewards, a.rejected_rewards, a.beta = rewards[0].ptr, rewards[1].ptr, 0.1
        need, run = _lib.preference_workspace_bytes(a), _lib.preference_loss_raw
    ws = Guarded(need)
    a.workspace, a.ws_bytes = ws.ptr, need
    _lib.check(run(a, torch.cuda.current_stream().cuda_stream), op)
    torch.cuda.synchronize()
    for x in (grad, ws, *scalars, *rewards):
        x.check()
    # between the rows of a strided gradient nothing is written either
    if not packed and ld > T:
        rows = grad.raw[grad.lo:grad.lo + (S - 1) * ld * 4].view(S - 1, ld * 4)
        assert (rows[:, T * 4:] == 0xA5).all()


def test_kernels_per_call():
    def count(f):
        torch.cuda.synchronize()
        n = _lib.launch_count()
        f()
        return _lib.launch_count() - n
    small, large = -torch.rand(8, 100, device="cuda"), -torch.rand(64, 4001, device="cuda")
    adv = torch.ones(64, device="cuda")
    mask = torch.ones(64, 4001, dtype=torch.bool, device="cuda")
    assert count(lambda: policy_loss_and_grad(small, small, adv[:8], mask=mask[:8, :100])) == 1
    assert count(lambda: policy_loss_and_grad(large, large, adv)) == 1                # nothing to count
    assert count(lambda: policy_loss_and_grad(large, large, adv, mask=mask, reduction="sum")) == 1
    for red in ("mean", "sequence_mean"):
        assert count(lambda: policy_loss_and_grad(large, large, adv, mask=mask, reduction=red)) == 2
    assert count(lambda: preference_loss_and_grad(small, small)) == 1
    assert count(lambda: preference_loss_and_grad(large, large, mask=mask)) == 1


def test_cuda_graph():
    """The calls capture, and a replay computes with what its inputs then hold."""
    lp = -torch.rand(40, 3000, device="cuda")
    adv = torch.randn(40, device="cuda")
    mask = torch.rand(40, 3000, device="cuda") < 0.5
    p = [torch.randn(5000, device="cuda")]
    m, v = [torch.zeros_like(p[0])], [torch.zeros_like(p[0])]
    plan = adamw_plan(p, m, v)

    def step():
        a = policy_loss_and_grad(lp, lp + 0.1, adv, mask=mask)
        b = preference_loss_and_grad(lp, mask=mask)
        plan.step([a[1].view(-1)[:5000]], step=1, lr=0.1)
        return (*a, *b)
    step()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        out = step()
    lp.copy_(-torch.rand(40, 3000, device="cuda"))
    mask.logical_not_()
    for t in (p[0], m[0], v[0]):
        t.fill_(0.5)
    graph.replay()
    got, state = [t.clone() for t in out], [t.clone() for t in (p[0], m[0], v[0])]
    for t in (p[0], m[0], v[0]):
        t.fill_(0.5)
    want = step()
    for x, y in zip(got, want):
        assert torch.equal(x, y)
    for x, y in zip(state, (p[0], m[0], v[0])):
        assert torch.equal(x, y)


def test_small_suites_pass_with_every_store_checked():
    out = subprocess.run([sys.executable, "-m", "pytest", "-m", "gpu", "-q", "-x", "-p", "no:cacheprovider",
                          "--flce-debug-lib", "tests/test_gpu_post_training.py", "tests/test_gpu_adamw.py",
                          "tests/test_gpu_post_training_canaries.py", "-k",
                          "not every_store and not cuda_graph and not unbiased and not decaying and not trains"],
                         cwd=ROOT, capture_output=True, text=True, timeout=1200)
    assert out.returncode == 0, out.stdout[-3000:] + out.stderr[-2000:]
    assert " passed" in out.stdout and "failed" not in out.stdout
