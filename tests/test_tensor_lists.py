"""flce_tensors: what the AdamW step asks of lists of tensors, on CPU tensors."""
import os

import numpy as np
import pytest
import torch

from linear_cross_entropy_tiled_gb300 import _lib


@pytest.fixture(scope="module", autouse=True)
def built():
    if not os.path.exists(_lib.TENSORS_PATH):
        import __graft_entry__
        __graft_entry__.build()


def lists():
    params = [torch.ones(3, 4), torch.ones(5), torch.ones(0, 2), torch.ones(())]
    return params, [torch.ones_like(p) for p in params], np.full((4, 8), 7, dtype=np.uint64)


def test_addresses_go_into_the_table_and_nowhere_else():
    params, grads, table = lists()
    assert _lib.tensors().gradients(grads, params, table.ctypes.data)
    assert table[:, 1].tolist() == [g.data_ptr() for g in grads]
    assert (np.delete(table, 1, axis=1) == 7).all()
    assert _lib.tensors().gradients([], [], table.ctypes.data)


@pytest.mark.parametrize("at", [0, 1, 3])
@pytest.mark.parametrize("what", ["dtype", "shape", "device", "sparse", "order", "none", "missing"])
def test_gradients_that_do_not_agree(what, at):
    params, grads, table = lists()
    p = params[at]
    if what == "dtype":
        grads[at] = grads[at].half()
    elif what == "shape":
        grads[at] = grads[at].reshape(*p.shape, 1)
    elif what == "device":
        grads[at] = torch.ones_like(p, device="meta")
    elif what == "sparse":
        if p.dim() == 0:
            pytest.skip("a scalar has no sparse form here")
        grads[at] = grads[at].to_sparse()
    elif what == "order":
        if p.dim() < 2:
            pytest.skip("one order only")
        grads[at] = grads[at].t().contiguous().t()
    elif what == "none":
        grads[at] = None
    else:
        del grads[at]
    assert not _lib.tensors().gradients(grads, params, table.ctypes.data)


def test_alike():
    alike = _lib.tensors().alike
    a = torch.ones(4, 4)
    assert alike([a, a], [a.detach(), a.view(4, 4)])
    for b in (a.clone(), a.t(), a.view(16), a[:2], a.view(torch.int32), a.to("meta"), a.to_sparse(), None):
        assert not alike([a], [b])
    assert not alike([a], [a, a]) and not alike([a, a], [a]) and alike([], [])


def test_arguments():
    t = _lib.tensors()
    for bad in ((), ((), [], 0), ([], (), 0), ([], [], "x")):
        with pytest.raises(TypeError):
            t.gradients(*bad)
    for bad in (([],), ([], ()), (None, [])):
        with pytest.raises(TypeError):
            t.alike(*bad)


def test_a_build_for_another_pytorch_is_refused(monkeypatch):
    monkeypatch.setattr(_lib, "_tensors", None)
    monkeypatch.setattr(torch, "__version__", "0.1")
    with pytest.raises(RuntimeError, match="was built for PyTorch"):
        _lib.tensors()


def test_a_missing_build_is_refused(monkeypatch, tmp_path):
    monkeypatch.setattr(_lib, "_tensors", None)
    monkeypatch.setattr(_lib, "TENSORS_PATH", str(tmp_path / "none.so"))
    with pytest.raises(RuntimeError, match="is missing"):
        _lib.tensors()


def test_losses_leave_tensors_that_are_not_on_a_gpu_alone():
    t, x = _lib.tensors(), torch.zeros(2, 3)
    assert t.policy(0, 0, x, None, x, None, None, None, None, 0.2, 0.2, 0.0, 0.0, 2, 1, 0, 1) is None
    assert t.preference(0, 0, x, None, None, None, None, 0.1, 0.0, 0.0, 0, 0, 0) is None
    assert t.policy(0, 0, None, *[None] * 6, 0.2, 0.2, 0.0, 0.0, 2, 1, 0, 1) is None
    for f in (t.policy, t.preference):
        with pytest.raises(TypeError):
            f(0, 0, x)
