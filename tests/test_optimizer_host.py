"""What optim.AdamW keeps and hands on, with the library's calls replaced by recorders (no GPU needed)."""
import weakref

import pytest
import torch

from activation_sparse_gated_tcgen05_gb300 import twell
from activation_sparse_gated_tcgen05_gb300.optim import AdamW


class Calls(list):
    """Each step call: its number, its parameters, its keywords."""

    def step(self, params, step, **kw):
        self.append((step, list(params.tensors[0]), kw))
        self.grads = [weakref.ref(g) for g in params.tensors[2]]
        for p, c in zip(params.tensors[0], params.tensors[1]):
            for t in (p, c):  # as a kernel writes: unseen by autograd
                if t is not None:
                    t.detach().view(torch.int16).numpy()[:] += 1


@pytest.fixture
def calls(monkeypatch):
    seen = Calls()
    monkeypatch.setattr(twell, "_ptr", lambda t: None if t is None else t.data_ptr())
    monkeypatch.setattr(twell, "twell_adamw_step", seen.step)
    monkeypatch.setattr(twell, "twell_grad_norm", lambda grads, max_norm, out, ws: None)
    monkeypatch.setattr(twell, "twell_grad_norm_workspace_bytes", lambda: 16)
    return seen


def parameters(*sizes):
    return [torch.ones(n, requires_grad=True) for n in sizes]


def give_grads(params):
    for p in params:
        p.grad = torch.ones_like(p)


@pytest.mark.parametrize("max_norm", [None, 1.0])
def test_gradients_are_released(calls, max_norm):
    p, q = parameters(5, 7)
    w = torch.ones(4, 3, requires_grad=True)
    opt = AdamW([p, q, w], max_norm=max_norm)
    for _ in range(3):
        give_grads((p, q))
        w.grad = torch.ones(3, 4).t()  # the kernel gets a contiguous copy
        held = [weakref.ref(t.grad) for t in (p, q, w)]
        opt.step()
        opt.zero_grad()
        assert [r() for r in held + calls.grads] == [None] * 6


def test_dropped_gradients_are_not_used_again(monkeypatch):
    """A list without its gradients is refused before the library reads a pointer."""
    monkeypatch.setattr(twell, "_ptr", lambda t: None if t is None else t.data_ptr())
    p, g, m, v = (torch.ones(3) for _ in range(4))
    L = twell.TwellParams([p], [g], [m], [v])
    L.drop_grads()
    for call in (lambda: twell.twell_adamw_step(L, 1),
                 lambda: twell.twell_grad_norm(L, 1.0, torch.zeros(2), torch.zeros(16384, dtype=torch.uint8))):
        with pytest.raises(ValueError, match="dropped"):
            call()
    L.set_grads([g])
    assert L.tensors[2] == [g] and L.grad_dtype == 1


@pytest.mark.parametrize("copies", [False, True])
def test_autograd_sees_what_a_step_wrote(calls, copies):
    """A backward of a forward from before the step raises, as after the steps of PyTorch's optimizers."""
    p, q, idle = parameters(6, 4, 2)
    opt = AdamW([p, q, idle], bf16_copies=copies)
    give_grads((p, q))
    values = [t for t in (p, q) for t in ((t, opt.copy_of(t)) if copies else (t,))]
    before, other = [t._version for t in values], idle._version
    loss = (p * p).sum()
    opt.step()
    assert all(t._version > v for t, v in zip(values, before)) and idle._version == other
    with pytest.raises(RuntimeError, match="inplace"):
        loss.backward()
