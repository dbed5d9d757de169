"""What optim.AdamW keeps and hands on, with the library's calls replaced by recorders (no GPU needed)."""
import copy
import ctypes
import io
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


def test_steps_count_by_parameter(calls):
    """A parameter's first gradient is its step 1, whatever the others have behind them."""
    p, q, r = parameters(5, 7, 3)
    opt = AdamW([dict(params=[p, q]), dict(params=[r])])
    for live in ((p,), (p, r), (p, q, r), (q,), (p, q)):
        opt.zero_grad()
        give_grads(live)
        opt.step()
    steps = [(n, sorted(t.numel() for t in ps)) for n, ps, _ in calls]
    assert steps == [(1, [5]), (2, [5]), (1, [3]), (3, [5]), (1, [7]), (2, [3]), (2, [7]), (4, [5]), (3, [7])]
    # no two lists of a step share their random numbers
    third = [(kw["seed"], n) for n, _, kw in calls[3:6]]
    assert len(set(third)) == 3


def test_counts_survive_a_state_dict(calls):
    p, q = parameters(5, 7)
    opt = AdamW([p, q], state_bits=8)
    for live in ((p,), (p, q)):
        opt.zero_grad()
        give_grads(live)
        opt.step()
    other = AdamW(parameters(5, 7), state_bits=8)
    other.load_state_dict(copy.deepcopy(opt.state_dict()))
    calls.clear()
    give_grads(other.param_groups[0]["params"])
    other.step()
    assert sorted((n, ps[0].numel()) for n, ps, _ in calls) == [(2, 7), (3, 5)]
    assert set(other.state_dict()["state"][0]) == set(opt.state_dict()["state"][0])


def test_a_state_dict_that_counts_by_group(calls):
    """Groups that hold the step for all their parameters, as this class wrote them before."""
    p, q = parameters(5, 7)
    moments = {i: {k: torch.full((n,), 0.5) for k in ("m", "v")} for i, n in enumerate((5, 7))}
    group = dict(lr=0.5, betas=(0.9, 0.99), eps=1e-8, weight_decay=0.0, step=41, params=[0, 1])
    opt = AdamW([p, q])
    opt.load_state_dict(dict(state=moments, param_groups=[group]))
    give_grads((p, q))
    opt.step()
    assert [(n, len(ps), kw["lr"]) for n, ps, kw in calls] == [(42, 2, 0.5)]
    assert float(opt.state[p]["m"][0]) == 0.5


def test_skipped_counts_are_shared_by_those_that_step_together(calls):
    """One count for each list: parameters that part take their own copy along, none is raised twice a step."""
    p, q, h = torch.ones(5, requires_grad=True), torch.ones(7, requires_grad=True), torch.ones(3).bfloat16().requires_grad_()
    opt = AdamW([p, q, h])

    def step(*live):
        calls.clear()
        opt.zero_grad()
        give_grads(live)
        opt.step()
        for _, ps, kw in calls:  # a skipped step, as the kernel counts it
            kw["skipped"].add_(1)
        return [kw["skipped"] for _, _, kw in calls]

    def counts():
        return [int(opt.state[t]["skipped"]) for t in (p, q, h)]

    one, two = step(p, q, h)
    assert one is not two and counts() == [1, 1, 1]
    assert [x is y for x, y in zip(step(p, q, h), (one, two))] == [True, True]
    alone, = step(p)
    assert alone is not one and counts() == [3, 2, 2]
    assert len({id(x) for x in step(p, q, h)}) == 3 and counts() == [4, 3, 3]
    other = AdamW([torch.ones(n, requires_grad=True) for n in (5, 7)] + [torch.ones(3).bfloat16().requires_grad_()])
    other.load_state_dict(copy.deepcopy(opt.state_dict()))
    calls.clear()
    give_grads(other.param_groups[0]["params"])
    other.step()
    assert sorted(int(kw["skipped"]) for _, _, kw in calls) == [3, 3, 4]
    assert len({kw["skipped"].data_ptr() for _, _, kw in calls}) == 3


def test_skipped_count_is_checked():
    lib = twell.load()
    args = (1e-3, 0.9, 0.999, 1e-8, 0.0, 1, 0, None, 1, 1, 32)
    assert lib.twell_adamw_step(None, 0, ctypes.byref(twell.AdamW(*args, 18)), None) == 3
    assert lib.twell_adamw_step(None, 0, ctypes.byref(twell.AdamW(*args, 16)), None) == 0


@pytest.mark.parametrize("how", ["deepcopy", "pickle"])
def test_copies_of_an_optimizer(calls, how):
    """A copied or pickled optimizer has its options, its parameters' states and bf16 copies, and steps."""
    p, q = parameters(5, 7)
    opt = AdamW([p, q], lr=0.25, state_bits=8, max_norm=2.0, bf16_copies=True, seed=9)
    give_grads((p,))
    opt.step()
    assert not opt.state[q]  # looked at, never stepped
    if how == "deepcopy":
        other = copy.deepcopy(opt)
    else:
        buf = io.BytesIO()
        torch.save(opt, buf)
        buf.seek(0)
        other = torch.load(buf, weights_only=False)
    assert (other.state_bits, other.max_norm, other.seed, other.param_groups[0]["lr"]) == (8, 2.0, 9, 0.25)
    p2, q2 = other.param_groups[0]["params"]
    assert p2 is not p and torch.equal(p2, p) and torch.equal(other.copy_of(p2), opt.copy_of(p))
    assert other.copy_of(p2).data_ptr() != opt.copy_of(p).data_ptr()
    calls.clear()
    give_grads((p2, q2))
    other.step()
    assert sorted((n, t[0].data_ptr()) for n, t, _ in calls) == sorted([(2, p2.data_ptr()), (1, q2.data_ptr())])
    # what the copy does not do to the original
    assert "m" not in opt.state[q] and p.grad is not None
