"""optim.AdamW as a PyTorch program uses it: what it holds, what it counts, and what autograd sees of its writes.
Tolerances of parameters: those of ten steps against torch's AdamW in fp64, 1e-5 (1 + |value|)."""
import copy

import pytest
import torch

from activation_sparse_gated_tcgen05_gb300 import twell
from activation_sparse_gated_tcgen05_gb300.autograd import sparse_gated_ffn
from activation_sparse_gated_tcgen05_gb300.optim import AdamW

pytestmark = pytest.mark.gpu


def randn(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


def test_gradients_are_released():
    p = torch.zeros(1 << 22, device="cuda", requires_grad=True)
    opt = AdamW([p], max_norm=1.0)
    p.grad = torch.ones_like(p)
    opt.step()
    held = torch.cuda.memory_allocated()
    opt.zero_grad()
    assert held - torch.cuda.memory_allocated() >= 4 << 22


@pytest.mark.parametrize("copies", [False, True])
def test_backward_after_a_step_raises(copies):
    """The FFN keeps the bf16 copies themselves for its backward: a step in between must not go unseen."""
    ws = [(randn(1024, 256, seed=k) * 0.06).requires_grad_() for k in range(3)]
    if not copies:
        ws = [w.detach().bfloat16().requires_grad_() for w in ws]
    opt = AdamW(ws, bf16_copies=copies)
    x = randn(64, 256, seed=5).bfloat16()

    def forward():
        return sparse_gated_ffn(x, *ws, tile_n=64, tile_cap=16, bf16=[opt.copy_of(w) for w in ws]).float().sum()

    forward().backward()
    late = forward()
    opt.step()
    with pytest.raises(RuntimeError, match="inplace"):
        late.backward()
    opt.zero_grad()
    forward().backward()  # a forward of the new weights
    opt.step()
    assert twell.twell_get_device_status() == 0


def compare(ours, theirs, begin):
    for p, q, s in zip(ours, theirs, begin):
        off = (p.detach().double() - q.detach()).abs()
        assert float((off - 1e-5 * (1 + s.abs())).max()) <= 0


def pair(sizes, seed=0):
    ours = [randn(n, seed=seed + k).requires_grad_() for k, n in enumerate(sizes)]
    return ours, [p.detach().double().clone().requires_grad_() for p in ours], [p.detach().double() for p in ours]


def test_late_parameters_against_torch():
    """Parameters that get their first gradient after 20 steps, or get one now and then."""
    ours, theirs, begin = pair((300, 40, 1000))
    a = AdamW(ours, lr=5e-3, weight_decay=0.1)
    b = torch.optim.AdamW(theirs, lr=5e-3, weight_decay=0.1)
    g = torch.Generator(device="cuda").manual_seed(3)
    for step in range(30):
        live = [True, step >= 20, step % 3 == 1]
        for p, q, on in zip(ours, theirs, live):
            grad = torch.randn(p.shape, generator=g, device="cuda") + 0.5
            p.grad, q.grad = (grad, grad.double()) if on else (None, None)
        a.step()
        b.step()
    compare(ours, theirs, begin)


@pytest.mark.parametrize("bits", [8, 32])
def test_the_first_step_of_a_late_parameter(bits):
    """Moments start at zero: |update| = lr |g| / (|g| + eps), whatever the other parameters' step."""
    p, q = randn(600).requires_grad_(), torch.zeros(600, device="cuda", requires_grad=True)
    opt = AdamW([p, q], lr=1e-2, weight_decay=0.0, state_bits=bits)
    for _ in range(50):
        p.grad = randn(600, seed=1)
        opt.step()
    q.grad = torch.sign(randn(600, seed=2)) * 0.3
    opt.step()
    assert torch.allclose(q.detach(), -1e-2 * torch.sign(q.grad), rtol=1e-5, atol=0.0)


def test_skipped_steps_against_torch():
    """A step whose norm is not finite is as if it had not been: torch's AdamW does not get it.  One parameter
    has no gradient in some of them, and one comes after the first of them."""
    ours, theirs, begin = pair((300, 40, 1000))
    a = AdamW([dict(params=ours[:2]), dict(params=ours[2:], lr=1e-2)], lr=5e-3, weight_decay=0.1, max_norm=1e4)
    b = torch.optim.AdamW([dict(params=theirs[:2]), dict(params=theirs[2:], lr=1e-2)], lr=5e-3, weight_decay=0.1)
    g = torch.Generator(device="cuda").manual_seed(3)
    for step in range(24):
        bad = step in (0, 1, 5, 6, 15)
        live = [True, step >= 3 and step != 6, step % 2 == 1 or step == 0]
        for p, q, on in zip(ours, theirs, live):
            grad = torch.randn(p.shape, generator=g, device="cuda") + 0.5
            p.grad, q.grad = (grad, grad.double()) if on else (None, None)
        if bad:
            ours[0].grad[7] = float("inf") if step % 2 else float("nan")
        a.step()
        if not bad:
            b.step()
    compare(ours, theirs, begin)
    assert bool(torch.isfinite(a.last_norm).all())


@pytest.mark.parametrize("bits", [8, 32])
def test_skipped_steps_survive_a_state_dict(bits):
    p, q = randn(700).requires_grad_(), randn(90, seed=4).requires_grad_()
    opt = AdamW([p, q], state_bits=bits, max_norm=1.0, seed=3)
    for step in range(5):
        p.grad, q.grad = randn(700, seed=step), randn(90, seed=step + 50) if step else None
        if step in (0, 3):
            p.grad[0] = float("nan")
        opt.step()
    others = [p.detach().clone().requires_grad_(), q.detach().clone().requires_grad_()]
    new = AdamW(others, state_bits=bits, max_norm=1.0, seed=3)
    new.load_state_dict(copy.deepcopy(opt.state_dict()))
    for step in range(5, 8):
        for o, params in ((opt, (p, q)), (new, others)):
            for k, x in enumerate(params):
                x.grad = randn(x.numel(), seed=step + 10 * k)
                if step == 6 and k == 0:
                    x.grad[1] = float("inf")
            o.step()
    assert torch.equal(p, others[0]) and torch.equal(q, others[1])


@pytest.mark.parametrize("bits", [8, 32])
def test_skipped_count_of_a_call(bits):
    """One call adds one, over however many launches its list takes, and only if it changed nothing; its
    corrections are those of step - skipped."""
    def params(seed):
        ps = [randn(37 + k % 5, seed=seed + k) for k in range(900)]
        st = [twell.alloc_adamw_state(p, bits) for p in ps]
        k8 = {} if bits == 32 else {k: [s[k] for s in st] for k in ("m_scale", "v_scale")}
        gs = [torch.ones_like(p) * 1e-2 for p in ps]
        return ps, twell.TwellParams(ps, gs, [s["m"] for s in st], [s["v"] for s in st], **k8)

    (a, A), (b, B) = params(0), params(0)
    skipped, scale = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.ones(1, device="cuda")
    for step, s in enumerate((1.0, float("nan"), float("inf"), 1.0), 1):
        scale.fill_(s)
        twell.twell_adamw_step(A, step, grad_scale=scale, skipped=skipped)
    assert int(skipped) == 2
    for step in (1, 2):
        twell.twell_adamw_step(B, step)
    for x, y in zip(a, b):
        # step 2 against step 4 less two: the corrections in fp32, a few 2^-24 of an update of lr
        assert float((x - y).abs().max()) <= 1e-8 + 2.0 ** -23 * float(x.abs().max())
    twell.twell_adamw_step(B, 3, grad_scale=torch.full((1,), float("nan"), device="cuda"))  # without a count
    with pytest.raises(ValueError, match="skipped"):
        twell.twell_adamw_step(B, 3, skipped=torch.zeros(1, device="cuda"))


def test_deepcopy_steps_on():
    p = randn(500).requires_grad_()
    opt = AdamW([p], bf16_copies=True, state_bits=8, max_norm=1.0, seed=2)
    p.grad = randn(500, seed=1)
    opt.step()
    other = copy.deepcopy(opt)
    (q,) = other.param_groups[0]["params"]
    q.grad = p.grad.clone()
    opt.step()
    other.step()
    assert torch.equal(p, q) and torch.equal(opt.copy_of(p), other.copy_of(q)) and opt.copy_of(p) is not other.copy_of(q)


def test_a_gradient_laid_out_another_way():
    """A transposed gradient's elements meet their own parameters.  The first step moves each by lr against its
    gradient's sign; none is 0."""
    w = randn(8, 16).requires_grad_()
    opt = AdamW([w], lr=0.1, weight_decay=0.0)
    w.grad = (torch.arange(128.0, device="cuda").view(16, 8) - 60.5).t()
    before = w.detach().clone()
    opt.step()
    # lr g / (|g| + eps): 0.1 to a few 2^-24 of the parameter
    assert torch.allclose(before - w.detach(), 0.1 * torch.sign(w.grad), rtol=0.0, atol=2e-6)
