"""optim.AdamW as a PyTorch program uses it: what it holds, what it counts, and what autograd sees of its writes.
Tolerances of parameters: those of ten steps against torch's AdamW in fp64, 1e-5 (1 + |value|)."""
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
