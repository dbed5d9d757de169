"""optim.AdamW as a PyTorch program uses it: what it holds, what it counts, and what autograd sees of its writes.
Tolerances of parameters: those of ten steps against torch's AdamW in fp64, 1e-5 (1 + |value|)."""
import pytest
import torch

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
