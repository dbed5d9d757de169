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
