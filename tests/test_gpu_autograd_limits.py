"""What the autograd functions refuse and accept."""
import pytest
import torch

from activation_sparse_gated_tcgen05_gb300.autograd import (SparseGatedFFNFunction, policy_loss, preference_loss,
                                                            sparse_gated_ffn, token_logp)

pytestmark = pytest.mark.gpu


def randn(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


@pytest.mark.parametrize("which", ["token_logp", "policy_loss", "preference_loss"])
def test_second_derivatives_are_refused(which):
    """The backward is a kernel that autograd cannot see into: a derivative of the gradient raises, the gradient
    itself does not."""
    x = randn(6, 30).requires_grad_()
    y = torch.arange(6, device="cuda")
    loss = {"token_logp": lambda: token_logp(x, y).sum(),
            "policy_loss": lambda: policy_loss(x, y, torch.ones(6, device="cuda"))[0],
            "preference_loss": lambda: preference_loss(x, y, torch.tensor([0, 3, 6], device="cuda"))[0]}[which]
    once, = torch.autograd.grad(loss(), x)
    d, = torch.autograd.grad(loss() + (x ** 2).sum(), x, create_graph=True)
    assert torch.allclose(d.detach(), once + 2 * x.detach(), rtol=1e-6, atol=1e-6)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        d.square().sum().backward()
    # of the incoming gradient as well
    up = torch.ones((), device="cuda", requires_grad=True)
    d, = torch.autograd.grad(loss() * up, x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        torch.autograd.grad(d.sum(), up)


def test_ffn_function_without_copies():
    """The class itself with the nine arguments it had before it took bf16 copies."""
    x, ws = randn(64, 256).bfloat16(), [(randn(1024, 256, seed=k) * 0.06).requires_grad_() for k in (1, 2, 3)]
    y = SparseGatedFFNFunction.apply(x, *ws, 2e-5, 64, 16, 0.03, None)
    y.float().sum().backward()
    got = [w.grad for w in ws]
    for w in ws:
        w.grad = None
    z = sparse_gated_ffn(x, *ws, tile_n=64, tile_cap=16)
    z.float().sum().backward()
    assert torch.equal(y, z) and all(torch.equal(a, w.grad) for a, w in zip(got, ws))
