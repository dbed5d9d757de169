"""Gradients of logits with a large common offset, of rows filled with a mask value, and of large scales,
through every kernel that writes gradients, against torch in 64 bits.

Tolerance: as for ordinary logits.  The exponent's argument is the difference from the row's maximum times
scale log2(e), each rounded once, 2e-7 of an argument t; p t stays below p (t < 100 where p counts), so 2e-5 of
(onehot + p) |c| covers it, with the sum's and the coefficient's own errors; the entry is rounded once (2^-8 of
itself in bf16).  Exponentials below 2^-126 are zero: 1e-37 at most.
"""
import pytest
import torch

from activation_sparse_gated_tcgen05_gb300 import twell

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
# around 2^14 / log2(e) = 11357, then every magnitude up to the type's range
OFFSETS = [0.0, 11000.0, -11300.0, 11400.0, -14000.0, 1e5, -1e5, 1e6, -1e6, 1e7, 3e7, -1e9, 1e9, 1e20, -1e20, 6e37,
           -8e37, 3e38]
# a warp, a block and a cluster to a row; many short rows; rings of 4, 8 and 16 warps
SHAPES = [(36, 700, "bf16"), (36, 700, "f32"), (36, 9001, "bf16"), (36, 9001, "f32"), (20, 140000, "bf16"),
          (20, 70001, "f32"), (2500, 7000, "bf16"), (3700, 21001, "bf16"), (3650, 12001, "f32"), (320, 60001, "bf16"),
          (306, 40001, "f32"), (160, 90001, "bf16"), (160, 50003, "f32")]


def rows(n):
    return [torch.full((n,), float("nan"), device="cuda") for _ in range(4)]


def worst(got, data, target, coef, scale):
    """Largest excess over the bound; rows a few at a time.  coef: d loss / d logp."""
    out = torch.zeros((), dtype=torch.float64, device="cuda")
    eps = 2.0 ** -8 if data.dtype == torch.bfloat16 else 1e-6
    for a in range(0, data.shape[0], 256):
        at = slice(a, min(data.shape[0], a + 256))
        z, y = data[at].double(), target[at][:, None]
        p = torch.softmax((z - z.amax(1, keepdim=True)) * scale, 1)
        c = scale * coef[at].double()[:, None]
        one = torch.zeros_like(p).scatter_(1, y, 1.0)
        want = c * (one - p)
        bound = 2e-5 * c.abs() * (one + p) + eps * want.abs() + 1e-37 * max(1.0, scale)
        off = (got[at].double() - want).abs() - bound
        out = torch.maximum(out, torch.where(torch.isfinite(off), off, float("inf")).max())
    return float(out)


def check(data, target, scale=1.0):
    T = data.shape[0]
    adv = torch.randn(T, generator=torch.Generator(device="cuda").manual_seed(T), device="cuda")
    L, P = twell.TwellLogits(data, target, scale), twell.TwellPolicy(adv)
    tok, logp, lse, coef = rows(T)
    d, loss = torch.full_like(data, float("nan")), torch.zeros((), device="cuda")
    twell.twell_policy_loss(L, P, loss, tok, logp, lse, coef, dlogits=d)
    assert worst(d, data, target, -adv, scale) <= 0.0
    two = torch.full_like(data, float("nan"))
    twell.twell_policy_loss(L, P, loss, tok, logp, lse, coef)
    twell.twell_logp_bwd(L, lse, coef, two)
    assert worst(two, data, target, -adv, scale) <= 0.0
    # in place of the logits
    for call in (lambda M: twell.twell_policy_loss(M, P, loss, tok, logp, lse, coef, dlogits=M.data),
                 lambda M: twell.twell_logp_bwd(M, lse, coef, M.data)):
        M = twell.TwellLogits(data.clone(), target, scale)
        call(M)
        assert worst(M.data, data, target, -adv, scale) <= 0.0
    assert twell.twell_get_device_status() == 0


@pytest.mark.parametrize("T,V,dtype", SHAPES)
def test_offsets_of_every_size(T, V, dtype):
    """Each row has an offset of its own; every third row is filled with it (a row of nothing but a mask
    value) and scores a token as likely as any other."""
    g = torch.Generator(device="cuda").manual_seed(T + V)
    x = torch.randn(T, V, generator=g, device="cuda") * 2.5
    x[::3] = 0.0
    offset = torch.tensor([OFFSETS[t % len(OFFSETS)] for t in range(T)], device="cuda")
    data = x.add_(offset[:, None]).to(DT[dtype])
    target = torch.randint(0, V, (T,), generator=g, device="cuda")
    check(data, target)


@pytest.mark.parametrize("T,V,dtype", [(36, 700, "f32"), (36, 9001, "f32"), (3650, 12001, "f32"), (160, 50003, "f32"),
                                       (160, 90001, "bf16")])
@pytest.mark.parametrize("scale", [1e6, 1e-3])
def test_scales(T, V, dtype, scale):
    """At scale 1e6 the logits lie a few units of their type from one another around 20 (fp32: 1.9 after the
    scale; bf16: equal)."""
    g = torch.Generator(device="cuda").manual_seed(T + V)
    x = torch.randn(T, V, generator=g, device="cuda")
    data = (20.0 + x * (2e-6 if scale > 1 else 100.0)).to(DT[dtype])
    data[::3] = -1e9
    target = torch.randint(0, V, (T,), generator=g, device="cuda")
    check(data, target, float(torch.tensor(scale, dtype=torch.float32)))
