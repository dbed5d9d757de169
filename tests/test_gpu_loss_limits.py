"""Losses at the limits of their formulas: what a term that does not count must not do to the ones that do."""
import numpy as np
import pytest
import torch

from activation_sparse_gated_tcgen05_gb300 import twell

from step_reference import logits_reference, policy_reference

pytestmark = pytest.mark.gpu


def rows(n):
    return [torch.full((n,), float("nan"), device="cuda") for _ in range(4)]


def logits(T, V, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, V, generator=g, device="cuda")
    return x, torch.randint(0, V, (T,), generator=g, device="cuda")


@pytest.mark.parametrize("T,V", [(8, 40), (8, 9000), (160, 50001)])
def test_no_advantage_under_a_ratio_past_the_type(T, V):
    """exp(logp - old) overflows fp32, the advantage is 0: the term and its gradient are 0, the KL term's stay.
    In 64 bits the ratio is finite."""
    x, y = logits(T, V)
    _, lp, _, live = logits_reference(x.double().cpu().numpy(), y.cpu().numpy())
    old, ref, adv = lp - 0.05, lp + 0.1, np.ones(T)
    old[::2] -= 100.0
    adv[::2] = 0.0
    dev = [torch.tensor(a, dtype=torch.float32, device="cuda") for a in (adv, old, ref)]
    want, c = policy_reference(lp, live, adv, None, old, ref, kl=0.1)
    for grad in (torch.empty_like(x), None):
        tok, logp, lse, coef = rows(T)
        loss = torch.zeros((), device="cuda")
        twell.twell_policy_loss(twell.TwellLogits(x, y), twell.TwellPolicy(dev[0], None, dev[1], dev[2], kl_coeff=0.1), loss,
                                tok, logp, lse, coef, dlogits=grad)
        # |A| r and the KL term's parts are at most 1.3, each off by a log-probability's 5e-6 + 1e-6 |value|
        assert np.all(np.abs(tok.double().cpu().numpy() - want) <= 4e-5)
        assert np.all(np.abs(coef.double().cpu().numpy() - c) <= 4e-5)
        assert abs(float(loss) - want.sum()) <= 4e-5 * T
        assert grad is None or bool(torch.isfinite(grad).all())


def test_no_advantage_keeps_a_row_that_is_nan():
    x, y = logits(4, 60)
    x[1, 3] = float("nan")
    tok, logp, lse, coef = rows(4)
    zero = torch.zeros(4, device="cuda")
    twell.twell_policy_loss(twell.TwellLogits(x, y), twell.TwellPolicy(zero, None, zero - 100.0), zero[:1].clone(), tok, logp,
                            lse, coef)
    assert torch.isnan(tok).tolist() == torch.isnan(coef).tolist() == [False, True, False, False]


def preference(x, y, start, **kw):
    T, pairs = x.shape[0], start.numel() // 2
    o = [torch.full((n,), float("nan"), device="cuda") for n in (1, pairs, 2 * pairs, T, T, T)]
    twell.twell_preference_loss(twell.TwellLogits(x, y), twell.TwellPreference(start, **kw), *o)
    return o


def test_rejected_answer_without_probability():
    """A rejected token of probability zero: the margin is infinite and the pair's loss 0, as
    -log sigmoid(inf) is; with smoothing the loss is infinite."""
    x, y = logits(8, 50)
    x[3, y[3]] = float("-inf")
    start = torch.tensor([0, 2, 4, 6, 8], device="cuda")
    loss, pair, gain, logp, lse, coef = preference(x, y, start, beta=0.5)
    other = preference(x[4:].contiguous(), y[4:].contiguous(), start[:3], beta=0.5)
    assert float(gain[1]) == float("-inf") and float(pair[0]) == 0.0
    assert torch.equal(pair[1:], other[1]) and abs(float(loss) - 0.5 * float(other[0])) <= 1e-6 * float(other[0])
    assert bool((coef[:4] == 0).all()) and bool((coef[4:] != 0).all())
    d = torch.full_like(x, float("nan"))
    twell.twell_logp_bwd(twell.TwellLogits(x, y), lse, coef, d)
    assert bool((d[:4] == 0).all()) and bool(torch.isfinite(d).all())
    assert float(preference(x, y, start, beta=0.5, label_smoothing=0.1)[1][0]) == float("inf")


@pytest.mark.parametrize("T,V", [(5, 300), (3, 9000), (3, 90000)])
@pytest.mark.parametrize("scale", [1e-36, 1e-38])
def test_masked_entries_at_the_smallest_scales(T, V, scale):
    """softmax(scale x) is uniform over what is not masked; ln of the count is right to 1e-6 and logp to LP."""
    x, y = logits(T, V)
    x[:, 1::2] = float("-inf")
    y = y - y % 2
    tok, logp, lse, coef = rows(T)
    twell.twell_token_logp(twell.TwellLogits(x, y, scale), logp, lse)
    want = -np.log((V + 1) // 2)
    assert np.all(np.abs(logp.double().cpu().numpy() - want) <= 5e-6 + 1e-6 * abs(want))
    x[0] = float("-inf")
    twell.twell_token_logp(twell.TwellLogits(x, y, scale), logp, lse)
    assert bool(torch.isnan(logp[0])) and bool(torch.isfinite(logp[1:]).all())
