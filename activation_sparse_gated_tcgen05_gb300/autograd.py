"""PyTorch autograd bindings of the sparse gated FFN and of the losses over
logits that train a model built on it.

Forward: gate GEMM with the TwELL pack in its epilogue, hybrid ELL / dense
routing, fused sparse up+down projection.  Backward: the sparse backward with
the L1 term on the gate activations (page 2 "Sakana AI and NVIDIA introduce
TwELL with CUDA kernels ...", sections "¿Qué hace distinto a TwELL frente a
ELL clásico?" and "Receta de entrenamiento").  This module only marshals
arguments to the C ABI (twell.py); every step runs in the library's kernels.

Weights are neuron-major [d_ff][d_model] (WgT, WuT, Wd).  They may be fp32
master parameters: the bf16 copies the kernels read are made here, and the
library's fp32 weight gradients are returned unrounded.  A program that keeps
bf16 copies of its masters (the optimizer of optim.py writes them) passes
them as `bf16`, and nothing is cast.

``token_logp``, ``policy_loss`` and ``preference_loss`` take logits [rows][vocab]
(bf16 or fp32, rows contiguous) and return fp32 results; their backward is one
kernel that reads the logits again, so they hold nothing of the logits' size
between forward and backward.  It has no derivative of its own: a second
derivative raises.  A training loop that wants loss and gradient
of the policy loss in one pass calls twell.twell_policy_loss with `dlogits`.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import twell


def ell_width_for(row_nnz: torch.Tensor, route_fraction: float) -> int:
    """ELL width W that routes about `route_fraction` of the rows to the dense
    fallback: the row count at sorted index floor((1 - route_fraction) * M)
    (the widest row when route_fraction = 0).  Reads the counts on the host."""
    M = row_nnz.numel()
    if M == 0:
        return 0
    s = torch.sort(row_nnz.to(torch.int64)).values
    if route_fraction <= 0:
        return int(s[-1].item())
    return int(s[min(M - 1, int((1.0 - route_fraction) * M))].item())


class SparseGatedFFNFunction(torch.autograd.Function):
    """y = (ReLU(x Wg) * (x Wu)) Wd with the gate packed into TwELL and
    consumed sparsely; backward adds l1_coeff to dL/da at every live entry."""

    @staticmethod
    def forward(ctx, x, wgT, wuT, wd, l1_coeff: float, tile_n: int, tile_cap: int,
                route_fraction: float, stats: Optional[dict], bf16=None):
        if x.dim() != 2:
            raise ValueError("x must be [tokens][d_model]")
        if bf16 is not None and not (len(bf16) == 3 and all(
                c.dtype == torch.bfloat16 and c.shape == w.shape
                for c, w in zip(bf16, (wgT, wuT, wd)))):
            raise ValueError("bf16 must be the bfloat16 copies of wgT, wuT and wd")
        M, d = x.shape
        f = wgT.shape[0]
        xb = x.to(torch.bfloat16).contiguous()
        wg, wu, wdb = (w.detach().to(torch.bfloat16).contiguous() for w in bf16 or (wgT, wuT, wd))
        shape = twell.make_shape(M, d, f, tile_n, tile_cap)
        tiles = twell.alloc_tiles(shape, x.device)
        twell.twell_pack(xb, wg, shape, tiles)
        row_nnz = twell.tiles_view(tiles, shape)[3]
        W = ell_width_for(row_nnz, route_fraction)
        route = twell.alloc_hybrid(shape, W, x.device)
        twell.hybrid_route(tiles, shape, route)
        # the routed-row count is on the device: read it and size the
        # workspace's dense-backup buffers for exactly those rows
        n_dense = int(route.n_dense[0].item())
        route.dense_cap = n_dense
        ws = torch.empty(twell.twell_workspace_bytes(shape, W, True, dense_cap=n_dense),
                         dtype=torch.uint8, device=x.device)
        y = torch.empty(M, d, dtype=torch.bfloat16, device=x.device)
        twell.twell_ffn_fwd(xb, wg, wu, wdb, shape, y, route=route, ws=ws)
        if stats is not None:
            stats["density"] = float(row_nnz.to(torch.float64).sum().item()) / max(1, M * f)
            stats["ell_width"] = W
            stats["routed_rows"] = n_dense
            stats["workspace_bytes"] = ws.numel()
        ctx.save_for_backward(xb, wg, wu, wdb)
        ctx.shape, ctx.route, ctx.ws, ctx.l1 = shape, route, ws, float(l1_coeff)
        ctx.in_dtypes = (x.dtype, wgT.dtype, wuT.dtype, wd.dtype)
        return y

    @staticmethod
    def backward(ctx, dy):
        xb, wg, wu, wdb = ctx.saved_tensors
        shape = ctx.shape
        dyb = dy.to(torch.bfloat16).contiguous()
        dx = torch.empty_like(xb)
        f, d = shape.d_ff, shape.d_model
        dws = [torch.empty(f, d, dtype=torch.float32, device=xb.device) for _ in range(3)]
        twell.twell_ffn_bwd(xb, wg, wu, wdb, dyb, shape, ctx.route, ctx.l1, dx, *dws, ctx.ws)
        xt, gt, ut, dt = ctx.in_dtypes
        grads = [g if g.dtype == t else g.to(t) for g, t in zip(dws, (gt, ut, dt))]
        return (dx if dx.dtype == xt else dx.to(xt), *grads, None, None, None, None, None, None)


def sparse_gated_ffn(x, wgT, wuT, wd, l1_coeff: float = 2e-5, tile_n: int = 128,
                     tile_cap: int = 32, route_fraction: float = 0.03,
                     stats: Optional[dict] = None, bf16=None):
    """Functional form; `stats`, if given, receives the gate density, the ELL
    width and the number of routed rows of this call (host reads).  `bf16`: bf16
    copies of (wgT, wuT, wd) to compute with in place of casting them here."""
    return SparseGatedFFNFunction.apply(x, wgT, wuT, wd, l1_coeff, tile_n, tile_cap,
                                        route_fraction, stats, bf16)


def _rows(n: int, like: torch.Tensor) -> torch.Tensor:
    return torch.empty(n, dtype=torch.float32, device=like.device)


def _vector(t):
    """fp32 contiguous form of a per-row argument (None stays None)."""
    return None if t is None else t.detach().to(torch.float32).contiguous()


class _Once(torch.autograd.Function):
    """A gradient that a kernel wrote, with what it depends on: its own derivative raises.  (PyTorch's
    once_differentiable looks at the incoming gradient alone, not at the logits.)"""

    @staticmethod
    def forward(ctx, d, *of):
        return d

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError("the losses over logits are once_differentiable: their gradients are a "
                           "kernel's and have no derivative")


def _once(d, *of):
    return _Once.apply(d, *of) if torch.is_grad_enabled() else d


class _TokenLogp(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, target, scale: float):
        L = twell.TwellLogits(logits.detach(), target, scale)
        logp, lse = _rows(L.rows, logits), _rows(L.rows, logits)
        twell.twell_token_logp(L, logp, lse)
        ctx.save_for_backward(logits, target, lse)
        ctx.scale = scale
        return logp

    @staticmethod
    def backward(ctx, dlogp):
        logits, target, lse = ctx.saved_tensors
        d = torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)
        twell.twell_logp_bwd(twell.TwellLogits(logits.detach(), target, ctx.scale), lse,
                             _vector(dlogp), d)
        return _once(d, logits, dlogp), None, None


def token_logp(logits, target, scale: float = 1.0):
    """Log-probability of each row's target under softmax(scale * logits), fp32 [rows];
    0 (and no gradient) for rows whose target is negative."""
    return _TokenLogp.apply(logits, target.contiguous(), float(scale))


class _CoefLoss(torch.autograd.Function):
    """A scalar loss of the targets' log-probabilities: `call(L, loss, logp, lse, coef)`
    computes it with its derivatives coef."""

    @staticmethod
    def forward(ctx, logits, target, scale: float, call):
        L = twell.TwellLogits(logits.detach(), target, scale)
        loss = torch.empty((), dtype=torch.float32, device=logits.device)
        logp, lse, coef = (_rows(L.rows, logits) for _ in range(3))
        call(L, loss, logp, lse, coef)
        ctx.save_for_backward(logits, target, lse, coef)
        ctx.scale = scale
        ctx.mark_non_differentiable(logp)
        return loss, logp

    @staticmethod
    def backward(ctx, dloss, _dlogp):
        logits, target, lse, coef = ctx.saved_tensors
        d = torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)
        twell.twell_logp_bwd(twell.TwellLogits(logits.detach(), target, ctx.scale), lse, coef, d,
                             dloss=_vector(dloss))
        return _once(d, logits, dloss), None, None, None


def policy_loss(logits, target, advantage, weight=None, old_logp=None, ref_logp=None,
                clip_low: float = 0.2, clip_high: float = 0.2, kl_coeff: float = 0.0,
                scale: float = 1.0):
    """(loss, logp): the clipped policy loss with its KL term, summed over the rows with their
    weights (see twell_policy_loss in include/twell.h), and the rows' log-probabilities, which
    carry no gradient."""
    policy = twell.TwellPolicy(*(_vector(t) for t in (advantage, weight, old_logp, ref_logp)),
                               clip_low=clip_low, clip_high=clip_high, kl_coeff=kl_coeff)

    def call(L, loss, logp, lse, coef):
        twell.twell_policy_loss(L, policy, loss, _rows(L.rows, loss), logp, lse, coef)

    return _CoefLoss.apply(logits, target.contiguous(), float(scale), call)


def preference_loss(logits, target, seq_start, ref_logp=None, beta: float = 0.1,
                    label_smoothing: float = 0.0, scale: float = 1.0):
    """(loss, logp): the mean preference loss over the pairs of sequences in seq_start (int64
    [2 pairs + 1]: sequence 2 p is the chosen answer of pair p, 2 p + 1 the rejected one; see
    twell_preference_loss in include/twell.h), and the rows' log-probabilities, which carry no
    gradient."""
    pref = twell.TwellPreference(seq_start.contiguous(), _vector(ref_logp), beta, label_smoothing)

    def call(L, loss, logp, lse, coef):
        twell.twell_preference_loss(L, pref, loss, _rows(pref.pairs, loss),
                                    _rows(2 * pref.pairs, loss), logp, lse, coef)

    return _CoefLoss.apply(logits, target.contiguous(), float(scale), call)
