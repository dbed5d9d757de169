"""AdamW over all parameters of a model in a few launches, with 32-bit or 8-bit
states, the clipping of the gradients' global norm, and the bf16 copies of
fp32 masters that the FFN's kernels read.

The class holds parameters and states as PyTorch optimizers do and marshals
them to twell_grad_norm and twell_adamw_step (include/twell.h), which do the
arithmetic.
"""
from __future__ import annotations

import torch

from . import twell


class AdamW(torch.optim.Optimizer):
    """params: tensors or groups, on one GPU, contiguous, fp32 or bf16.

    state_bits   32 (fp32 moments) or 8 (e4m3 codes with a scale for each 256 elements, rounded
                 stochastically; `seed` and the step choose the random numbers).  The stored
                 sqrt(v) is right on average and scatters around it, a step's size with it: 17 %
                 (mean + 1.3 %) after 4000 steps of random gradients at beta2 = 0.999
    max_norm     clips the global norm of all gradients (all fp32 or all bf16 then).  A step
                 whose norm is not finite changes nothing.  `last_norm` (fp32 [2] on the GPU)
                 holds the last norm and the factor it led to
    bf16_copies  keeps a bf16 copy of every fp32 parameter, see copy_of()

    lr, betas, eps, weight_decay may differ between groups.  Steps are counted for each
    parameter from its first gradient on (state[p]["step"]); those that changed nothing are
    counted on the GPU (state[p]["skipped"]) and do not count for the bias corrections.  step()
    launches on the current stream and reads nothing back."""

    def __init__(self, params, lr: float = 1e-3, betas=(0.9, 0.999), eps: float = 1e-8,
                 weight_decay: float = 0.01, state_bits: int = 32, max_norm: float = None,
                 bf16_copies: bool = False, seed: int = 0):
        if state_bits not in (8, 32):
            raise ValueError("state_bits must be 8 or 32")
        if not lr >= 0.0 or not eps >= 0.0 or not weight_decay >= 0.0:
            raise ValueError("lr, eps and weight_decay must not be negative")
        if not all(0.0 <= b < 1.0 for b in betas):
            raise ValueError("betas must lie in [0, 1)")
        if max_norm is not None and not max_norm > 0.0:
            raise ValueError("max_norm must be positive")
        self.state_bits, self.max_norm, self.seed = state_bits, max_norm, int(seed)
        self._keep_copies, self._copies, self._lists = bf16_copies, {}, {}
        self._skips = {}  # each skipped count by its id: the tensor, how many parameters share it
        self.last_norm, self._ws = None, None
        super().__init__(params, dict(lr=lr, betas=tuple(betas), eps=eps,
                                      weight_decay=weight_decay))

    def __getstate__(self):
        """For copy and pickle: PyTorch's part and the options, the copies and the last norm; what
        describes or shares tensors is made anew."""
        keep = ("state_bits", "max_norm", "seed", "_keep_copies", "_copies", "last_norm")
        return dict(super().__getstate__(), **{k: getattr(self, k) for k in keep})

    def __setstate__(self, state):
        super().__setstate__(state)
        self._lists, self._skips, self._ws = {}, {}, None
        for st in self.state.values():
            count = st.get("skipped")
            if count is not None:
                self._skips.setdefault(id(count), [count, 0])[1] += 1

    def add_param_group(self, group):
        super().add_param_group(group)
        for p in self.param_groups[-1]["params"]:
            if p.dtype not in (torch.float32, torch.bfloat16):
                raise ValueError("parameters must be float32 or bfloat16")
            if not p.is_contiguous():
                raise ValueError("parameters must be contiguous")
            if self._keep_copies and p.dtype == torch.float32:
                self._copies[p] = p.detach().to(torch.bfloat16)

    def copy_of(self, p: torch.Tensor) -> torch.Tensor:
        """The bf16 copy of a parameter, as of the last step (a bf16 parameter is its own)."""
        return p.detach() if p.dtype == torch.bfloat16 else self._copies[p]

    @torch.no_grad()
    def refresh_copies(self):
        """Makes the copies anew after the parameters were written by other means than step()."""
        for p, c in self._copies.items():
            c.copy_(p)

    def _state(self, p):
        st = self.state[p]
        if "m" not in st:
            st.update(twell.alloc_adamw_state(p, self.state_bits), step=0, skipped=None)
        return st

    def _skipped(self, states):
        """The count of skipped steps that exactly the parameters of these states share: each call
        raises it once.  Parameters that have so far stepped together with others leave with a copy
        of theirs."""
        old = states[0]["skipped"]
        shared = self._skips.get(id(old))
        if shared is not None and shared[1] == len(states):
            return old
        if old is None:
            new = torch.zeros(1, dtype=torch.int32, device=states[0]["m"].device)
        else:
            new = old.clone()
        if shared is not None:
            shared[1] -= len(states)
            if shared[1] <= 0:
                del self._skips[id(old)]
        for st in states:
            st["skipped"] = new
        self._skips[id(new)] = [new, len(states)]
        return new

    def _list(self, key, params, grads, states, copies):
        """The description of these parameters with their gradients; made again when a tensor
        has moved."""
        names = ("m", "v") + (("m_scale", "v_scale") if self.state_bits == 8 else ())
        where = [p.data_ptr() for p in params] + [s[n].data_ptr() for s in states for n in names]
        where += [0 if c is None else c.data_ptr() for c in copies]
        if key not in self._lists or self._lists[key][0] != where:
            scales = {n: [s[n] for s in states] for n in names[2:]}
            made = twell.TwellParams([p.detach().view(-1) for p in params], grads,
                                     [s["m"] for s in states], [s["v"] for s in states],
                                     copies=[None if c is None else c.view(-1) for c in copies],
                                     **scales)
            self._lists[key] = (where, made)
        else:
            self._lists[key][1].set_grads(grads)
        return self._lists[key][1]

    @torch.no_grad()
    def step(self, closure=None):
        loss = None
        if closure is not None:
            with torch.enable_grad():
                loss = closure()
        # (parameter, gradient) by group
        live = [[(p, g if g.is_contiguous() else g.contiguous())
                 for p, g in [(p, p.grad) for p in group["params"]] if g is not None]
                for group in self.param_groups]
        grads = [g for pairs in live for _, g in pairs]
        if not grads:
            return loss
        factor = None
        if self.max_norm is not None:
            if len({g.dtype for g in grads}) > 1:
                raise ValueError("max_norm needs gradients of one type")
            dev = grads[0].device
            if self.last_norm is None:
                self.last_norm = torch.zeros(2, dtype=torch.float32, device=dev)
            if self._ws is None:
                self._ws = torch.empty(twell.twell_grad_norm_workspace_bytes(), dtype=torch.uint8,
                                       device=dev)
            twell.twell_grad_norm(twell.TwellGrads(grads), self.max_norm,
                                  self.last_norm, self._ws)
            factor = self.last_norm[1:]
        for i, (group, pairs) in enumerate(zip(self.param_groups, live)):
            # one list for each pair of types and each count of steps within the group
            kinds = {}
            for p, g in pairs:
                st = self._state(p)
                kinds.setdefault((p.dtype, g.dtype, st["step"], id(st["skipped"])), []).append((p, g, st))
            for j, ((dtype, _, done, _), members) in enumerate(kinds.items()):
                ps, gs, states = map(list, zip(*members))
                copied = self._keep_copies and dtype == torch.float32
                copies = [self._copies[p] for p in ps] if copied else [None] * len(ps)
                tensors = self._list((i, j), ps, gs, states, copies)
                try:
                    twell.twell_adamw_step(
                        tensors, step=done + 1, lr=float(group["lr"]), beta1=group["betas"][0],
                        beta2=group["betas"][1], eps=group["eps"], weight_decay=group["weight_decay"],
                        seed=self.seed + 64 * i + j % 64 + (j // 64 << 40), grad_scale=factor,
                        skipped=self._skipped(states))
                finally:
                    tensors.drop_grads()  # the list is kept, what zero_grad() frees is not
                for st in states:
                    st["step"] = done + 1
                # the kernels' writes, for what autograd saved before them
                torch.autograd.graph.increment_version(ps + copies if copied else ps)
        return loss

    def load_state_dict(self, state_dict):
        """Restores groups and moments.  (PyTorch would cast the moments to the parameters' types.)
        Takes dictionaries that count steps by group as well."""
        saved = state_dict["state"]
        groups = [dict(g) for g in state_dict["param_groups"]]
        by_group = [(i, k, step) for i, (g, step) in enumerate([(g, g.pop("step", 0)) for g in groups])
                    for k in g["params"]]
        super().load_state_dict({"state": {}, "param_groups": groups})
        params = [p for g in self.param_groups for p in g["params"]]
        counts = {}  # parameters with the same history share a count again
        self._skips.clear()
        for (i, k, step), p in zip(by_group, params):
            if not saved.get(k):  # no step has reached this parameter yet
                continue
            want = twell.alloc_adamw_state(p, self.state_bits)
            got = dict(saved[k])
            step, skipped = int(got.pop("step", step)), int(got.pop("skipped", 0))
            if set(got) != set(want) or any(
                    got[n].shape != t.shape or got[n].dtype != t.dtype for n, t in want.items()):
                raise ValueError("the saved moments are of another form (state_bits) or size")
            for n, t in want.items():
                t.copy_(got[n])
            key = (i, step, skipped)
            if key not in counts:
                counts[key] = torch.full((1,), skipped, dtype=torch.int32, device=p.device)
                self._skips[id(counts[key])] = [counts[key], 0]
            self._skips[id(counts[key])][1] += 1
            self.state[p] = dict(want, step=step, skipped=counts[key])
        self._lists.clear()
        self.refresh_copies()
