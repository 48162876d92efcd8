"""torch.optim front end: one optimizer over Muon and aux AdamW param groups.

The interface follows the README of the Muon repository ("Muon: An
optimizer for the hidden layers of neural networks", section "Usage"): a
list of param groups, each with ``use_muon``; Muon groups take ``lr``,
``weight_decay`` (and ``momentum``, ``nesterov``, ``ns_steps``), AdamW groups
take ``lr``, ``betas``, ``eps``, ``weight_decay``.  Which parameters are
"hidden" is the caller's choice, as the README says.

AdamW groups take three keys more: ``state_bits`` (32, or 8 for moments in
8 bits), ``max_grad_norm`` (clip the 2-norm over the group's gradients; a step
whose norm is not finite changes nothing) and ``seed`` (round 8-bit codes and
bf16 parameters stochastically; None, the default, rounds to nearest).

A group with 8-bit moments and a beta2 near 1 needs a seed.  Rounding to
nearest loses a change smaller than half a code: with beta2 = 0.999 a second
moment can grow but hardly shrink, and where a block's gradients are of one
magnitude it drifts upward (1.2 times the right value after 4000 steps, 1.8
after 16000), which shortens the steps.

This file only keeps optimizer state tensors and hands pointers to the
library: every update runs in libmuon_b200.so.
"""

from __future__ import annotations

from itertools import chain
from operator import index
from typing import Iterable

import torch

from .binding import MuonContext, default_adamw_hparams, default_adamw_plan_hparams, default_hparams
from .plans import state8_zeros

MUON_DEFAULTS = dict(lr=0.02, weight_decay=0.01, momentum=0.95, nesterov=True, ns_steps=5,
                     scale_mode="original")
ADAMW_DEFAULTS = dict(lr=3e-4, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.01, state_bits=32,
                      max_grad_norm=None, seed=None)

# A plan that this many steps have not used is dropped: parameters whose gradients come and go ask for other plans,
# and each holds its tensors.
PLAN_STEPS = 16


def _check_adamw_group(g):
    """Refuse values of the keys beyond AdamW's own that no step can take."""
    if g.get("state_bits", 32) not in (8, 32):
        raise ValueError("state_bits must be 8 or 32")
    clip, seed = g.get("max_grad_norm"), g.get("seed")
    try:
        if clip is not None and not clip >= 0:
            raise ValueError("max_grad_norm must be >= 0")
        if seed is not None and not 0 <= index(seed) < 1 << 32:
            raise ValueError("seed must lie in [0, 2^32)")
    except TypeError:
        raise ValueError("max_grad_norm must be a number and seed an integer") from None


def _own_types(value, p):
    """A saved value of the state of p on its device, tensors copied: codes as
    they are, others in fp32."""
    if isinstance(value, torch.Tensor):
        dtype = torch.float32 if value.is_floating_point() else value.dtype
        return value.detach().to(device=p.device, dtype=dtype, copy=True).contiguous()
    if isinstance(value, dict):
        return {k: _own_types(v, p) for k, v in value.items()}
    return type(value)(_own_types(v, p) for v in value) if isinstance(value, (list, tuple)) else value


class MuonWithAuxAdam(torch.optim.Optimizer):
    """Muon for groups with use_muon=True (parameters of two or more
    dimensions, stepped as rows x prod(other dims) matrices), AdamW for the
    rest.  Parameters must be contiguous CUDA tensors on one device, fp32, or
    bf16 in AdamW groups; gradients fp32 or bf16.

    A group's state_bits may be changed between steps, after loading a
    checkpoint for instance: its moments are converted at the next step, which
    synchronises the device; when that fails the old ones stay.  A step skipped
    for a norm that is not finite still counts; one that raises does not, for
    groups that use any of the three keys or bf16 parameters.

    Device-side failures (a bounded wait inside a kernel that gave up) are
    flagged on the GPU; from then on the library leaves every parameter and
    state tensor untouched until the flag is read.  step() reads it every
    `check_every` steps (0: never; each read synchronises the device) and
    raises MuonError when it is set; check() reads it on demand."""

    def __init__(self, param_groups: Iterable[dict], device: int = None, check_every: int = 100):
        groups = []
        for g in param_groups:
            g = dict(g)
            if "use_muon" not in g:
                raise ValueError("every param group needs use_muon")
            base = MUON_DEFAULTS if g["use_muon"] else ADAMW_DEFAULTS
            for k, v in base.items():
                g.setdefault(k, v)
            if not g["use_muon"]:
                _check_adamw_group(g)
            groups.append(g)
        super().__init__(groups, dict())
        for g in self.param_groups:
            for p in g["params"]:
                if not p.is_cuda or not p.is_contiguous() or not (
                        p.dtype == torch.float32 or p.dtype == torch.bfloat16 and not g["use_muon"]):
                    raise ValueError("parameters must be contiguous fp32 CUDA tensors (bf16 too in AdamW groups)")
                if g["use_muon"] and p.dim() < 2:
                    raise ValueError("Muon parameters need two or more dimensions")
        first = next(p for g in self.param_groups for p in g["params"])
        self.ctx = MuonContext(first.device.index if device is None else device)
        self.check_every = int(check_every)
        self._steps = 0
        self._plans = {}       # what the AdamW groups' plans were built over, the plans, and the step that last used each

    def check(self):
        """Synchronise and raise MuonError if a device-side wait gave up since
        the last check (the library then skipped every update)."""
        self.ctx.check_device()

    @torch.no_grad()
    def step(self, closure=None):
        loss = None
        if closure is not None:
            with torch.enable_grad():
                loss = closure()
        for g in self.param_groups:        # all of them, before any is stepped
            if not g.get("use_muon", True):
                _check_adamw_group(g)
        for i, g in enumerate(self.param_groups):
            params = [p for p in g["params"] if p.grad is not None]
            if not params:
                continue
            if g["use_muon"]:
                self._muon(g, params)
            elif (g.get("state_bits", 32) == 8 or g.get("max_grad_norm") is not None or g.get("seed") is not None
                  or any(p.dtype != torch.float32 or "exp_avg_scale" in self.state[p] for p in params)):
                self._adamw_planned(i, g, params)
            else:
                self._adamw(g, params)
        stale = [key for key, plan in self._plans.items() if plan[3] < self._steps - PLAN_STEPS]
        for key in stale:
            del self._plans[key]
        self._steps += 1
        if self.check_every and self._steps % self.check_every == 0:
            self.check()
        return loss

    def _muon(self, g, params):
        hp = default_hparams(lr=g["lr"], weight_decay=g["weight_decay"], momentum=g["momentum"],
                             nesterov=g["nesterov"], ns_steps=g["ns_steps"], scale_mode=g["scale_mode"])
        by_shape = {}
        for p in params:
            st = self.state[p]
            if "momentum_buffer" not in st:
                st["momentum_buffer"] = torch.zeros_like(p)
            w = p.view(p.shape[0], -1)
            grad = p.grad.reshape(p.shape[0], -1).contiguous()
            buf = st["momentum_buffer"].view(p.shape[0], -1)
            key = (tuple(w.shape), grad.dtype)
            e = by_shape.setdefault(key, dict(weights=[], grads=[], momentum=[]))
            e["weights"].append(w)
            e["grads"].append(grad)
            e["momentum"].append(buf)
        self.ctx.step(list(by_shape.values()), hp)

    def _adamw(self, g, params):
        b1, b2 = g["betas"]
        hp = default_adamw_hparams(lr=g["lr"], beta1=b1, beta2=b2, eps=g["eps"], weight_decay=g["weight_decay"])
        by_step = {}
        for p in params:
            st = self.state[p]
            if "step" not in st:
                st["step"] = 0
                st["exp_avg"] = torch.zeros_like(p)
                st["exp_avg_sq"] = torch.zeros_like(p)
            st["step"] += 1
            by_step.setdefault(st["step"], []).append(p)
        for step, ps in by_step.items():
            self.ctx.adamw_step([p.view(-1) for p in ps], [p.grad.reshape(-1).contiguous() for p in ps],
                                [self.state[p]["exp_avg"].view(-1) for p in ps],
                                [self.state[p]["exp_avg_sq"].view(-1) for p in ps], step, hp)

    # -- AdamW through plans ------------------------------------------------
    def _moments(self, params, bits):
        """Zero moments where there are none; those of the other form are
        converted, and replaced when that is known to have happened."""
        convert = []
        for p in params:
            st = self.state[p]
            if "step" not in st:
                st.update(state8_zeros(p) if bits == 8 else dict(
                    exp_avg=torch.zeros_like(p, dtype=torch.float32),
                    exp_avg_sq=torch.zeros_like(p, dtype=torch.float32)), step=0)
            elif ("exp_avg_scale" in st) != (bits == 8):
                convert.append(p)
        if not convert:
            return
        wide, codes, scales, converted = [], [], [], []
        for p in convert:
            st = self.state[p]
            full = {k: st[k] if bits == 8 else torch.empty_like(p, dtype=torch.float32) for k in ("exp_avg", "exp_avg_sq")}
            small = state8_zeros(p) if bits == 8 else {k: st[k] for k in ("exp_avg", "exp_avg_sq", "exp_avg_scale",
                                                                         "exp_avg_sq_scale")}
            for k in ("exp_avg", "exp_avg_sq"):
                wide.append(full[k].contiguous())
                codes.append(small[k])
                scales.append(small[k + "_scale"])
            converted.append(small if bits == 8 else full)
        plan = self.ctx.state8_plan(wide, codes, scales)
        plan.pack() if bits == 8 else plan.unpack()
        plan.close()
        # after a device-side failure the kernels have written nothing
        self.ctx.check_device()
        for p, new in zip(convert, converted):
            st = self.state[p]
            st.pop("exp_avg_scale", None)
            st.pop("exp_avg_sq_scale", None)
            st.update(new)
        # plans over the old moments would keep them allocated
        gone = set(map(id, convert))
        self._plans = {key: plan for key, plan in self._plans.items() if key[1] == "norm" or gone.isdisjoint(key[2])}

    def _plan(self, key, tensors, grads, build):
        """The plan of `key`, rebuilt when its tensors or the gradients' types
        changed, with these gradients."""
        at = [t.data_ptr() for t in tensors] + [(g.dtype, g.numel()) for g in grads]
        ptrs = [g.data_ptr() for g in grads]
        had = self._plans.get(key)
        if had is None or had[0] != at:
            had = self._plans[key] = [at, ptrs, build(), 0]
        elif had[1] != ptrs:
            had[2].bind_grads(grads)
            had[1] = ptrs
        had[3] = self._steps
        had[2].forget_grads()      # a gradient freed by zero_grad is not kept to the next step
        return had[2]

    def _adamw_planned(self, group, g, params):
        bits, clip, seed = int(g.get("state_bits", 32)), g.get("max_grad_norm"), g.get("seed")
        seed = None if seed is None else index(seed)
        self._moments(params, bits)
        b1, b2 = g["betas"]
        hp = default_adamw_plan_hparams(lr=g["lr"], beta1=b1, beta2=b2, eps=g["eps"], weight_decay=g["weight_decay"])
        grads = {p: p.grad.reshape(-1).contiguous() for p in params}
        factor = None
        if clip is not None:
            gs = list(grads.values())
            norm = self._plan((group, "norm", tuple(map(id, params))), [], gs, lambda: self.ctx.grad_norm_plan(gs))
            factor = norm.run(float(clip))[1:]
        by_step = {}
        for p in params:
            by_step.setdefault(self.state[p]["step"] + 1, []).append(p)
        names = ["exp_avg", "exp_avg_sq"] + (["exp_avg_scale", "exp_avg_sq_scale"] if bits == 8 else [])
        for step, ps in by_step.items():
            lists = [[p.detach().view(-1) for p in ps]] + [[self.state[p][k].view(-1) for p in ps] for k in names]
            gs = [grads[p] for p in ps]
            plan = self._plan((group, bits, tuple(map(id, ps))), list(chain(*lists)), gs,
                              lambda: self.ctx.adamw_plan(lists[0], gs, *lists[1:]))
            plan.step(step, hp, grad_scale=factor, seed=seed)
            for p in ps:
                self.state[p]["step"] = step

    def load_state_dict(self, state_dict):
        """As torch.optim.Optimizer's, except that 8-bit codes stay what they
        are and every other state tensor becomes fp32 (the base class casts
        state to the parameter's type, which would round the moments and
        scales of bf16 parameters and turn codes into numbers).  Pre-hooks
        come before this and post-hooks after it."""
        fresh = {}

        def last_pre_hook(opt, sd):
            saved = chain.from_iterable(g["params"] for g in sd["param_groups"])
            own = dict(zip(saved, chain.from_iterable(g["params"] for g in self.param_groups)))
            fresh.update((own[k], _own_types(st, own[k])) for k, st in sd["state"].items() if k in own)
            for st in fresh.values():
                if "step" in st:
                    st["step"] = int(st["step"])
            # no tensor is left for the base class, whose cast would hold every 8-bit moment in 32 bits at once
            return dict(sd, state={k: st for k, st in sd["state"].items() if k not in own})

        def first_post_hook(opt):
            self.state.update(fresh)
            self._plans.clear()

        hooks = [self.register_load_state_dict_pre_hook(last_pre_hook),
                 self.register_load_state_dict_post_hook(first_post_hook, prepend=True)]
        try:
            super().load_state_dict(state_dict)
        finally:
            for h in hooks:
                h.remove()
