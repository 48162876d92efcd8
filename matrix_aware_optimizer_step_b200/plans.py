"""Plans: lists of tensors laid out once for calls that repeat every step.

`MuonContext.adamw_plan`, `grad_norm_plan` and `state8_plan` build them.  A
plan holds references to its tensors and uses their memory in place, so they
must not be resized or moved to other storage while it lives; gradients can
be replaced with `bind_grads`.  Calls only launch kernels: they allocate
nothing, copy nothing and can be captured into a CUDA graph.  Arithmetic
happens in the library; this file checks arguments and passes pointers.

8-bit moments keep one int8 (first moment) or uint8 (second moment) code per
element and one fp32 scale per 256 consecutive elements; `state8_zeros` makes
zero moments of that form.
"""

from __future__ import annotations

import ctypes
import struct
from typing import Optional, Sequence

import torch

from .binding import (MUON_BF16, MUON_F32, MUON_OK, AdamwPlanHparams, GradTensor, MuonError, PlanTensor, State8Tensor,
                      default_adamw_plan_hparams, load_library)

STATE8_BLOCK = 256


def state8_scales(numel: int) -> int:
    """How many scales the 8-bit form of numel elements has."""
    return (int(numel) + STATE8_BLOCK - 1) // STATE8_BLOCK


def state8_zeros(like) -> dict:
    """Zero 8-bit moments for the parameter `like`: exp_avg (int8) and
    exp_avg_sq (uint8) of its shape, exp_avg_scale and exp_avg_sq_scale."""
    n = state8_scales(like.numel())
    return dict(exp_avg=torch.zeros(like.shape, dtype=torch.int8, device=like.device),
                exp_avg_sq=torch.zeros(like.shape, dtype=torch.uint8, device=like.device),
                exp_avg_scale=torch.zeros(n, dtype=torch.float32, device=like.device),
                exp_avg_sq_scale=torch.zeros(n, dtype=torch.float32, device=like.device))


def _check(t, what: str, device: int, numel: Optional[int] = None, dtypes=None):
    if t.get_device() != device or not t.is_contiguous():
        raise ValueError(f"{what}: tensors must be contiguous CUDA tensors on device {device}")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{what}: {t.numel()} elements where {numel} are wanted")
    if dtypes is not None and t.dtype not in dtypes:
        raise TypeError(f"{what}: unsupported dtype {t.dtype}")


# the structs of the header, packed a list at a time (a ctypes field costs as
# much as packing a struct)
_PLAN_TENSOR, _GRAD_TENSOR, _STATE8_TENSOR = struct.Struct("@qii7Q"), struct.Struct("@qiiQ"), struct.Struct("@qii3Q")
assert (_PLAN_TENSOR.size, _GRAD_TENSOR.size, _STATE8_TENSOR.size) == tuple(
    map(ctypes.sizeof, (PlanTensor, GradTensor, State8Tensor)))
_CODE = {torch.float32: MUON_F32, torch.bfloat16: MUON_BF16}


def _array(cls, packed):
    """A ctypes array of `cls` from its packed elements."""
    return (cls * max(1, len(packed))).from_buffer_copy(b"".join(packed) or bytes(ctypes.sizeof(cls)))


def _scalar_ptr(t, what: str, device: int, dtype) -> int:
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.numel() < 1:
        raise TypeError(f"{what}: a {dtype} tensor of one element is wanted")
    if not t.is_cuda or t.device.index != device:
        raise ValueError(f"{what}: must be on CUDA device {device}")
    return t.data_ptr()


_FLOATS = (torch.float32, torch.bfloat16)


def _current_stream(device: int) -> int:
    return torch.cuda.current_stream(device).cuda_stream


# the same pointer without building a Stream object: a third of a small call's host time
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _current_stream)


class _Plan:
    """A library plan, the context it belongs to and the tensors it uses."""

    def __init__(self, ctx, keep):
        if not ctx._ctx:
            raise ValueError("the context is closed")
        self._ctx = ctx
        self._lib = load_library()
        self._h = ctypes.c_void_p()
        self.device = int(ctx.device)
        self._keep = keep

    def _create(self, fn, arr, n, *more):
        st = fn(self._ctx._ctx, arr, n, *more, ctypes.byref(self._h))
        if st != MUON_OK:
            self._h = ctypes.c_void_p()
        self._ctx._check(st, fn.__name__)

    def _failed(self, st, what):
        if not self._h:
            raise MuonError(st, f"{what}: the plan is closed")
        if not self._ctx._ctx:
            raise MuonError(st, f"{what}: the context is closed")
        self._ctx._check(st, what)

    def _stream(self, stream) -> int:
        if stream is None:
            return _current_stream(self.device)
        return stream if isinstance(stream, int) else stream.cuda_stream

    def close(self):
        """Free the plan (synchronises the device).  Graphs that captured its
        calls must not be replayed afterwards."""
        if self._h:
            self._lib.muon_plan_destroy(self._h)
            self._h = ctypes.c_void_p()
        self._keep = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class _GradPlan(_Plan):
    def __init__(self, ctx, grads, keep):
        super().__init__(ctx, keep)
        self._grads = list(grads)
        self._like = [(g.numel(), g.dtype) for g in self._grads]

    def bind_grads(self, grads: Sequence):
        """Use these gradients from the next call on: the same number, sizes
        and types, in the same order.  Captured graphs keep the old ones."""
        grads = list(grads)
        if len(grads) != len(self._like):
            raise ValueError(f"bind_grads: {len(grads)} gradients for a plan of {len(self._like)}")
        for g, (n, dt) in zip(grads, self._like):
            _check(g, "bind_grads", self.device, n, (dt,))
        arr = (ctypes.c_void_p * max(1, len(grads)))(*[g.data_ptr() for g in grads])
        st = self._lib.muon_plan_bind_grads(self._h, arr, len(grads))
        if st != MUON_OK:
            self._failed(st, "muon_plan_bind_grads")
        self._grads = grads

    def forget_grads(self):
        """Stop holding references to the bound gradients.  The plan goes on
        using their addresses: the caller keeps them alive for each call, or
        binds others first."""
        self._grads = None


class AdamwPlan(_GradPlan):
    """AdamW over a list of tensors; built by MuonContext.adamw_plan."""

    def __init__(self, ctx, params, grads, exp_avgs, exp_avg_sqs, exp_avg_scales=None, exp_avg_sq_scales=None,
                 param_copies=None):
        params, grads, ms, vs = list(params), list(grads), list(exp_avgs), list(exp_avg_sqs)
        n = len(params)
        s8 = exp_avg_scales is not None or exp_avg_sq_scales is not None
        if s8 and (exp_avg_scales is None or exp_avg_sq_scales is None):
            raise ValueError("adamw_plan: 8-bit moments need both lists of scales")
        mss = list(exp_avg_scales) if s8 else [None] * n
        vss = list(exp_avg_sq_scales) if s8 else [None] * n
        copies = list(param_copies) if param_copies is not None else [None] * n
        if any(len(x) != n for x in (grads, ms, vs, mss, vss, copies)):
            raise ValueError("adamw_plan: the lists differ in length")
        super().__init__(ctx, grads, (params, ms, vs, mss, vss, copies))
        self.state_bits = 8 if s8 else 32
        packed, device = [], self.device
        mtype, vtype = ((torch.int8,), (torch.uint8,)) if s8 else ((torch.float32,), (torch.float32,))
        for p, g, m, v, ms_, vs_, c in zip(params, grads, ms, vs, mss, vss, copies):
            k = p.numel()
            _check(p, "adamw_plan params", device, None, _FLOATS)
            _check(g, "adamw_plan grads", device, k, _FLOATS)
            _check(m, "adamw_plan exp_avgs", device, k, mtype)
            _check(v, "adamw_plan exp_avg_sqs", device, k, vtype)
            if s8:
                _check(ms_, "adamw_plan scales", device, state8_scales(k), (torch.float32,))
                _check(vs_, "adamw_plan scales", device, state8_scales(k), (torch.float32,))
            if c is not None:
                _check(c, "adamw_plan param_copies", device, k, (torch.bfloat16,))
                if p.dtype != torch.float32:
                    raise TypeError("adamw_plan: a bf16 copy goes with an fp32 parameter")
            packed.append(_PLAN_TENSOR.pack(k, _CODE[p.dtype], _CODE[g.dtype], p.data_ptr(), g.data_ptr(), m.data_ptr(),
                                            v.data_ptr(), ms_.data_ptr() if s8 else 0, vs_.data_ptr() if s8 else 0,
                                            0 if c is None else c.data_ptr()))
        self._default = default_adamw_plan_hparams()
        self._step = self._lib.muon_adamw_plan_step
        self._create(self._lib.muon_adamw_plan_create, _array(PlanTensor, packed), n, self.state_bits)

    def step(self, step, hp: Optional[AdamwPlanHparams] = None, lr=None, grad_scale=None, seed: Optional[int] = None,
             stream=None):
        """One step.  `step` counts from 1: an int, or an int64 CUDA tensor
        that the kernels read (for captured graphs; below 1 nothing is
        written).  `lr`: an fp32 CUDA tensor instead of hp.lr.  `grad_scale`:
        an fp32 CUDA tensor that multiplies every gradient, such as [1:] of a
        norm plan's result; when it is not finite nothing is written.  `seed`:
        None rounds 8-bit codes and bf16 parameters to nearest, an int in
        [0, 2^32) stochastically, by numbers hashed from it, the step, the
        tensor's place in the list and the element."""
        step_ptr = lr_ptr = scale_ptr = None
        if isinstance(step, torch.Tensor):
            step_ptr = _scalar_ptr(step, "step", self.device, torch.int64)
            step = 0
        if lr is not None:
            lr_ptr = _scalar_ptr(lr, "lr", self.device, torch.float32)
        if grad_scale is not None:
            scale_ptr = _scalar_ptr(grad_scale, "grad_scale", self.device, torch.float32)
        if seed is not None and not 0 <= seed < 1 << 32:
            raise ValueError("seed must lie in [0, 2^32)")
        st = self._step(self._h, self._default if hp is None else hp, int(step), step_ptr, lr_ptr, scale_ptr,
                        seed is not None, seed or 0,
                        _current_stream(self.device) if stream is None else self._stream(stream))
        if st != MUON_OK:
            self._failed(st, "muon_adamw_plan_step")


class GradNormPlan(_GradPlan):
    """The 2-norm over a list of gradients and the factor that clips it;
    built by MuonContext.grad_norm_plan."""

    def __init__(self, ctx, grads):
        grads = list(grads)
        super().__init__(ctx, grads, None)
        packed = []
        for g in grads:
            _check(g, "grad_norm_plan", self.device, None, _FLOATS)
            packed.append(_GRAD_TENSOR.pack(g.numel(), _CODE[g.dtype], 0, g.data_ptr()))
        self._create(self._lib.muon_grad_norm_plan_create, _array(GradTensor, packed), len(grads))
        n = ctypes.c_size_t()
        self._lib.muon_grad_norm_out_bytes(self._h, ctypes.byref(n))
        self._floats = n.value // 4
        self._result = self.new_output()[:2]
        self._result_ptr = self._result.data_ptr()
        torch.cuda.current_stream(self.device).synchronize()      # zeroed, whichever stream runs first
        self._run = self._lib.muon_grad_norm_run

    def new_output(self):
        """A result buffer, zeroed on the current stream: its first two
        elements are the result, the rest is the call's workspace.  Runs that may overlap in time (other streams,
        captured graphs that replay side by side) need one each."""
        return torch.zeros(self._floats, dtype=torch.float32, device=torch.device("cuda", self.device))

    def run(self, max_norm: float = float("inf"), out=None, stream=None):
        """fp32 [norm, min(1, max_norm / (norm + 1e-6))]; the factor is NaN
        when the norm is not finite.  `out`: a buffer of new_output(), the
        plan's own by default, which the next run overwrites."""
        if out is None:
            result, ptr = self._result, self._result_ptr
        else:
            _check(out, "out", self.device, self._floats, (torch.float32,))
            result, ptr = out[:2], out.data_ptr()
        st = self._run(self._h, float(max_norm), ptr, _current_stream(self.device) if stream is None else self._stream(stream))
        if st != MUON_OK:
            self._failed(st, "muon_grad_norm_run")
        return result


class State8Plan(_Plan):
    """Conversion between moments and their 8-bit form; built by
    MuonContext.state8_plan."""

    def __init__(self, ctx, values, codes, scales):
        values, codes, scales = list(values), list(codes), list(scales)
        n = len(values)
        if len(codes) != n or len(scales) != n:
            raise ValueError("state8_plan: the lists differ in length")
        super().__init__(ctx, (values, codes, scales))
        packed = []
        for x, c, s in zip(values, codes, scales):
            k = x.numel()
            _check(x, "state8_plan values", self.device, None, _FLOATS)
            _check(c, "state8_plan codes", self.device, k, (torch.int8, torch.uint8))
            _check(s, "state8_plan scales", self.device, state8_scales(k), (torch.float32,))
            packed.append(_STATE8_TENSOR.pack(k, _CODE[x.dtype], c.dtype == torch.uint8, x.data_ptr(), c.data_ptr(),
                                              s.data_ptr()))
        self._create(self._lib.muon_state8_plan_create, _array(State8Tensor, packed), n)

    def pack(self, stream=None):
        """Values to codes and scales, rounded to nearest."""
        st = self._lib.muon_state8_pack(self._h, self._stream(stream))
        if st != MUON_OK:
            self._failed(st, "muon_state8_pack")

    def unpack(self, stream=None):
        """Codes and scales to the values they stand for."""
        st = self._lib.muon_state8_unpack(self._h, self._stream(stream))
        if st != MUON_OK:
            self._failed(st, "muon_state8_unpack")
