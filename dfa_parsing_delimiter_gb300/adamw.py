"""AdamW steps over many tensors at once (pp.h, pp_adamw).

  adamw_state         the state of a list of parameters -> AdamWState
  pp_adamw / adamw_step       one step, in place
  pp_adamw_values / AdamWState.values   what 8-bit states stand for

Marshalling only, by the rules of the lm module: everything is computed by
libpp's kernels on the given stream (default: the current one), arguments that
do not fit raise ValueError, errors of the library RuntimeError.
"""
from __future__ import annotations

import ctypes

import torch
from torch.autograd.graph import increment_version

from . import lm
from .lm import FTYPE, _call, _need, _new, _on_stream

_MOST = torch.finfo(torch.float32).max
BLOCK = 256  # elements that share an exponent; each tensor's state begins at a multiple
_vp, _u64, _i32, _f32, _f64 = ctypes.c_void_p, ctypes.c_uint64, ctypes.c_int32, ctypes.c_float, ctypes.c_double


class AdamWTensor(ctypes.Structure):
    """pp_adamw_tensor."""
    _fields_ = [("d_param", _vp), ("d_grad", _vp), ("n", _u64), ("first", _u64), ("weight_decay", _f32),
                ("param_type", _i32), ("grad_type", _i32)]


class AdamWStateStruct(ctypes.Structure):
    """pp_adamw_state."""
    _fields_ = [("d_exp_avg", _vp), ("d_exp_avg_sq", _vp), ("d_exp_avg_exponent", _vp), ("d_exp_avg_sq_exponent", _vp),
                ("d_master", _vp), ("d_counters", _vp), ("n", _u64), ("bits", _i32), ("seed", ctypes.c_uint32),
                ("nearest", _i32)]


class AdamWOpts(ctypes.Structure):
    """pp_adamw_opts."""
    _fields_ = [("lr", _f64), ("beta1", _f64), ("beta2", _f64), ("eps", _f64), ("d_lr", _vp), ("d_grad_scale", _vp),
                ("d_skip", _vp)]


def declare(L: ctypes.CDLL) -> None:
    """The entry points' argument types."""
    L.pp_adamw.restype = L.pp_adamw_values.restype = ctypes.c_int
    L.pp_adamw.argtypes = [_vp, ctypes.c_size_t, _vp, _vp, _vp]
    L.pp_adamw_values.argtypes = [_vp, ctypes.c_int, _vp, _vp, _vp]


class AdamWState:
    """The state of a list of parameters; adamw_state makes one.  Flat tensors
    over all parameters, of which `split` gives each one's part:

      exp_avg, exp_avg_sq     float32, or uint8 codes (bits 8) with
      exp_avg_exponent, exp_avg_sq_exponent   uint8, one for every 256 codes
      master                  float32 copies of the parameters, or None
      step                    int32 without dimensions: steps done
    """

    def __init__(self, shapes, device, bits: int, master: bool, seed: int, nearest: bool):
        _need(bits in (32, 8), f"bits: want 32 or 8, got {bits}")
        self.bits, self.seed, self.nearest = bits, int(seed) & 0xFFFFFFFF, bool(nearest)
        self.shapes = [torch.Size(s) for s in shapes]
        self.sizes = tuple(s.numel() for s in self.shapes)
        first, n = [], 0
        for size in self.sizes:
            first.append(n)
            n += -(-size // BLOCK) * BLOCK
        self.first, self.n = tuple(first), n
        kind = torch.float32 if bits == 32 else torch.uint8

        def zeros(size, dtype):
            return torch.zeros(size, dtype=dtype, device=device)

        self.exp_avg, self.exp_avg_sq = zeros(n, kind), zeros(n, kind)
        self.exp_avg_exponent = zeros(n // BLOCK, torch.uint8) if bits == 8 else None
        self.exp_avg_sq_exponent = zeros(n // BLOCK, torch.uint8) if bits == 8 else None
        self.master = zeros(n, torch.float32) if master else None
        self._counters = zeros(2, torch.int32)
        self.step = self._counters[0]

    def split(self, flat: torch.Tensor) -> list[torch.Tensor]:
        """Each parameter's part of a flat tensor of the state."""
        return [flat[a:a + n].view(s) for a, n, s in zip(self.first, self.sizes, self.shapes)]

    def state_dict(self) -> dict:
        """The state's tensors by name, as `load` takes them; of 8-bit states also
        how they are rounded, `seed` (int64) and `nearest` (bool), on the host."""
        names = ("exp_avg", "exp_avg_sq", "exp_avg_exponent", "exp_avg_sq_exponent", "master", "step")
        d = {k: getattr(self, k) for k in names if getattr(self, k) is not None}
        if self.bits == 8:
            d.update(seed=torch.tensor(self.seed), nearest=torch.tensor(self.nearest))
        return d

    def load(self, **tensors) -> None:
        """Copies tensors of state_dict's names into the state (None, or not given:
        that one stays).  A captured graph keeps the seed that it was captured with."""
        mine = self.state_dict()
        tensors = {k: t for k, t in tensors.items() if t is not None}
        for k, t in tensors.items():
            _need(k in mine, f"{k}: not part of this state")
            _need(t.shape == mine[k].shape and t.dtype == mine[k].dtype,
                  f"{k}: want {tuple(mine[k].shape)} of {mine[k].dtype}, got {tuple(t.shape)} of {t.dtype}")
        for k, t in tensors.items():
            if k == "seed":
                self.seed = int(t) & 0xFFFFFFFF
            elif k == "nearest":
                self.nearest = bool(t)
            else:
                mine[k].copy_(t)

    def _struct(self) -> AdamWStateStruct:
        return AdamWStateStruct(*[None if t is None else t.data_ptr() for t in (
            self.exp_avg, self.exp_avg_sq, self.exp_avg_exponent, self.exp_avg_sq_exponent, self.master,
            self._counters)], self.n, self.bits, self.seed, self.nearest)

    def values(self, dtype=torch.float32, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
        """(exp_avg, exp_avg_sq) as numbers, flat: what 8-bit codes stand for
        (exactly in float32 and bfloat16), or the 32-bit ones in `dtype` (in
        float32 the state's own tensors, which the next step changes)."""
        _need(dtype in FTYPE, "dtype: want float32, float16 or bfloat16")
        if self.bits == 32:
            with _on_stream(stream):
                return self.exp_avg.to(dtype), self.exp_avg_sq.to(dtype)
        m, v = (_new((self.n,), dtype, self._counters, stream) for _ in range(2))
        L = lm.pp.lib()
        _call(L.pp_adamw_values, "pp_adamw_values", self._counters, stream, ctypes.byref(self._struct()), FTYPE[dtype],
              m.data_ptr(), v.data_ptr())
        return m, v


def adamw_state(params, bits: int = 32, master: bool = False, seed: int = 0, nearest: bool = False) -> AdamWState:
    """The state of the first step for these parameters (float32, float16 or
    bfloat16, contiguous, on one device).  bits: 32, or 8 for a byte a value
    and a shared exponent, rounded by random bits from `seed` or, with
    `nearest`, to nearest.  master: keep 32-bit copies of the parameters, so
    that steps smaller than a 16-bit parameter's rounding add up.  The state is
    made on the current stream: steps on another one wait for that first."""
    params = list(params)
    _need(len(params) > 0, "params: want a tensor at least")
    device, spans = params[0].device, []
    for i, p in enumerate(params):
        _need(p.dtype in FTYPE and p.device == device and p.is_contiguous() and p.is_leaf,
              f"params: want contiguous leaves of float32, float16 or bfloat16 on one device (tensor {i})")
        if p.numel():
            spans.append((p.data_ptr(), p.data_ptr() + p.numel() * p.element_size()))
    spans.sort()
    _need(all(a[1] <= b[0] for a, b in zip(spans, spans[1:])), "params: tensors that overlap")
    s = AdamWState([p.shape for p in params], device, bits, master, seed, nearest)
    if master:
        with torch.no_grad():
            for part, p in zip(s.split(s.master), params):
                part.copy_(p)
    return s


def _number(t, like: torch.Tensor, name: str) -> int:
    """Address of a float32 tensor of one element, 0 for None."""
    if t is None:
        return 0
    _need(t.dtype is torch.float32 and t.numel() == 1 and t.get_device() == like.get_device(),
          f"{name}: want one float32 on the state's device")
    return t.data_ptr()


def adamw_step(params, grads, state: AdamWState, lr=1e-3, betas=(0.9, 0.999), eps: float = 1e-8, weight_decay=1e-2,
               grad_scale=None, skip=None, stream=None) -> None:
    """pp_adamw: one step of the parameters that `state` was made for, in
    place.  grads: a tensor or None (that parameter and its state stay) for
    each, or None for the parameters' own .grad.  weight_decay: a number, or
    one for each.  lr may be, and grad_scale (which the gradients are
    multiplied by) and skip (not 0: nothing changes) are, one float32 on the
    device, which a captured graph reads anew each time."""
    if not isinstance(params, (list, tuple)):
        params = list(params)
    if grads is None:
        grads = [p.grad for p in params]
    elif not isinstance(grads, (list, tuple)):
        grads = list(grads)
    like = state._counters
    lr_at = 0
    if isinstance(lr, torch.Tensor):
        lr, lr_at = 0.0, _number(lr, like, "lr")
    else:
        _need(0.0 <= lr <= _MOST, f"lr: want a number from 0 on that 32 bits hold, got {lr}")
    _need(0.0 <= betas[0] < 1.0 and 0.0 <= betas[1] < 1.0, f"betas: want numbers from 0 to below 1, got {betas}")
    _need(0.0 <= eps <= _MOST, f"eps: want a number from 0 on that 32 bits hold, got {eps}")
    c = lm._lib()
    scale_at, skip_at = _number(grad_scale, like, "grad_scale"), _number(skip, like, "skip")
    _call(c.adamw, "pp_adamw", like, stream, params, grads, state.sizes, state.first, weight_decay, like.get_device(),
          state.exp_avg.data_ptr(), state.exp_avg_sq.data_ptr(),
          0 if state.bits == 32 else state.exp_avg_exponent.data_ptr(),
          0 if state.bits == 32 else state.exp_avg_sq_exponent.data_ptr(),
          0 if state.master is None else state.master.data_ptr(), like.data_ptr(), state.n, state.bits, state.seed,
          state.nearest, lr, betas[0], betas[1], eps, lr_at, scale_at, skip_at)
    changed = [p for p, g in zip(params, grads) if g is not None]
    try:
        increment_version(changed)
    except RuntimeError:  # there are inference tensors, which have no version
        increment_version([p for p in changed if not p.is_inference()])
