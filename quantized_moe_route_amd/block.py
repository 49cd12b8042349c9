"""The dense operators of an MoE block and its optimizer step (include/moe_block.h): binding.

GatedFFN, BlockNorm and AdamW allocate outputs and workspaces with PyTorch, check what they are
given (device, type, shape, contiguity) and pass addresses and the current stream of their own
device to the HIP kernels.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass
from typing import Optional, Sequence

from . import _lib as C

ACTS = {"swiglu": C.MOE_ACT_SWIGLU, "situ": C.MOE_ACT_SITU}
GATES = {"none": C.MOE_GATE_NONE, "channel": C.MOE_GATE_CHANNEL, "token": C.MOE_GATE_TOKEN, "full": C.MOE_GATE_FULL}


def _torch():
    import torch
    return torch


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _dtype_code(dtype, what: str) -> int:
    torch = _torch()
    if dtype == torch.bfloat16:
        return C.MOE_DT_BF16
    if dtype == torch.float32:
        return C.MOE_DT_F32
    raise TypeError(f"{what}: unsupported dtype {dtype} (bf16 or fp32)")


class _Handle:
    """A C handle with its workspace on one device."""

    _destroy: str = ""
    _h = None

    def _create(self, device, desc, size_fn: str, create):
        torch = _torch()
        L = C.lib()
        self.device, self.desc = device, desc
        self._index = device.index
        n = ctypes.c_size_t()
        C.check(getattr(L, size_fn)(ctypes.byref(desc), ctypes.byref(n)), size_fn)
        self.workspace_bytes = n.value
        with torch.cuda.device(device):
            self.workspace = torch.empty(max(256, n.value), dtype=torch.uint8, device=device)
            self._home = torch.cuda.current_stream(device).cuda_stream
            h = ctypes.c_void_p()
            create(L, self.workspace.data_ptr(), self.workspace.numel(), ctypes.byref(h))
        self._h = h

    def _call(self, fn: str, *args):
        """fn(handle, *args, stream) on the handle's device and its current stream."""
        torch = _torch()
        if self._h is None:
            raise RuntimeError(f"{fn}: the handle is closed")
        if torch.cuda.current_device() != self._index:
            with torch.cuda.device(self._index):
                return self._call(fn, *args)
        stream = torch._C._cuda_getCurrentRawStream(self._index)
        if stream != self._home and not torch.cuda.is_current_stream_capturing():
            # not reused for others while this stream works in it
            self.workspace.record_stream(torch.cuda.current_stream(self._index))
        status = getattr(C.lib(), fn)(self._h, *args, stream)
        if status:
            C.check(status, fn)

    def _take(self, t, what: str, shape, *dtypes):
        """Checks one tensor argument and returns it."""
        if t.shape == shape and t.dtype in dtypes and t.device == self.device and t.is_contiguous():
            return t
        if t.device != self.device:
            raise ValueError(f"{what} is on {t.device}, the operator on {self.device}")
        if t.shape != shape:
            raise ValueError(f"{what} has shape {tuple(t.shape)}, not {tuple(shape)}")
        if t.dtype not in dtypes:
            raise TypeError(f"{what} has dtype {t.dtype}, not {' or '.join(str(d) for d in dtypes)}")
        raise ValueError(f"{what} is not contiguous")

    def _new(self, shape, dtype):
        return _torch().empty(shape, dtype=dtype, device=self.device)

    def close(self):
        if self._h:
            getattr(C.lib(), self._destroy)(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class GatedFFN(_Handle):
    """y = act(x Wg^T, x Wu^T) Wd^T over borrowed bf16 weights Wg, Wu [I][D] and Wd [D][I].

    act: ACTS["swiglu"] or ACTS["situ"].  backward=False leaves the gradients' workspace out.
    """

    _destroy = "moe_ffn_destroy"

    def __init__(self, w_gate, w_up, w_down, *, max_tokens: int, act: int = C.MOE_ACT_SWIGLU, backward: bool = True):
        bf16 = _torch().bfloat16
        self.I, self.D = (int(n) for n in w_gate.shape)
        self.device = w_gate.device
        self._take(w_gate, "w_gate", (self.I, self.D), bf16)
        self._take(w_up, "w_up", (self.I, self.D), bf16)
        self._take(w_down, "w_down", (self.D, self.I), bf16)
        self._keep = (w_gate, w_up, w_down)
        d = C.MoeFfnDesc()
        C.lib().moe_ffn_desc_init(ctypes.byref(d))
        d.width, d.inter, d.max_tokens, d.act = self.D, self.I, max_tokens, act
        d.flags = C.MOE_FFN_BACKWARD if backward else 0
        self._create(w_gate.device, d, "moe_ffn_workspace_size", lambda L, ws, n, out: C.check(
            L.moe_ffn_create(ctypes.byref(d), *(w.data_ptr() for w in self._keep), ws, n, out), "moe_ffn_create"))

    def new_saved_gu(self, T: int):
        return self._new((T, 2, self.I), _torch().float32)

    def forward(self, x, y=None, *, out_dtype=None, accumulate: bool = False, saved_gu=None):
        """y [T][D] (bf16 by default, or fp32); accumulate=True adds onto the y given."""
        torch = _torch()
        T = int(x.shape[0])
        self._take(x, "x", (T, self.D), torch.bfloat16)
        if y is None:
            if accumulate:
                raise ValueError("accumulate needs y")
            y = self._new((T, self.D), out_dtype or torch.bfloat16)
        self._take(y, "y", (T, self.D), *([out_dtype] if out_dtype else [torch.bfloat16, torch.float32]))
        if saved_gu is not None:
            self._take(saved_gu, "saved_gu", (T, 2, self.I), torch.float32)
        self._call("moe_ffn_forward", x.data_ptr(), T, y.data_ptr(), _dtype_code(y.dtype, "y"), int(accumulate), _ptr(saved_gu))
        return y

    def backward(self, x, dy, *, saved_gu=None, dx=None, dw=None, dx_dtype=None, dw_dtype=None, accumulate: bool = False,
                 need_dx: bool = True, need_dw: bool = True):
        """(dx, (dw_gate, dw_up, dw_down)); None in the place of what is not needed.  dx and dw may be
        given; accumulate=True adds onto the dx given."""
        torch = _torch()
        T = int(x.shape[0])
        self._take(x, "x", (T, self.D), torch.bfloat16)
        self._take(dy, "dy", (T, self.D), torch.bfloat16)
        if saved_gu is not None:
            self._take(saved_gu, "saved_gu", (T, 2, self.I), torch.float32)
        if dx is None and need_dx:
            if accumulate:
                raise ValueError("accumulate needs dx")
            dx = self._new((T, self.D), dx_dtype or torch.bfloat16)
        if dw is None:
            shapes = ((self.I, self.D), (self.I, self.D), (self.D, self.I))
            dw = tuple(self._new(s, dw_dtype or torch.bfloat16) if need_dw else None for s in shapes)
        dw = tuple(dw)
        kinds = {t.dtype for t in dw if t is not None}
        if len(kinds) > 1:
            raise TypeError("the weight gradients have one dtype")
        if dx is not None:
            self._take(dx, "dx", (T, self.D), *([dx_dtype] if dx_dtype else [torch.bfloat16, torch.float32]))
        for t, w, name in zip(dw, self._keep, ("dw_gate", "dw_up", "dw_down")):
            if t is not None:
                self._take(t, name, w.shape, *([dw_dtype] if dw_dtype else [torch.bfloat16, torch.float32]))
        self._call("moe_ffn_backward", x.data_ptr(), dy.data_ptr(), T, _ptr(saved_gu), _ptr(dx),
                   C.MOE_DT_F32 if dx is None else _dtype_code(dx.dtype, "dx"), int(accumulate), *(_ptr(t) for t in dw),
                   _dtype_code(kinds.pop(), "dw") if kinds else C.MOE_DT_F32)
        return dx, dw


@dataclass
class NormForward:
    """What BlockNorm.forward wrote: r (the given one without y), x (None without w_next), rstd [2][T]."""
    r: object
    x: object
    rstd: object


@dataclass
class NormGrads:
    dr: object
    dy: object
    dgate: object
    dw_post: object
    dw_next: object


class BlockNorm(_Handle):
    """Between two blocks: r' = res_scale r + branch_scale gate * rmsnorm(y; w_post), x = rmsnorm(r'; w_next).

    w_post / w_next: [D] bf16 or fp32 (one dtype), None where that norm is missing.  gate: "none", "channel"
    ([D] fp32), "token" ([T] fp32) or "full" ([T][D] of y's dtype).
    """

    _destroy = "moe_norm_destroy"

    def __init__(self, width: int, *, max_tokens: int, w_post=None, w_next=None, gate: str = "none", eps_post: float = 1e-6,
                 eps_next: float = 1e-6, res_scale: float = 1.0, branch_scale: float = 1.0, r_dtype=None, y_dtype=None,
                 x_dtype=None, device=None, backward: bool = True):
        torch = _torch()
        self.D, self.gate = width, gate
        if gate not in GATES:
            raise ValueError(f"gate {gate!r} is not one of {', '.join(GATES)}")
        ws = [w for w in (w_post, w_next) if w is not None]
        if not ws and device is None:
            raise ValueError("a BlockNorm without weights needs a device")
        device = ws[0].device if ws else torch.device(device)
        if device.type == "cuda" and device.index is None:
            device = torch.device("cuda", torch.cuda.current_device())
        self.device = device
        self.r_dtype, self.y_dtype = r_dtype or torch.float32, y_dtype or torch.float32
        self.x_dtype, self.w_dtype = x_dtype or torch.bfloat16, ws[0].dtype if ws else torch.float32
        for w, name in ((w_post, "w_post"), (w_next, "w_next")):
            if w is not None:
                self._take(w, name, (width,), self.w_dtype)
        self._keep = (w_post, w_next)
        d = C.MoeNormDesc()
        C.lib().moe_norm_desc_init(ctypes.byref(d))
        d.width, d.max_tokens, d.gate = width, max_tokens, GATES[gate]
        d.r_dtype, d.y_dtype = _dtype_code(self.r_dtype, "r"), _dtype_code(self.y_dtype, "y")
        d.x_dtype, d.w_dtype = _dtype_code(self.x_dtype, "x"), _dtype_code(self.w_dtype, "w_post and w_next")
        d.eps_post, d.eps_next, d.res_scale, d.branch_scale = eps_post, eps_next, res_scale, branch_scale
        d.flags = (C.MOE_NORM_POST if w_post is not None else 0) | (C.MOE_NORM_NEXT if w_next is not None else 0) | \
            (C.MOE_NORM_BACKWARD if backward else 0)
        self._create(device, d, "moe_norm_workspace_size", lambda L, p, n, out: C.check(
            L.moe_norm_create(ctypes.byref(d), _ptr(w_post), _ptr(w_next), p, n, out), "moe_norm_create"))

    def _gate_shape(self, T):
        return {"channel": (self.D,), "token": (T,), "full": (T, self.D)}[self.gate]

    def _gate_dtype(self):
        return self.y_dtype if self.gate == "full" else _torch().float32

    def _take_gate(self, gate, y, T):
        if (gate is not None) != (y is not None and self.gate != "none"):
            raise ValueError(f"gate={self.gate!r} and y decide whether a gate is given")
        if gate is not None:
            self._take(gate, "gate", self._gate_shape(T), self._gate_dtype())

    def forward(self, r, y=None, *, gate=None, r_out=None, x=None) -> NormForward:
        """Without y the residual passes unchanged and only x is formed.  r_out=r updates it in place."""
        torch = _torch()
        T = int(r.shape[0])
        self._take(r, "r", (T, self.D), self.r_dtype)
        self._take_gate(gate, y, T)
        if y is not None:
            self._take(y, "y", (T, self.D), self.y_dtype)
            r_out = self._new((T, self.D), self.r_dtype) if r_out is None else self._take(r_out, "r_out", (T, self.D), self.r_dtype)
        elif r_out is not None:
            raise ValueError("r_out needs y")
        if self._keep[1] is not None:
            x = self._new((T, self.D), self.x_dtype) if x is None else self._take(x, "x", (T, self.D), self.x_dtype)
        elif x is not None:
            raise ValueError("x needs w_next")
        rstd = self._new((2, T), torch.float32)
        self._call("moe_norm_forward", r.data_ptr(), _ptr(y), _ptr(gate), T, _ptr(r_out), _ptr(x), rstd.data_ptr())
        return NormForward(r if y is None else r_out, x, rstd)

    def backward(self, f: NormForward, y=None, *, gate=None, dr_out=None, dx=None, need_dgate: bool = True,
                 need_dw: bool = True) -> NormGrads:
        """Gradients for the upstream dr_out (None: zero) and dx, with forward's result f and its y and gate."""
        torch = _torch()
        T = int(f.r.shape[0])
        shape = (T, self.D)
        self._take(f.r, "f.r", shape, self.r_dtype)
        self._take(f.rstd, "f.rstd", (2, T), torch.float32)
        self._take_gate(gate, y, T)
        if y is not None:
            self._take(y, "y", shape, self.y_dtype)
        if dr_out is not None:
            self._take(dr_out, "dr_out", shape, self.r_dtype)
        if (dx is not None) != (self._keep[1] is not None):
            raise ValueError("dx is given exactly where there is w_next")
        if dx is not None:
            self._take(dx, "dx", shape, self.x_dtype)
        dr = self._new(shape, self.r_dtype)
        dy = None if y is None else self._new(shape, self.y_dtype)
        dgate = self._new(self._gate_shape(T), self._gate_dtype()) if gate is not None and need_dgate else None
        dw = [self._new((self.D,), self.w_dtype) if need_dw and w is not None and used else None
              for w, used in ((self._keep[0], y is not None), (self._keep[1], True))]
        self._call("moe_norm_backward", _ptr(y), _ptr(gate), f.r.data_ptr(), f.rstd.data_ptr(), _ptr(dr_out), _ptr(dx), T,
                   dr.data_ptr(), _ptr(dy), _ptr(dgate), _ptr(dw[0]), _ptr(dw[1]))
        return NormGrads(dr, dy, dgate, *dw)


class AdamW(_Handle):
    """One AdamW step over all tensors at once.

    params, grads: lists of bf16 or fp32 tensors (grads of the same shapes, read at every step; replace them
    with set_grads).  m, v: the states, fp32 like the parameters, or uint8 / float8_e4m3fn with m_scale and v_scale
    ([ceil(n / 256)] fp32); new_state() makes zero ones.  master: fp32 copies that the step updates, or None (a list
    may hold None).  weight_decay and lr_scale: one number or one for each tensor.  step: steps taken so far.
    """

    _destroy = "moe_adamw_destroy"

    def __init__(self, params: Sequence, grads: Sequence, *, m: Sequence, v: Sequence, m_scale: Optional[Sequence] = None,
                 v_scale: Optional[Sequence] = None, master: Optional[Sequence] = None, betas=(0.9, 0.999), eps: float = 1e-8,
                 weight_decay=0.01, lr_scale=1.0, max_norm: float = 0.0, step: int = 0, device=None):
        torch = _torch()
        n = len(params)
        none = [None] * n
        self.params, self.m, self.v = list(params), list(m), list(v)
        self.m_scale, self.v_scale, self.master = (list(none if t is None else t) for t in (m_scale, v_scale, master))
        per = lambda a: list(a) if isinstance(a, (list, tuple)) else [a] * n  # noqa: E731
        self.weight_decay, self.lr_scale = per(weight_decay), per(lr_scale)
        for name in ("m", "v", "m_scale", "v_scale", "master", "weight_decay", "lr_scale"):
            if len(getattr(self, name)) != n:
                raise ValueError(f"{name} has {len(getattr(self, name))} entries for {n} parameters")
        if not n and device is None:
            raise ValueError("an AdamW without parameters needs a device")
        device = self.params[0].device if n else torch.device(device)
        if device.type == "cuda" and device.index is None:
            device = torch.device("cuda", torch.cuda.current_device())
        self.device = device
        self.e4m3 = m_scale is not None
        f32 = torch.float32
        states = (torch.uint8, torch.float8_e4m3fn) if self.e4m3 else (f32,)
        for i, p in enumerate(self.params):
            self._take(p, f"params[{i}]", p.shape, torch.bfloat16, f32)
            self._take(self.m[i], f"m[{i}]", p.shape, *states)
            self._take(self.v[i], f"v[{i}]", p.shape, *states)
            for s, name in ((self.m_scale[i], "m_scale"), (self.v_scale[i], "v_scale")):
                if (s is not None) != self.e4m3:
                    raise ValueError(f"{name}[{i}]: 8-bit states have scales, fp32 states none")
                if s is not None:
                    self._take(s, f"{name}[{i}]", (-(-p.numel() // 256),), f32)
            if self.master[i] is not None:
                self._take(self.master[i], f"master[{i}]", p.shape, f32)
        d = C.MoeAdamwDesc()
        C.lib().moe_adamw_desc_init(ctypes.byref(d))
        d.beta1, d.beta2, d.eps, d.max_norm = betas[0], betas[1], eps, max_norm
        d.state = C.MOE_STATE_E4M3 if self.e4m3 else C.MOE_STATE_F32
        d.max_tensors, d.max_elements = max(1, n), sum(p.numel() for p in self.params)
        self._create(device, d, "moe_adamw_workspace_size", lambda L, p, nb, out: C.check(
            L.moe_adamw_create(ctypes.byref(d), p, nb, out), "moe_adamw_create"))
        self.set_grads(grads)
        self.set_step(step)

    @staticmethod
    def new_state(params: Sequence, e4m3: bool = False) -> dict:
        """Zero m, v (and scales) for these parameters, as keyword arguments of AdamW."""
        torch = _torch()
        if not e4m3:
            return {k: [torch.zeros_like(p, dtype=torch.float32) for p in params] for k in ("m", "v")}
        codes = {k: [torch.zeros_like(p, dtype=torch.uint8) for p in params] for k in ("m", "v")}
        return codes | {k: [torch.zeros(-(-p.numel() // 256), dtype=torch.float32, device=p.device) for p in params]
                        for k in ("m_scale", "v_scale")}

    def set_grads(self, grads: Sequence):
        """Read the gradients from these tensors from now on (enqueued on the current stream)."""
        torch = _torch()
        grads = list(grads)
        if len(grads) != len(self.params):
            raise ValueError(f"{len(grads)} gradients for {len(self.params)} parameters")
        for i, (g, p) in enumerate(zip(grads, self.params)):
            self._take(g, f"grads[{i}]", p.shape, torch.bfloat16, torch.float32)
        n = len(grads)
        tab = (C.MoeAdamwTensor * max(1, n))()
        for i, (p, g) in enumerate(zip(self.params, grads)):
            e = tab[i]
            e.param, e.grad, e.m, e.v = p.data_ptr(), g.data_ptr(), self.m[i].data_ptr(), self.v[i].data_ptr()
            e.master, e.m_scale, e.v_scale = _ptr(self.master[i]), _ptr(self.m_scale[i]), _ptr(self.v_scale[i])
            e.n, e.param_dtype, e.grad_dtype = p.numel(), _dtype_code(p.dtype, "param"), _dtype_code(g.dtype, "grad")
            e.weight_decay, e.lr_scale = self.weight_decay[i], self.lr_scale[i]
        self._call("moe_adamw_bind", tab, n)
        self.grads = grads

    def set_step(self, step: int):
        """The number of steps taken so far (kept on the device, counted by every step and replay)."""
        self._call("moe_adamw_set_step", step)

    def step(self, lr, grad_norm=None):
        """lr: a number, or a one-element fp32 device tensor read when the step runs.  grad_norm: a one-element
        fp32 device tensor that receives the norm before clipping (with max_norm)."""
        f32 = _torch().float32
        on_device = hasattr(lr, "data_ptr")
        if on_device:
            self._take(lr, "lr", lr.shape if lr.numel() == 1 else (1,), f32)
        if grad_norm is not None:
            self._take(grad_norm, "grad_norm", grad_norm.shape if grad_norm.numel() == 1 else (1,), f32)
        self._call("moe_adamw_step", 0.0 if on_device else float(lr), lr.data_ptr() if on_device else None, _ptr(grad_norm))
