"""Binding of include/nvfp4_train.h: the operators of a quantization-aware-distillation step
around ``fakequant_ste`` and ``qad_kl``: layer norm (forward with the amax of its result, and
backward), the global gradient norm with its clip factor, and AdamW over many tensors at once
with the states in 32 bits or in 8.

``nvfp4_*`` mirror the C ABI one to one; the wrappers allocate with torch and check shapes,
types and devices. Tensors are CUDA, contiguous and on one device, which need not be the current
one; the work goes to ``stream``, or to the current stream of the tensors' device. A ``stream`` that is
not the current one must be ordered behind it (``stream.wait_stream``), because inputs come from there and
outputs are allocated there, and the current one behind ``stream`` before it uses the outputs.
Memory of the inputs and outputs is held until the work is done, that of a list or plan as long as its
caller keeps it: keep it until then.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import math
from typing import NamedTuple

from . import _check, _ptr, _stream, load

__all__ = [
    "TYPE_BF16", "TYPE_F32", "OptTensor", "nvfp4_layer_norm", "nvfp4_layer_norm_workspace",
    "nvfp4_layer_norm_backward", "nvfp4_tensor_plan_bytes", "nvfp4_tensor_plan", "nvfp4_grad_norm", "nvfp4_adamw",
    "Normed", "layer_norm", "layer_norm_forward", "layer_norm_backward",
    "GradientList", "AdamWPlan", "gradient_list", "adamw_plan", "grad_norm", "adamw",
]

TYPE_BF16, TYPE_F32 = 0, 1
_GRAD_NORM_WORKSPACE = 16400
_STATE_ALIGN = 128      # elements: a tensor's states start on a multiple of it


class OptTensor(ctypes.Structure):
    """nvfp4_opt_tensor."""
    _fields_ = [("param", ctypes.c_void_p), ("grad", ctypes.c_void_p), ("master", ctypes.c_void_p),
                ("exp_avg", ctypes.c_void_p), ("exp_avg_sq", ctypes.c_void_p), ("exp_avg_scale", ctypes.c_void_p),
                ("exp_avg_sq_scale", ctypes.c_void_p), ("numel", ctypes.c_int64), ("first", ctypes.c_int64),
                ("weight_decay", ctypes.c_float), ("param_type", ctypes.c_int32), ("grad_type", ctypes.c_int32),
                ("state_bits", ctypes.c_int32)]


# ---- the C ABI, one to one -------------------------------------------------------------------

def nvfp4_layer_norm(x, x_type, weight, bias, w_type, rows, cols, eps, y, mean=None, rstd=None, amax=None, stream=None):
    _check(load().nvfp4_layer_norm(_ptr(x), x_type, _ptr(weight), _ptr(bias), w_type, rows, cols, eps, _ptr(y),
                                   _ptr(mean), _ptr(rstd), _ptr(amax), _stream(stream)), "nvfp4_layer_norm")


def nvfp4_layer_norm_workspace(rows, cols) -> int:
    return load().nvfp4_layer_norm_workspace(rows, cols)


def nvfp4_layer_norm_backward(dy, x, x_type, weight, w_type, mean, rstd, rows, cols, dx, dweight=None, dbias=None,
                              workspace=None, workspace_bytes=0, stream=None):
    _check(load().nvfp4_layer_norm_backward(_ptr(dy), _ptr(x), x_type, _ptr(weight), w_type, _ptr(mean), _ptr(rstd),
                                            rows, cols, _ptr(dx), _ptr(dweight), _ptr(dbias), _ptr(workspace),
                                            workspace_bytes, _stream(stream)), "nvfp4_layer_norm_backward")


def nvfp4_tensor_plan_bytes(tensors, count) -> int:
    return load().nvfp4_tensor_plan_bytes(tensors, count)


def nvfp4_tensor_plan(tensors, count, image, image_bytes) -> int:
    """Writes the plan to host memory and returns the number of chunks."""
    chunks = ctypes.c_int64()
    _check(load().nvfp4_tensor_plan(tensors, count, image, image_bytes, ctypes.byref(chunks)), "nvfp4_tensor_plan")
    return chunks.value


def nvfp4_grad_norm(plan, chunks, max_norm, norm, scale, workspace, stream=None):
    _check(load().nvfp4_grad_norm(_ptr(plan), chunks, max_norm, _ptr(norm), _ptr(scale), _ptr(workspace),
                                  _stream(stream)), "nvfp4_grad_norm")


def nvfp4_adamw(plan, chunks, state_bits, control, lr, lr_device, beta1, beta2, eps, seed, scale=None, amax=None, count=0,
                stream=None):
    _check(load().nvfp4_adamw(_ptr(plan), chunks, state_bits, _ptr(control), lr, _ptr(lr_device), beta1, beta2, eps, seed,
                              _ptr(scale), _ptr(amax), count, _stream(stream)), "nvfp4_adamw")


# ---- what the wrappers share ---------------------------------------------------------------------
#
# A step calls these operators many times on small tensors, where the host's part of a call is what
# counts: torch is looked up once, and a stream is taken as a number.

_torch = None
_types = {}
_HERE = contextlib.nullcontext()


def _load_torch():
    global _torch, _types
    import torch

    _types = {torch.bfloat16: TYPE_BF16, torch.float32: TYPE_F32}
    _torch = torch
    return torch


def _type_of(t, what):
    code = _types.get(t.dtype)
    if code is None:
        raise ValueError(f"nvfp4: {what} must be BF16 or FP32, not {t.dtype}")
    return code


def _on(device):
    """A context in which `device` is current."""
    return _HERE if _torch._C._cuda_getDevice() == device.index else _torch.cuda.device(device)


def _raw(stream, device):
    """The stream as a number; None: the current one of `device`."""
    if stream is None:
        return _torch._C._cuda_getCurrentRawStream(device.index)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _lend(stream, *tensors):
    """Memory that torch's current stream allocated and `stream` works on is kept until that work is done."""
    given = [t for t in tensors if t is not None]
    device = given[0].device
    raw = _raw(stream, device)
    if raw != _raw(None, device):
        if isinstance(stream, int):
            stream = _torch.cuda.ExternalStream(stream, device=device)
        for t in given:
            t.record_stream(stream)


def _address(t):
    if not t.is_contiguous():
        raise ValueError("nvfp4: tensors must be contiguous")
    return t.data_ptr()


def _same(t, x, shape, what, dtype=None):
    if t.get_device() != x.get_device():
        raise ValueError(f"nvfp4: {what} must be on {x.device}, not {t.device}")
    if t.shape != shape:
        raise ValueError(f"nvfp4: {what} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"nvfp4: {what} must be {dtype}, not {t.dtype}")


# ---- layer norm ----------------------------------------------------------------------------------

class Normed(NamedTuple):
    y: "object"       # as x
    mean: "object"    # float32 [rows] or None
    rstd: "object"    # float32 [rows] or None
    amax: "object"    # float32 [1] or None: max |y|, the amax of y's quantization


def _rows(x):
    """(rows, cols, type) of a norm's input."""
    if _torch is None:
        _load_torch()
    shape = x.shape
    if not shape or shape[-1] < 1:
        raise ValueError("layer_norm: x must have a last dimension of at least 1")
    if not x.is_cuda:
        raise ValueError("nvfp4: tensors must live on a CUDA device")
    return x.numel() // shape[-1], shape[-1], _type_of(x, "x")


def _affine(x, weight, bias, cols):
    """The type of weight and bias, which agree."""
    if weight is None and bias is None:
        return TYPE_F32
    first = bias if weight is None else weight
    _same(first, x, (cols,), "bias" if weight is None else "weight")
    if bias is not None and bias is not first:
        _same(bias, x, (cols,), "bias", first.dtype)
    return _type_of(first, "weight and bias")


def layer_norm_forward(x, weight=None, bias=None, eps: float = 1e-5, with_stats=True, with_amax=False,
                       stream=None) -> Normed:
    """Layer norm of BF16 or FP32 x over its last dimension; weight and bias (BF16 or FP32, [cols])
    may be None. ``with_stats`` returns what the backward pass needs, ``with_amax`` the amax of
    y, ready for ``quantize`` and ``quantize_for_gemm``. No autograd: see ``layer_norm``."""
    rows, cols, x_type = _rows(x)
    w_type = _affine(x, weight, bias, cols)
    device, mean, rstd, top = x.device, None, None, None
    with _on(device):
        source = _address(x)   # refuses what is not contiguous before anything is allocated
        w, b = None if weight is None else _address(weight), None if bias is None else _address(bias)
        y = _torch.empty_like(x)
        if with_stats:
            mean = _torch.empty(rows, dtype=_torch.float32, device=device)
            rstd = _torch.empty(rows, dtype=_torch.float32, device=device)
        if with_amax:
            top = _torch.empty(1, dtype=_torch.float32, device=device)
        status = load().nvfp4_layer_norm(source, x_type, w, b, w_type, rows, cols, eps, y.data_ptr(),
                                         mean.data_ptr() if with_stats else None, rstd.data_ptr() if with_stats else None,
                                         top.data_ptr() if with_amax else None, _raw(stream, device))
        if status:
            _check(status, "nvfp4_layer_norm")
        if stream is not None:
            _lend(stream, x, weight, bias, y, mean, rstd, top)
    return Normed(y, mean, rstd, top)


@functools.lru_cache(maxsize=256)
def _workspace(rows, cols, device):
    """nvfp4_layer_norm_workspace on `device`, which is current."""
    return load().nvfp4_layer_norm_workspace(rows, cols)


def layer_norm_backward(dy, x, weight, mean, rstd, with_weight=True, with_bias=True, stream=None):
    """(dx, dweight, dbias) of layer norm from its input and the statistics of its forward pass.
    dweight and dbias have the weight's type (FP32 without one); None where not asked for."""
    rows, cols, x_type = _rows(x)
    _same(dy, x, x.shape, "dy", x.dtype)
    _same(mean, x, (rows,), "mean", _torch.float32)
    _same(rstd, x, (rows,), "rstd", _torch.float32)
    w_type = _affine(x, weight, None, cols)
    device, dweight, dbias, work, size = x.device, None, None, None, 0
    with _on(device):
        sources = _address(dy), _address(x)
        w = None if weight is None else _address(weight)
        dx = _torch.empty_like(x)
        dtype = _torch.float32 if weight is None else weight.dtype
        if with_weight:
            dweight = _torch.empty(cols, dtype=dtype, device=device)
        if with_bias:
            dbias = _torch.empty(cols, dtype=dtype, device=device)
        if with_weight or with_bias:
            size = _workspace(rows, cols, device.index)
            work = _torch.empty(size, dtype=_torch.uint8, device=device)
        status = load().nvfp4_layer_norm_backward(*sources, x_type, w, w_type, _address(mean), _address(rstd), rows, cols, dx.data_ptr(),
                                                  dweight.data_ptr() if with_weight else None, dbias.data_ptr() if with_bias else None,
                                                  work.data_ptr() if size else None, size, _raw(stream, device))
        if status:
            _check(status, "nvfp4_layer_norm_backward")
        if stream is not None:
            _lend(stream, dy, x, weight, mean, rstd, dx, dweight, dbias, work)
    return dx, dweight, dbias


@functools.lru_cache(maxsize=None)
def _layer_norm_function():
    torch = _torch

    class _LayerNorm(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, weight, bias, eps, with_amax):
            r = layer_norm_forward(x, weight, bias, eps, True, with_amax)
            ctx.save_for_backward(x, weight, r.mean, r.rstd)
            ctx.bias_dtype = None if bias is None else bias.dtype
            if not with_amax:
                return r.y
            ctx.mark_non_differentiable(r.amax)
            return r.y, r.amax

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, dy, *_):
            x, weight, mean, rstd = ctx.saved_tensors
            needs = ctx.needs_input_grad
            dx, dweight, dbias = layer_norm_backward(dy.contiguous(), x, weight, mean, rstd, needs[1], needs[2])
            if dbias is not None:
                dbias = dbias.to(ctx.bias_dtype)
            return dx if needs[0] else None, dweight, dbias, None, None

    return _LayerNorm


def _has_tangent(*tensors):
    """Whether one of them is dual (forward-mode differentiation)."""
    forward_ad = _torch.autograd.forward_ad
    if forward_ad._current_level < 0:   # not inside a dual level: the usual case, at the price of one look
        return False
    return any(t is not None and forward_ad.unpack_dual(t).tangent is not None for t in tensors)


def layer_norm(x, weight=None, bias=None, eps: float = 1e-5, with_amax=False):
    """y, or (y, amax): layer norm with autograd through x, weight and bias. The amax [1] is that
    of y's quantization (``fakequant_ste(y, amax_values=amax)``, ``quantize_for_gemm``). Derivatives
    are those of the backward pass: forward-mode ones are refused, as in ``fakequant_ste``."""
    torch = _torch or _load_torch()
    if (torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in (x, weight, bias))) or _has_tangent(x, weight, bias):
        return _layer_norm_function().apply(x, weight, bias, eps, with_amax)
    r = layer_norm_forward(x, weight, bias, eps, False, with_amax)
    return (r.y, r.amax) if with_amax else r.y


# ---- lists of tensors ------------------------------------------------------------------------------

class GradientList:
    """Gradients whose norm ``grad_norm`` takes: their table on the device, and the kernel's
    scratch. The tensors are the ones given: write new gradients into them. Calls with one list
    must not overlap on the GPU."""

    def __init__(self, grads, device, records):
        torch = _torch
        self.grads, self.device, self.count = grads, device, len(records)
        self.held = [g.detach() for g in grads]   # their memory, which the table points to, whatever becomes of the tensors
        array = (OptTensor * max(1, len(records)))(*records)
        size = nvfp4_tensor_plan_bytes(array, len(records))
        if size < 0:
            raise ValueError("nvfp4: too many tensors or elements in one list")
        image = torch.empty(size, dtype=torch.uint8)
        self.chunks = nvfp4_tensor_plan(array, len(records), image.data_ptr(), size)
        self.table = image.to(device)
        self.work = torch.zeros(_GRAD_NORM_WORKSPACE, dtype=torch.uint8, device=device)
        self.table_ptr, self.work_ptr = self.table.data_ptr(), self.work.data_ptr()


class AdamWPlan(GradientList):
    """Parameters, gradients and AdamW states of one list (see ``adamw_plan``).

    ``exp_avg``, ``exp_avg_sq`` (and ``master``, ``exp_avg_scale``, ``exp_avg_sq_scale``) are flat
    buffers; those of tensor i start at ``offsets[i]`` (scales at ``offsets[i] // 32``), and
    ``state(i)`` gives them as views. With 8-bit states ``exp_avg_sq`` holds codes of the second
    moment's root. ``amax`` [count] is written by every ``adamw`` (None without ``with_amax``)."""

    def check_parameters(self):
        """Refuses a step on memory that is no longer the parameters'."""
        if list(map(_torch.Tensor.data_ptr, self.params)) != self.addresses:
            raise ValueError("nvfp4: a parameter's memory is no longer the one that the plan was made with (as after .to() or an assignment "
                             "to .data): make a new plan")

    def check_gradients(self):
        """Refuses a step on gradients that are no longer the parameters' own."""
        for p, g in self.own_gradients:
            now = p.grad
            if now is not g and (now is None or now.data_ptr() != g.data_ptr() or now.dtype != g.dtype or not now.is_contiguous()):
                raise ValueError("nvfp4: a parameter's .grad is no longer the gradient that the plan was made with: clear gradients in "
                                 "place (zero_grad(set_to_none=False)), or make a new plan")

    def steps(self) -> int:
        """Steps taken so far (waits for the current stream)."""
        return int(self.control[4].item())

    def set_steps(self, steps: int):
        """Sets the count of steps, as after loading the states of a checkpoint."""
        self.control.copy_(_control(steps, self.betas))

    def state(self, i: int) -> dict:
        at, n = self.offsets[i], self.numels[i]
        out = {"exp_avg": self.exp_avg[at:at + n], "exp_avg_sq": self.exp_avg_sq[at:at + n]}
        if self.master is not None:
            out["master"] = self.master[at:at + n]
        if self.state_bits == 8:
            blocks = slice(at // 32, at // 32 + (n + 31) // 32)
            out["exp_avg_scale"], out["exp_avg_sq_scale"] = self.exp_avg_scale[blocks], self.exp_avg_sq_scale[blocks]
        return out


def _control(steps, betas):
    """nvfp4_adamw_control after `steps` steps, as 8 words on the host."""
    torch = _torch
    if not 0 <= steps < 1 << 32:
        raise ValueError("nvfp4: the number of steps must be in [0, 2^32)")
    powers = torch.tensor([betas[0] ** steps, betas[1] ** steps], dtype=torch.float64).view(torch.int32)
    count = torch.tensor([steps - (1 << 32) if steps >= 1 << 31 else steps, 0, 0, 0], dtype=torch.int32)
    return torch.cat([powers, count])


def _list_of(tensors, what):
    if _torch is None:
        _load_torch()
    tensors = list(tensors)
    if not tensors or not sum(t.numel() for t in tensors):
        raise ValueError(f"nvfp4: {what} are empty")
    for t in tensors:
        if t.device != tensors[0].device:
            raise ValueError(f"nvfp4: {what} must be on one device")
        _ptr(t)   # CUDA and contiguous
    return tensors


def gradient_list(grads) -> GradientList:
    """A list of BF16 or FP32 gradients for ``grad_norm``."""
    grads = _list_of(grads, "grads")
    with _on(grads[0].device):
        return GradientList(grads, grads[0].device,
                            [OptTensor(grad=g.data_ptr(), numel=g.numel(), grad_type=_type_of(g, "a gradient")) for g in grads])


def adamw_plan(params, grads, state_bits: int = 32, masters=False, weight_decay=0.01, betas=(0.9, 0.999),
               eps: float = 1e-8, seed: int = 0, step: int = 0, with_amax=False) -> AdamWPlan:
    """AdamW over `params` (BF16 or FP32) with the gradients in `grads`, which keep their memory
    from step to step (assign them to ``p.grad`` and clear them in place). Where a parameter's ``.grad``
    is the given gradient, ``adamw`` and ``grad_norm`` refuse the plan once it has been replaced, as by
    ``zero_grad()``, which sets it to None; other gradients are read where they were. A parameter that
    was given other memory, as by ``module.to()``, is refused likewise.

    ``state_bits``: 32, or 8 (E4M3 with a power-of-two scale for each 32 elements). ``masters``: an
    FP32 master of every BF16 parameter; without one a BF16 parameter is rounded stochastically.
    ``weight_decay``: one number, or one for each tensor. ``seed`` (32 bits) of the stochastic
    rounding. ``step``: steps taken before. States start at zero, masters at the parameters."""
    params, grads = _list_of(params, "params"), _list_of(grads, "grads")
    torch = _torch
    if len(params) != len(grads):
        raise ValueError("adamw_plan: one gradient for each parameter")
    decays = [float(weight_decay)] * len(params) if isinstance(weight_decay, (int, float)) else [float(d) for d in weight_decay]
    if len(decays) != len(params):
        raise ValueError("adamw_plan: one weight decay, or one for each parameter")
    if state_bits not in (32, 8):
        raise ValueError("adamw_plan: state_bits must be 32 or 8")
    if not (0 <= betas[0] < 1 and 0 <= betas[1] < 1) or not 0 <= eps < math.inf or not 0 <= seed < 1 << 32:
        raise ValueError("adamw_plan: betas must be in [0, 1), eps finite and >= 0, seed in [0, 2^32)")
    device = params[0].device
    offsets, total = [], 0
    for p, g in zip(params, grads):
        _same(g, p, p.shape, "a gradient")
        offsets.append(total)
        total += -(-p.numel() // _STATE_ALIGN) * _STATE_ALIGN
    flat = {}
    with _on(device), torch.no_grad():
        master = torch.zeros(total, dtype=torch.float32, device=device) if masters else None
        for name in ("exp_avg", "exp_avg_sq"):
            if state_bits == 32:
                flat[name] = torch.zeros(total, dtype=torch.float32, device=device)
            else:
                flat[name] = torch.zeros(total, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn)
                flat[name + "_scale"] = torch.ones(total // 32, dtype=torch.uint8, device=device).view(torch.float8_e8m0fnu)
        records = []
        for p, g, at, decay in zip(params, grads, offsets, decays):
            record = OptTensor(param=p.data_ptr(), grad=g.data_ptr(), numel=p.numel(), first=at, weight_decay=decay,
                               param_type=_type_of(p, "a parameter"), grad_type=_type_of(g, "a gradient"), state_bits=state_bits)
            if masters and p.dtype == torch.bfloat16:
                master[at:at + p.numel()].copy_(p.detach().reshape(-1))
                record.master = master.data_ptr() + 4 * at
            for name in ("exp_avg", "exp_avg_sq"):
                setattr(record, name, flat[name].data_ptr() + at * flat[name].element_size())
                if state_bits == 8:
                    setattr(record, name + "_scale", flat[name + "_scale"].data_ptr() + at // 32)
            records.append(record)
        plan = AdamWPlan(grads, device, records)
        plan.params, plan.offsets, plan.numels = params, offsets, [p.numel() for p in params]
        plan.held += [p.detach() for p in params]
        plan.addresses = [p.data_ptr() for p in params]
        plan.own_gradients = [(p, g) for p, g in zip(params, grads) if p.is_leaf and p.grad is g]
        # every parameter's version, whether it requires a gradient or not: views share their base's
        plan.versioned = list({id(b): b for b in (p if p._base is None else p._base for p in params)}.values())
        plan.state_bits, plan.betas, plan.eps, plan.seed = state_bits, (float(betas[0]), float(betas[1])), float(eps), seed
        plan.master, plan.exp_avg, plan.exp_avg_sq = master, flat["exp_avg"], flat["exp_avg_sq"]
        plan.exp_avg_scale, plan.exp_avg_sq_scale = flat.get("exp_avg_scale"), flat.get("exp_avg_sq_scale")
        plan.control = _control(step, plan.betas).to(device)
        plan.amax = torch.zeros(len(params), dtype=torch.float32, device=device) if with_amax else None
        plan.control_ptr, plan.amax_ptr = plan.control.data_ptr(), plan.amax.data_ptr() if with_amax else None
    return plan


def grad_norm(grads: GradientList, max_norm: float = math.inf, stream=None):
    """(norm, scale), each [1] on the device: the norm of all gradients of the list together and
    min(1, max_norm / (norm + 1e-6)). A norm that is not finite gives a NaN scale, with which
    ``adamw`` leaves everything as it is."""
    if not isinstance(grads, GradientList):
        raise ValueError("grad_norm: needs a list of gradient_list, or a plan of adamw_plan")
    if isinstance(grads, AdamWPlan):
        grads.check_gradients()
    device = grads.device
    with _on(device):
        norm = _torch.empty(1, dtype=_torch.float32, device=device)
        scale = _torch.empty(1, dtype=_torch.float32, device=device)
        status = load().nvfp4_grad_norm(grads.table_ptr, grads.chunks, max_norm, norm.data_ptr(), scale.data_ptr(), grads.work_ptr,
                                        _raw(stream, device))
        if status:
            _check(status, "nvfp4_grad_norm")
        if stream is not None:
            _lend(stream, norm, scale)
    return norm, scale


def adamw(plan: AdamWPlan, lr, scale=None, stream=None):
    """One AdamW step, in place: autograd's graphs that saved a parameter notice (not at a replay of
    a captured call). ``lr``: a number, or an FP32 [1] tensor that the kernel reads (a captured call
    then follows it; the count of steps is kept on the device anyway). ``scale``: an FP32 [1] factor
    of the gradients, as ``grad_norm`` gives it."""
    if not isinstance(plan, AdamWPlan):
        raise ValueError("adamw: needs a plan of adamw_plan")
    plan.check_parameters()
    plan.check_gradients()
    lr_tensor = None
    if isinstance(lr, _torch.Tensor):
        _same(lr, plan.control, (1,), "lr", _torch.float32)
        lr, lr_tensor = 0.0, lr
    if scale is not None:
        _same(scale, plan.control, (1,), "scale", _torch.float32)
    with _on(plan.device):
        status = load().nvfp4_adamw(plan.table_ptr, plan.chunks, plan.state_bits, plan.control_ptr, float(lr),
                                    None if lr_tensor is None else lr_tensor.data_ptr(), plan.betas[0], plan.betas[1], plan.eps, plan.seed,
                                    None if scale is None else scale.data_ptr(), plan.amax_ptr, plan.count, _raw(stream, plan.device))
        if status:
            _check(status, "nvfp4_adamw")
        if stream is not None:
            _lend(stream, plan.control, lr_tensor, scale)
    _torch.autograd.graph.increment_version(plan.versioned)
