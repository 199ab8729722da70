"""The operators at a layer's ends: the norm of the recurrence's output with
its gate, the norms on both sides of the residual's addition, rows in 8 bits
and the product of 8-bit integers.

Thin bindings over libgdr.so, re-exported by the package, in the manner of
:mod:`._layer_ops`: PyTorch provides device memory, the current stream and
autograd; every computation runs in the library's HIP kernels.
"""
from __future__ import annotations

import ctypes

import torch
from torch.autograd.function import once_differentiable

from ._layer_ops import (_DT, _FORMATS, _QUANTISED, _bytes, _code, _expect, _fits, _launch, _like,
                         _need_gpu, _new, _ptr, _token_rows)
from ._lib import (GatedNormProblem, GdrError, Int8MatmulProblem, QuantizeProblem,
                   SandwichNormProblem, lib)

_ACTIVATIONS = {None: 0, "none": 0, "silu": 1, "swish": 1, "sigmoid": 2}


def _activation(name, needed):
    code = _ACTIVATIONS.get(name)
    if code is None or (needed and code == 0):
        raise GdrError(10, "activation must be 'silu' or 'sigmoid'%s, got %r"
                       % ("" if needed else " or None", name))
    return code


def _rows(x):
    """(x, stride): x [..., D] as rows one stride apart, a slice of a wider
    tensor in place, else a copy."""
    if x.dim() == 1 or x.is_contiguous():
        return (x if x.is_contiguous() else x.contiguous()), x.shape[-1]
    return _token_rows(x.unsqueeze(0) if x.dim() == 2 else x.flatten(0, -3) if x.dim() > 3 else x, 1)


def _count(x, name="x"):
    """(rows, D) of x [..., D]."""
    if x.dim() < 1:
        raise GdrError(2, "%s must be [..., D], got %s" % (name, tuple(x.shape)))
    D = x.shape[-1]
    rows = x.numel() // D if D else 0
    _fits(name, rows, D)
    return rows, D


def _format(fmt, group_size):
    if fmt not in _QUANTISED:
        raise GdrError(10, "format must be 'fp8' or 'int8', got %r" % (fmt,))
    # the number of scales follows from it before the library sees it
    if group_size not in (0, 128):
        raise GdrError(10, "group_size must be 0 (the row) or 128, got %r" % (group_size,))
    return _FORMATS[fmt], int(group_size)


def _eight_bits(x, D, fmt, group_size):
    """New (q, scale) of rows x [..., D]."""
    groups = 1 if group_size == 0 else -(-D // 128)
    return _new(x, _QUANTISED[fmt]), x.new_empty(x.shape[:-1] + (groups,), dtype=torch.float32)


# ---- RMS norm with a gate ------------------------------------------------------

class _Gated:
    """The checked arguments of one gated norm call."""

    def __init__(self, x, gate, weight, eps, norm_group, norm_before_gate, activation, fmt=0,
                 scale_group=0):
        rows, D = _count(x)
        if not isinstance(norm_group, int) or norm_group < 0:
            raise GdrError(10, "norm_group must be 0 (the row) or its columns, got %r" % (norm_group,))
        size = norm_group or D
        act = _activation(activation, True)
        _need_gpu("x", x)
        dt = _code(x, "x")
        if size < 1 or D % size:
            raise GdrError(2, "the %d columns must be a multiple of norm_group, got %d" % (D, size))
        _expect("gate", gate, x.shape, (x.dtype,), x.device)
        shared = weight.dim() == 1 and weight.shape[0] == size
        self.weight = _like("weight", weight, (size,) if shared else (D,), (x.dtype, torch.float32),
                            x.device)
        self.x, xs = _rows(x)
        self.gate, zs = _rows(gate)
        self.groups = D // size
        self.p = GatedNormProblem(rows, D, size, dt, _DT[weight.dtype], 1 if shared else 0,
                                  0 if norm_before_gate else 1, act, fmt, scale_group, float(eps),
                                  xs, zs)
        self.ref = ctypes.byref(self.p)


def gated_rms_norm_fwd(x, gate, weight, eps=1e-6, norm_group=0, norm_before_gate=True,
                       activation="silu"):
    """:func:`gated_rms_norm` without autograd: ``(y, rstd)``, ``rstd`` (fp32,
    ``x.shape[:-1] + (groups,)``) for :func:`gated_rms_norm_bwd`."""
    c = _Gated(x, gate, weight, eps, norm_group, norm_before_gate, activation)
    y = _new(x)
    rstd = x.new_empty(x.shape[:-1] + (c.groups,), dtype=torch.float32)
    _launch(x, lib.gdr_gated_norm_fwd, c.ref, _ptr(c.x), _ptr(c.gate), _ptr(c.weight), _ptr(y), None,
            _ptr(rstd))
    return y, rstd


def gated_rms_norm_bwd(dy, x, gate, weight, rstd, norm_group=0, norm_before_gate=True,
                       activation="silu"):
    """The gradient of :func:`gated_rms_norm`: ``(dx, dgate, dweight)``; ``rstd``
    comes from :func:`gated_rms_norm_fwd`."""
    c = _Gated(x, gate, weight, 0.0, norm_group, norm_before_gate, activation)
    dev = x.device
    dy = _like("dy", dy, x.shape, (x.dtype,), dev)
    rstd = _like("rstd", rstd, x.shape[:-1] + (c.groups,), (torch.float32,), dev)
    dx, dgate, dw = _new(x), _new(x), torch.empty_like(c.weight)
    n = lib.gdr_gated_norm_bwd_workspace_size(c.ref)
    ws = _bytes(n, dev)
    _launch(x, lib.gdr_gated_norm_bwd, c.ref, _ptr(dy), _ptr(c.x), _ptr(c.gate), _ptr(c.weight),
            _ptr(rstd), _ptr(dx), _ptr(dgate), _ptr(dw), _ptr(ws), n)
    return dx, dgate, dw


class _GatedRmsNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, gate, weight, eps, *how):
        y, rstd = gated_rms_norm_fwd(x, gate, weight, eps, *how)
        ctx.save_for_backward(x, gate, weight, rstd)
        ctx.how = how
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        return gated_rms_norm_bwd(dy, *ctx.saved_tensors, *ctx.how) + (None,) * 4


def gated_rms_norm(x, gate, weight, eps=1e-6, norm_group=0, norm_before_gate=True,
                   activation="silu"):
    """Root-mean-square norm of a recurrence's output with its gate, with
    autograd.

    Over each group of ``norm_group`` consecutive columns of the last dimension
    (a head, 8 or more; 0: all of them) ``y = weight * x / rms(x) * act(gate)``, as a
    gated delta rule's layer has it, or with ``norm_before_gate=False`` ``y = weight
    * v / rms(v)``, ``v = x * act(gate)``, as a selective scan's has it; ``rms(v) =
    sqrt(mean(v^2) + eps)``, ``act`` ``"silu"`` or ``"sigmoid"``.  x and gate ``[..., D]``
    in bf16, fp16 or fp32 (slices of a wider projection are read in place);
    weight ``[norm_group]`` for all groups or ``[D]``, in x's dtype or fp32; D up
    to 16384.  Gradients flow to x, gate and weight."""
    return _GatedRmsNorm.apply(x, gate, weight, eps, norm_group, norm_before_gate, activation)


def gated_rms_norm_quant(x, gate, weight, eps=1e-6, norm_group=0, norm_before_gate=True,
                         activation="silu", format="fp8", group_size=0):
    """:func:`gated_rms_norm` with its output in 8 bits, for a projection in 8
    bits: ``(q, scale)`` as :func:`rms_norm_quant` gives them, the scales over
    the whole row or 128 columns of it.  No autograd."""
    fmt, group = _format(format, group_size)
    c = _Gated(x, gate, weight, eps, norm_group, norm_before_gate, activation, fmt, group)
    q, scale = _eight_bits(x, c.p.D, format, group)
    _launch(x, lib.gdr_gated_norm_fwd, c.ref, _ptr(c.x), _ptr(c.gate), _ptr(c.weight), _ptr(q),
            _ptr(scale), None)
    return q, scale


# ---- the norms on both sides of a residual's addition ----------------------------

class _Sandwich:
    """The checked arguments of one sandwich norm call."""

    def __init__(self, x, post_weight, pre_weight, gate, residual_scale, activation, eps, res_dtype,
                 fmt=0, group=0):
        rows, D = _count(x)
        act = _activation(activation, False)
        _need_gpu("x", x)
        dt, dev = _code(x, "x"), x.device
        alpha = 1.0
        if residual_scale is not None and not isinstance(residual_scale, torch.Tensor):
            alpha, residual_scale = float(residual_scale), None
        self.pre = _like("pre_weight", pre_weight, (D,), (x.dtype, torch.float32), dev)
        self.post = _like("post_weight", post_weight, (D,), (pre_weight.dtype,), dev)
        self.scale = _like("residual_scale", residual_scale, (D,), (pre_weight.dtype,), dev)
        self.x, xs = _rows(x)
        self.gate, zs = None, D
        if gate is not None:
            _expect("gate", gate, x.shape, (x.dtype,), dev)
            self.gate, zs = _rows(gate)
        self.p = SandwichNormProblem(rows, D, dt, _DT.get(res_dtype, -1), _DT[pre_weight.dtype],
                                     act, fmt, group, float(eps), alpha, xs, zs)
        self.ref = ctypes.byref(self.p)

    def inputs(self):
        return _ptr(self.gate), _ptr(self.post), _ptr(self.scale), _ptr(self.pre)


def _sandwich_fwd(x, residual, post_weight, pre_weight, gate, residual_scale, activation, eps,
                  fmt=None, group_size=0, need_rstd=False):
    code, group = (0, 0) if fmt is None else _format(fmt, group_size)
    c = _Sandwich(x, post_weight, pre_weight, gate, residual_scale, activation, eps, residual.dtype,
                  code, group)
    residual = _like("residual", residual, x.shape, (x.dtype, torch.float32), x.device)
    h = torch.empty_like(residual)
    y, scale = (_new(x), None) if fmt is None else _eight_bits(x, c.p.D, fmt, group)
    rx = rh = None
    if need_rstd:
        rh = x.new_empty(x.shape[:-1], dtype=torch.float32)
        rx = None if post_weight is None else torch.empty_like(rh)
    _launch(x, lib.gdr_sandwich_norm_fwd, c.ref, _ptr(c.x), _ptr(residual), *c.inputs(), _ptr(y),
            _ptr(scale), _ptr(h), _ptr(rx), _ptr(rh))
    return y, scale, h, rx, rh


def sandwich_rms_norm_fwd(x, residual, post_weight, pre_weight, gate=None, residual_scale=None,
                          activation="sigmoid", eps=1e-6):
    """:func:`sandwich_rms_norm` without autograd: ``(y, h, rstd_x, rstd_h)``,
    the last two (fp32, one per row; ``rstd_x`` ``None`` without a post_weight) for
    :func:`sandwich_rms_norm_bwd`."""
    y, _, h, rx, rh = _sandwich_fwd(x, residual, post_weight, pre_weight, gate, residual_scale,
                                    activation, eps, need_rstd=True)
    return y, h, rx, rh


def sandwich_rms_norm_bwd(dy, dh, x, h, post_weight, pre_weight, rstd_x, rstd_h, gate=None,
                          residual_scale=None, activation="sigmoid"):
    """The gradient of :func:`sandwich_rms_norm`: ``(dx, dresidual, dpost_weight,
    dpre_weight, dgate, dresidual_scale)``, ``None`` in the place of an input that
    is ``None`` or a number.  ``h``, ``rstd_x`` and ``rstd_h`` come from
    :func:`sandwich_rms_norm_fwd`; ``dh`` (optional) is the gradient of ``h``."""
    c = _Sandwich(x, post_weight, pre_weight, gate, residual_scale, activation, 0.0, h.dtype)
    dev = x.device
    dy = _like("dy", dy, x.shape, (x.dtype,), dev)
    h = _like("h", h, x.shape, (x.dtype, torch.float32), dev)
    dh = _like("dh", dh, x.shape, (h.dtype,), dev)
    rstd_h = _like("rstd_h", rstd_h, x.shape[:-1], (torch.float32,), dev)
    if (rstd_x is None) != (post_weight is None):
        raise GdrError(10, "rstd_x comes with post_weight, and only then")
    rstd_x = _like("rstd_x", rstd_x, x.shape[:-1], (torch.float32,), dev)
    dx, dres = _new(x), _new(x, h.dtype)
    dgate = None if gate is None else _new(x)
    new = lambda t: None if t is None else torch.empty_like(t)  # noqa: E731
    dpost, dscale, dpre = new(c.post), new(c.scale), new(c.pre)
    n = lib.gdr_sandwich_norm_bwd_workspace_size(c.ref)
    ws = _bytes(n, dev)
    _launch(x, lib.gdr_sandwich_norm_bwd, c.ref, _ptr(dy), _ptr(dh), _ptr(c.x), _ptr(h), *c.inputs(),
            _ptr(rstd_x), _ptr(rstd_h), _ptr(dx), _ptr(dres), _ptr(dgate), _ptr(dpost), _ptr(dscale),
            _ptr(dpre), _ptr(ws), n)
    return dx, dres, dpost, dpre, dgate, dscale


class _SandwichRmsNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, post_weight, pre_weight, gate, residual_scale, activation, eps):
        ctx.set_materialize_grads(False)
        y, h, rx, rh = sandwich_rms_norm_fwd(x, residual, post_weight, pre_weight, gate,
                                             residual_scale, activation, eps)
        tensor = isinstance(residual_scale, torch.Tensor)
        ctx.save_for_backward(x, h, post_weight, pre_weight, rx, rh, gate,
                              residual_scale if tensor else None)
        ctx.number, ctx.activation = None if tensor else residual_scale, activation
        return y, h

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh):
        x, h, post, pre, rx, rh, gate, scale = ctx.saved_tensors
        if dy is None:
            dy = torch.zeros(x.shape, dtype=x.dtype, device=x.device)
        return sandwich_rms_norm_bwd(dy, dh, x, h, post, pre, rx, rh, gate,
                                     ctx.number if scale is None else scale,
                                     ctx.activation) + (None, None)


def sandwich_rms_norm(x, residual, post_weight, pre_weight, gate=None, residual_scale=None,
                      activation="sigmoid", eps=1e-6):
    """From a block's output to the next block's input, with autograd: ``(y,
    h)``.

    ``h = residual + residual_scale * act(gate) * n`` with ``n = post_weight * x / rms(x)``
    (x itself where ``post_weight`` is ``None``), rounded to the residual's dtype, and
    ``y = pre_weight * h / rms(h)`` of this rounded stream; ``rms(v) = sqrt(mean(v^2) +
    eps)``.  x ``[..., D]`` (bf16, fp16 or fp32), residual like it or in fp32;
    post_weight, pre_weight ``[D]`` in x's dtype or fp32, both in the same;
    ``gate`` (optional) like x, ``activation`` ``"sigmoid"``, ``"silu"`` or ``None``; x and
    gate may be slices of wider tensors; ``residual_scale`` (optional) a number or
    ``[D]`` in the weights' dtype; D up to 16384.  Gradients flow to every tensor,
    also from ``h``."""
    return _SandwichRmsNorm.apply(x, residual, post_weight, pre_weight, gate, residual_scale,
                                  activation, eps)


def sandwich_rms_norm_quant(x, residual, post_weight, pre_weight, gate=None, residual_scale=None,
                            activation="sigmoid", eps=1e-6, format="fp8", group_size=0):
    """:func:`sandwich_rms_norm` with y in 8 bits, for a projection in 8 bits:
    ``(q, scale, h)``, q and scale as :func:`rms_norm_quant` gives them.  No
    autograd."""
    if format is None:
        raise GdrError(10, "format must be 'fp8' or 'int8', got None")
    return _sandwich_fwd(x, residual, post_weight, pre_weight, gate, residual_scale, activation, eps,
                         format, group_size)[:3]


# ---- rows and products in 8 bits ---------------------------------------------------

def quantize_rows(x, format="int8", group_size=0):
    """Rows x ``[..., D]`` (bf16, fp16 or fp32; D up to 65536) in 8 bits with a
    scale per row or per 128 columns, ``(q, scale)`` as :func:`rms_norm_quant`
    gives them of its y: weights ``[N, K]`` for :func:`int8_matmul` as they are
    loaded, activations that come from no norm.  No autograd."""
    fmt, group = _format(format, group_size)
    rows, D = _count(x)
    _need_gpu("x", x)
    src, stride = _rows(x)
    p = QuantizeProblem(rows, D, _code(x, "x"), fmt, group, stride)
    q, scale = _eight_bits(x, D, format, group)
    _launch(x, lib.gdr_quantize_rows, ctypes.byref(p), _ptr(src), _ptr(q), _ptr(scale))
    return q, scale


def _scales(name, t, shape, device):
    """One fp32 scale for each row of shape, also with a last dimension of 1."""
    if t.dim() and t.shape == shape + (1,):
        t = t.squeeze(-1)
    return _like(name, t, shape, (torch.float32,), device)


def _moved(t):
    """A contiguous copy at an address of its own."""
    return t.clone(memory_format=torch.contiguous_format)


def int8_matmul(x, x_scale, weight, w_scale, bias=None, out_dtype=torch.bfloat16):
    """Product of 8-bit integers with a scale per token and per channel: y
    ``[..., N]`` in ``out_dtype`` (bf16, fp16 or fp32),
    ``y = x_scale * w_scale * (x @ weight.T) + bias``.

    x ``[..., K]`` int8 (a slice of a wider tensor is read in place) with
    ``x_scale`` ``x.shape[:-1]`` or ``x.shape[:-1] + (1,)`` fp32, as
    :func:`rms_norm_quant`, :func:`gated_rms_norm_quant`,
    :func:`sandwich_rms_norm_quant` and :func:`quantize_rows` give them with
    ``format="int8"``; weight ``[N, K]`` int8 with ``w_scale`` ``[N]`` or ``[N, 1]``; bias
    ``[N]`` in out_dtype or fp32; K up to 65536.  The sums over K are exact.  No
    autograd."""
    M, K = _count(x)
    if weight.dim() != 2:
        raise GdrError(2, "weight must be [N, K], got %s" % (tuple(weight.shape),))
    N = weight.shape[0]
    _fits("weight", N)
    if x.dtype != torch.int8:
        raise GdrError(4, "x must be torch.int8, got %s" % x.dtype)
    out = _DT.get(out_dtype)
    if out is None:
        raise GdrError(4, "out_dtype must be bf16, fp16 or fp32, got %s" % (out_dtype,))
    _need_gpu("x", x)
    dev, lead = x.device, x.shape[:-1]
    weight = _like("weight", weight, (N, K), (torch.int8,), dev)
    x_scale = _scales("x_scale", x_scale, lead, dev)
    w_scale = _scales("w_scale", w_scale, (N,), dev)
    bias = _like("bias", bias, (N,), (out_dtype, torch.float32), dev)
    src, stride = (x, K) if x.is_contiguous() else _rows(x)
    # a multiple of 16 bytes from row to row asks for such an address
    if stride > 1 << 22 or (K % 16 == 0 and stride % 16 == 0 and src.data_ptr() % 16):
        src, stride = _moved(src), K
    if K % 16 == 0 and weight.data_ptr() % 16:
        weight = _moved(weight)
    p = Int8MatmulProblem(M, N, K, out, out if bias is None else _DT[bias.dtype], stride)
    ref = ctypes.byref(p)
    n = lib.gdr_int8_matmul_workspace_size(ref) if (K | stride) % 16 else 0
    ws = _bytes(n, dev) if n else None
    y = x.new_empty(lead + (N,), dtype=out_dtype)
    _launch(x, lib.gdr_int8_matmul, ref, _ptr(src), _ptr(x_scale), _ptr(weight), _ptr(w_scale),
            _ptr(bias), _ptr(y), _ptr(ws), n)
    return y
