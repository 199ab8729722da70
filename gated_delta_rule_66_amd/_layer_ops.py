"""The operators around the recurrence in a layer: the short causal
convolution, the selective state space scan and the RMS norm with the
residual's addition.

Thin bindings over libgdr.so, re-exported by the package: PyTorch provides
device memory, the current stream and autograd; every computation runs in the
library's HIP kernels.  Errors are :class:`GdrError`, as everywhere in the
package.
"""
from __future__ import annotations

import ctypes

import torch
from torch.autograd.function import once_differentiable

from ._lib import (GDR_BF16, GDR_FP16, GDR_FP32, ConvProblem, GdrError, NormProblem, SsmProblem, check,
                   lib)

_DT = {torch.bfloat16: GDR_BF16, torch.float16: GDR_FP16, torch.float32: GDR_FP32}


def _ptr(t):
    return None if t is None else t.data_ptr()


def _code(t, name):
    try:
        return _DT[t.dtype]
    except KeyError:
        raise GdrError(4, "%s has the unsupported dtype %s" % (name, t.dtype)) from None


# the current device and the current stream's handle without objects around
# them: a fifth of a small call's time on the host otherwise
_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda i: torch.cuda.current_stream(i).cuda_stream)


def _launch(t, f, *args):
    """f on t's device, which is made the current one, and its current stream."""
    i = t.get_device()
    if i == _device():
        status = f(*args, _raw_stream(i))
    else:
        with torch.cuda.device(i):
            status = f(*args, _raw_stream(i))
    check(status)


def _new(t, dtype=None):
    """A new contiguous tensor of t's shape and device (t's dtype by default)."""
    if t.is_contiguous():
        return torch.empty_like(t, dtype=dtype)
    return t.new_empty(t.shape, dtype=dtype)


def _fits(name, *sizes):
    """The library takes sizes in 32 bits, and a conversion would drop the
    higher ones without a word: a size that does not fit is refused here."""
    if max(sizes) >= 1 << 31:
        raise GdrError(2, "%s has a size that does not fit 32 bits: %s" % (name, sizes))


def _need_gpu(name, t):
    if not t.is_cuda:
        raise GdrError(8, "%s is on %s; the kernels run on an MI355X" % (name, t.device))


def _expect(name, t, shape, dtypes, device):
    """t must have this shape, one of these dtypes and this device."""
    if t.shape == shape and t.dtype in dtypes and t.device == device:
        return
    if tuple(t.shape) != tuple(shape):
        raise GdrError(2, "%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if t.dtype not in dtypes:
        raise GdrError(4, "%s must be %s, got %s"
                       % (name, " or ".join(str(d) for d in dtypes), t.dtype))
    if t.device != device:
        raise GdrError(8, "%s is on %s but x is on %s" % (name, t.device, device))


def _like(name, t, shape, dtypes, device):
    """:func:`_expect` (None passes), and t contiguous."""
    if t is None:
        return None
    if t.shape != shape or t.dtype not in dtypes or t.device != device:
        _expect(name, t, shape, dtypes, device)
    return t if t.is_contiguous() else t.contiguous()


def _token_rows(x, inner, most=1 << 62):
    """(x, stride): x [B, T, ...] as rows one token stride (at most `most`)
    apart, the last `inner` dimensions contiguous; copied only when it is not
    laid out so."""
    if x.is_contiguous():
        shape = x.shape
        return x, shape[2] if inner == 1 else shape[2] * shape[3]
    B, T = x.shape[0], x.shape[1]
    width = 1
    ok = True
    for d in range(1, inner + 1):
        if x.shape[-d] != 1 and x.stride(-d) != width:
            ok = False
        width *= x.shape[-d]
    if ok:
        s = x.stride(1) if T > 1 else (x.stride(0) if B > 1 else width)
        if width <= s <= most and (B == 1 or T == 1 or x.stride(0) == T * s):
            return x, s
    return x.contiguous(), width


def _seqs(x, cu_seqlens, cu_seqlens_cpu):
    """(N, device offsets, host offsets) of packed sequences, or (B, None, None)."""
    if cu_seqlens is None:
        if cu_seqlens_cpu is not None:
            raise GdrError(6, "cu_seqlens_cpu is given without cu_seqlens")
        return x.shape[0], None, None
    if cu_seqlens_cpu is None:
        # one blocking device-to-host copy (pass cu_seqlens_cpu to avoid it)
        cu_seqlens_cpu = cu_seqlens.detach().to("cpu")
    for t in (cu_seqlens, cu_seqlens_cpu):
        if t.dtype.is_floating_point or t.dtype.is_complex or t.dtype == torch.bool:
            raise GdrError(6, "cu_seqlens must hold integers, got %s" % t.dtype)
    wide = cu_seqlens_cpu.to(device="cpu")
    host = wide.to(torch.int32).contiguous()
    if wide.dtype != torch.int32 and not torch.equal(host.to(wide.dtype), wide):
        raise GdrError(6, "cu_seqlens has offsets that do not fit 32 bits")
    dev = cu_seqlens.to(device=x.device, dtype=torch.int32).contiguous()
    if host.dim() != 1 or host.numel() < 2 or dev.shape != host.shape:
        raise GdrError(6, "cu_seqlens needs one offset per sequence and the end, got shape %s"
                       % (tuple(host.shape),))
    return host.numel() - 1, dev, host


_written = torch.autograd.graph.increment_version


def _in_place(name, t):
    """t is written through its pointer, unseen by autograd: no gradient can
    pass the update (the caller then tells autograd of it: _written)."""
    if t.requires_grad and torch.is_grad_enabled():
        raise GdrError(10, "%s requires grad and is updated in place; no gradient passes the update "
                           "(detach it, or call this under torch.no_grad())" % name)


def _bytes(n, device):
    return torch.empty(max(n, 1), dtype=torch.uint8, device=device)


# ---- short causal convolution -------------------------------------------------

def _activation(name):
    if name in (None, "none"):
        return 0
    if name in ("silu", "swish"):
        return 1
    raise GdrError(10, "activation must be None or 'silu', got %r" % (name,))


class _Conv:
    """The checked arguments of one convolution call."""

    def __init__(self, x, weight, bias, activation, state, cu_seqlens, cu_seqlens_cpu):
        if x.dim() != 3 or weight.dim() != 2:
            raise GdrError(2, "x must be [B, T, D] and weight [D, W], got %s and %s"
                           % (tuple(x.shape), tuple(weight.shape)))
        B, T, D = x.shape
        W = weight.shape[1]
        _fits("x or weight", B, T, D, W)
        _need_gpu("x", x)
        dev = x.device
        dt = _code(x, "x")
        self.weight = _like("weight", weight, (D, W), (x.dtype, torch.float32), dev)
        self.bias = _like("bias", bias, (D,), (weight.dtype,), dev)
        N, self.cu, self.cu_host = _seqs(x, cu_seqlens, cu_seqlens_cpu)
        self.state_shape = (N, W - 1, D)
        self.state = _like("initial_state", state, self.state_shape, (x.dtype,), dev)
        self.x, stride = _token_rows(x, 1)
        self.p = ConvProblem(B, T, D, W, N, _ptr(self.cu), _ptr(self.cu_host), dt,
                             _code(weight, "weight"), _activation(activation), stride)
        self.ref = ctypes.byref(self.p)   # the library checks the problem in every call


def causal_conv1d_fwd(x, weight, bias=None, activation="silu", initial_state=None,
                      output_final_state=True, cu_seqlens=None, cu_seqlens_cpu=None):
    """:func:`causal_conv1d` without autograd: ``(y, final_state)``."""
    c = _Conv(x, weight, bias, activation, initial_state, cu_seqlens, cu_seqlens_cpu)
    y = _new(x)
    last = None
    if output_final_state:
        last = x.new_empty(c.state_shape)
    _launch(x, lib.gdr_conv1d_fwd, c.ref, _ptr(c.x), _ptr(c.weight), _ptr(c.bias), _ptr(c.state),
            _ptr(y), _ptr(last))
    return y, last


def causal_conv1d_bwd(x, weight, bias, dy, dfinal_state=None, activation="silu",
                      initial_state=None, cu_seqlens=None, cu_seqlens_cpu=None):
    """The gradient of :func:`causal_conv1d`: ``(dx, dweight, dbias,
    dinitial_state)``, the last two ``None`` without a bias or an initial
    state.  ``dfinal_state`` (optional) is the gradient of the final state."""
    c = _Conv(x, weight, bias, activation, initial_state, cu_seqlens, cu_seqlens_cpu)
    dev = x.device
    dy = _like("dy", dy, x.shape, (x.dtype,), dev)
    dfinal_state = _like("dfinal_state", dfinal_state, c.state_shape, (x.dtype,), dev)
    dx = _new(x)
    dw = torch.empty_like(c.weight)
    db = None if bias is None else torch.empty_like(c.bias)
    ds = None if c.state is None else torch.empty_like(c.state)
    n = lib.gdr_conv1d_bwd_workspace_size(c.ref)
    ws = _bytes(n, dev)
    _launch(x, lib.gdr_conv1d_bwd, c.ref, _ptr(c.x), _ptr(c.weight), _ptr(c.bias), _ptr(dy),
            _ptr(dfinal_state), _ptr(c.state), _ptr(dx), _ptr(dw), _ptr(db), _ptr(ds), _ptr(ws), n)
    return dx, dw, db, ds


class _CausalConv1d(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, activation, initial_state, output_final_state, cu_seqlens,
                cu_seqlens_cpu):
        ctx.set_materialize_grads(False)
        if cu_seqlens is not None and cu_seqlens_cpu is None:
            cu_seqlens_cpu = cu_seqlens.detach().to("cpu")
        y, last = causal_conv1d_fwd(x, weight, bias, activation, initial_state,
                                    output_final_state, cu_seqlens, cu_seqlens_cpu)
        ctx.save_for_backward(x, weight, bias, initial_state, cu_seqlens, cu_seqlens_cpu)
        ctx.activation = activation
        return y, last

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dlast):
        x, weight, bias, state, cu, cu_cpu = ctx.saved_tensors
        if dy is None:
            dy = torch.zeros(x.shape, dtype=x.dtype, device=x.device)
        dx, dw, db, ds = causal_conv1d_bwd(x, weight, bias, dy, dlast, ctx.activation, state, cu,
                                           cu_cpu)
        return dx, dw, db, None, ds, None, None, None


def causal_conv1d(x, weight, bias=None, activation="silu", initial_state=None,
                  output_final_state=False, cu_seqlens=None, cu_seqlens_cpu=None):
    """Short causal depthwise convolution with autograd: ``(y, final_state)``.

    ``y[t] = act(bias + sum_j weight[:, j] * x[t - (W-1) + j])`` per channel,
    ``W`` = 2, 3 or 4, ``activation`` ``"silu"`` or ``None``.  x ``[B, T, D]``
    (bf16, fp16 or fp32; a slice of a wider projection is read in place);
    weight ``[D, W]`` and bias ``[D]`` in x's dtype or fp32.  States ``[N, W-1,
    D]`` in x's dtype hold the last ``W-1`` inputs, oldest first; without
    ``initial_state`` what precedes a sequence is zero.  ``cu_seqlens``: packed
    sequences (``B == 1``), ``N = len(cu_seqlens) - 1``; sequences may be empty.
    Gradients flow to x, weight, bias and initial_state."""
    return _CausalConv1d.apply(x, weight, bias, activation, initial_state,
                               bool(output_final_state), cu_seqlens, cu_seqlens_cpu)


def causal_conv1d_update(x, conv_state, weight, bias=None, activation="silu"):
    """One or a few tokens per sequence on a cached state (decode): returns y,
    shaped like x (``[B, D]`` or ``[B, T, D]``), and updates ``conv_state``
    ``[B, W-1, D]`` in place.  No autograd: a graph that saved ``conv_state``
    raises in its backward, as after any in-place operation, and a
    ``conv_state`` that requires grad is refused while grad mode is on."""
    squeeze = x.dim() == 2
    x3 = x.unsqueeze(1) if squeeze else x
    if not conv_state.is_contiguous():
        raise GdrError(10, "conv_state is updated in place and must be contiguous")
    _in_place("conv_state", conv_state)
    c = _Conv(x3, weight, bias, activation, conv_state, None, None)
    y = _new(x3)
    _launch(x, lib.gdr_conv1d_update, c.ref, _ptr(c.x), _ptr(conv_state), _ptr(c.weight),
            _ptr(c.bias), _ptr(y))
    _written(conv_state)
    return y.squeeze(1) if squeeze else y


# ---- selective state space scan --------------------------------------------------

class _Ssm:
    """The checked arguments of one scan call."""

    def __init__(self, x, dt, A_log, B, C, D, dt_bias, dt_softplus, state, cu_seqlens,
                 cu_seqlens_cpu, keep_states=False):
        if x.dim() != 4 or B.dim() != 4:
            raise GdrError(2, "x must be [B, T, H, V] and B [B, T, G, K], got %s and %s"
                           % (tuple(x.shape), tuple(B.shape)))
        b, T, H, V = x.shape
        G, K = B.shape[2], B.shape[3]
        _fits("x or B", b, T, H, V, G, K)
        _need_gpu("x", x)
        dev = x.device
        code = _code(x, "x")
        _expect("B", B, (b, T, G, K), (x.dtype,), dev)
        _expect("C", C, (b, T, G, K), (x.dtype,), dev)
        self.dt = _like("dt", dt, (b, T, H), (x.dtype, torch.float32), dev)
        self.A_log = _like("A_log", A_log, (H,), (x.dtype, torch.float32), dev)
        self.D = _like("D", D, (H,), (A_log.dtype,), dev)
        self.dt_bias = _like("dt_bias", dt_bias, (H,), (A_log.dtype,), dev)
        N, self.cu, self.cu_host = _seqs(x, cu_seqlens, cu_seqlens_cpu)
        self.state_shape = (N, H, K, V)
        self.state = _aligned(_like("initial_state", state, self.state_shape, (torch.float32,), dev))
        self.x, xs = _token_rows(x, 2, 1 << 23)
        self.B, bs = _token_rows(B, 2, 1 << 23)
        self.C, cs = _token_rows(C, 2, 1 << 23)
        self.p = SsmProblem(b, T, H, G, K, V, N, _ptr(self.cu), _ptr(self.cu_host), code,
                            _DT[dt.dtype], _DT[A_log.dtype], 1 if dt_softplus else 0,
                            1 if keep_states else 0, xs, bs, cs)
        self.ref = ctypes.byref(self.p)

    def inputs(self):
        return (_ptr(self.x), _ptr(self.dt), _ptr(self.A_log), _ptr(self.B), _ptr(self.C),
                _ptr(self.D), _ptr(self.dt_bias))


def _aligned(t):
    """States are read 16 bytes at a time."""
    return t if t is None or t.data_ptr() % 16 == 0 else t.clone()


def _scan_fwd(x, dt, A_log, B, C, D, dt_bias, dt_softplus, initial_state, output_final_state,
              cu_seqlens, cu_seqlens_cpu, keep_states):
    c = _Ssm(x, dt, A_log, B, C, D, dt_bias, dt_softplus, initial_state, cu_seqlens,
             cu_seqlens_cpu, keep_states)
    y = _new(x)
    last = None
    if output_final_state:
        last = x.new_empty(c.state_shape, dtype=torch.float32)
    n = lib.gdr_ssm_fwd_workspace_size(c.ref)
    ws = _bytes(n, x.device) if n else None
    _launch(x, lib.gdr_ssm_fwd, c.ref, *c.inputs(), _ptr(c.state), _ptr(y), _ptr(last), _ptr(ws), n)
    return y, last, ws


def _scan_bwd(x, dt, A_log, B, C, dy, D, dt_bias, dt_softplus, dht, initial_state, cu_seqlens,
              cu_seqlens_cpu, keep_states, kept):
    c = _Ssm(x, dt, A_log, B, C, D, dt_bias, dt_softplus, initial_state, cu_seqlens,
             cu_seqlens_cpu, keep_states)
    dev = x.device
    dy = _like("dy", dy, x.shape, (x.dtype,), dev)
    dht = _aligned(_like("dht", dht, c.state_shape, (torch.float32,), dev))
    new = lambda t: None if t is None else _new(t)  # noqa: E731
    dx, ddt, dA, dB, dC, dD, db, dh0 = (new(t) for t in (x, dt, A_log, B, C, D, dt_bias,
                                                         initial_state))
    n = lib.gdr_ssm_bwd_workspace_size(c.ref)
    ws = _bytes(n, dev)
    _launch(x, lib.gdr_ssm_bwd, c.ref, *c.inputs(), _ptr(dy), _ptr(dht), _ptr(c.state), _ptr(kept),
            _ptr(dx), _ptr(ddt), _ptr(dA), _ptr(dB), _ptr(dC), _ptr(dD), _ptr(db), _ptr(dh0),
            _ptr(ws), n)
    return dx, ddt, dA, dB, dC, dD, db, dh0


def chunk_selective_scan_fwd(x, dt, A_log, B, C, D=None, dt_bias=None, dt_softplus=True,
                             initial_state=None, output_final_state=True, cu_seqlens=None,
                             cu_seqlens_cpu=None):
    """:func:`chunk_selective_scan` without autograd: ``(y, final_state)``."""
    return _scan_fwd(x, dt, A_log, B, C, D, dt_bias, dt_softplus, initial_state,
                     output_final_state, cu_seqlens, cu_seqlens_cpu, False)[:2]


def chunk_selective_scan_bwd(x, dt, A_log, B, C, dy, D=None, dt_bias=None, dt_softplus=True,
                             dht=None, initial_state=None, cu_seqlens=None, cu_seqlens_cpu=None):
    """The gradient of :func:`chunk_selective_scan`: ``(dx, ddt, dA_log, dB, dC,
    dD, ddt_bias, dh0)``, ``None`` in the place of an input that is ``None``.
    ``dht`` (optional) is the gradient of the final state."""
    return _scan_bwd(x, dt, A_log, B, C, dy, D, dt_bias, dt_softplus, dht, initial_state,
                     cu_seqlens, cu_seqlens_cpu, False, None)


class _SelectiveScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, dt, A_log, B, C, D, dt_bias, dt_softplus, initial_state,
                output_final_state, cu_seqlens, cu_seqlens_cpu, keep):
        ctx.set_materialize_grads(False)
        if cu_seqlens is not None and cu_seqlens_cpu is None:
            cu_seqlens_cpu = cu_seqlens.detach().to("cpu")
        ctx.keep = keep and any(ctx.needs_input_grad)
        y, last, kept = _scan_fwd(x, dt, A_log, B, C, D, dt_bias, dt_softplus, initial_state,
                                  output_final_state, cu_seqlens, cu_seqlens_cpu, ctx.keep)
        ctx.save_for_backward(x, dt, A_log, B, C, D, dt_bias, initial_state, cu_seqlens,
                              cu_seqlens_cpu, kept if ctx.keep else None)
        ctx.dt_softplus = dt_softplus
        return y, last

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dlast):
        x, dt, A_log, B, C, D, dt_bias, state, cu, cu_cpu, kept = ctx.saved_tensors
        if dy is None:
            dy = torch.zeros(x.shape, dtype=x.dtype, device=x.device)
        dx, ddt, dA, dB, dC, dD, db, dh0 = _scan_bwd(
            x, dt, A_log, B, C, dy, D, dt_bias, ctx.dt_softplus, dlast, state, cu, cu_cpu,
            ctx.keep, kept)
        return dx, ddt, dA, dB, dC, dD, db, None, dh0, None, None, None, None


def chunk_selective_scan(x, dt, A_log, B, C, D=None, dt_bias=None, dt_softplus=True,
                         initial_state=None, output_final_state=False, cu_seqlens=None,
                         cu_seqlens_cpu=None, recompute_states=False):
    """Selective state space scan (one decay per head) with autograd: ``(y,
    final_state)``.

    Per head with state S ``[K, V]``: ``S_t = exp(-exp(A_log) dt_t) S_{t-1} + dt_t
    B_t x_t^T`` and ``y_t = S_t^T C_t + D x_t``, ``dt_t = softplus(dt + dt_bias)`` (the
    sum itself with ``dt_softplus=False``): the recurrence of Mamba-2 layers, the
    gated delta rule's gate without its delta term.  x ``[B, T, H, V]``, B and C
    ``[B, T, G, K]`` in bf16 or fp16 (slices of one projection are read in
    place), H a multiple of G, K and V 64 or 128; dt ``[B, T, H]`` in x's dtype or
    fp32; A_log, D, dt_bias ``[H]`` in x's dtype or fp32; states ``[N, H, K, V]``
    fp32.  ``cu_seqlens``: packed sequences (``B == 1``), which may be empty.
    Gradients flow to every tensor; for them the forward keeps its inputs and the
    fp32 states between the segments that it cut long sequences into (K * V * 4
    bytes per segment and head); ``recompute_states=True`` keeps only the inputs
    and recomputes the states in the backward instead."""
    return _SelectiveScan.apply(x, dt, A_log, B, C, D, dt_bias, bool(dt_softplus), initial_state,
                                bool(output_final_state), cu_seqlens, cu_seqlens_cpu,
                                torch.is_grad_enabled() and not recompute_states)


def fused_recurrent_selective_scan(x, dt, A_log, B, C, D=None, dt_bias=None, dt_softplus=True,
                                   initial_state=None, output_final_state=True, cu_seqlens=None,
                                   cu_seqlens_cpu=None, inplace_final_state=False):
    """The scan one token at a time (decode steps, a few speculative tokens):
    ``(y, final_state)`` of :func:`chunk_selective_scan`, the state read once
    and written once.  With ``inplace_final_state`` the fp32 ``initial_state``
    is updated in place and returned (a graph that saved it raises in its
    backward, as after any in-place operation, and one that requires grad is
    refused while grad mode is on).  No autograd."""
    if inplace_final_state and (initial_state is None or not initial_state.is_contiguous()
                                or initial_state.data_ptr() % 16):
        raise GdrError(10, "inplace_final_state needs a contiguous, 16-byte aligned initial_state")
    if inplace_final_state:
        _in_place("initial_state", initial_state)
    c = _Ssm(x, dt, A_log, B, C, D, dt_bias, dt_softplus, initial_state, cu_seqlens,
             cu_seqlens_cpu)
    y = _new(x)
    last = None
    if inplace_final_state:
        last = initial_state
    elif output_final_state:
        last = x.new_empty(c.state_shape, dtype=torch.float32)
    _launch(x, lib.gdr_ssm_step, c.ref, *c.inputs(), _ptr(c.state), _ptr(y), _ptr(last))
    if inplace_final_state:
        _written(last)
    return y, last


# ---- RMS norm with the residual's addition ----------------------------------------

_FORMATS = {None: 0, "fp8": 1, "int8": 2}
_QUANTISED = {"fp8": torch.float8_e4m3fn, "int8": torch.int8}


class _Norm:
    """The checked arguments of one norm call on rows of D columns."""

    def __init__(self, x, weight, eps, res_dtype, fmt=None, group_size=0):
        if x.dim() < 1 or weight.dim() != 1:
            raise GdrError(2, "x must be [..., D] and weight [D], got %s and %s"
                           % (tuple(x.shape), tuple(weight.shape)))
        D = x.shape[-1]
        rows = x.numel() // D if D else 0
        _fits("x", rows, D)
        if fmt not in _FORMATS:
            raise GdrError(10, "format must be 'fp8' or 'int8', got %r" % (fmt,))
        # the number of scales follows from it before the library sees it
        if group_size not in (0, 128):
            raise GdrError(10, "group_size must be 0 (the row) or 128, got %r" % (group_size,))
        _need_gpu("x", x)
        dt = _code(x, "x")
        self.weight = _like("weight", weight, (D,), (x.dtype, torch.float32), x.device)
        # rows one stride apart (a slice of a wider tensor), else a copy
        stride = D
        if x.dim() == 1 or x.is_contiguous():
            x = x if x.is_contiguous() else x.contiguous()
        else:
            flat = x.unsqueeze(0) if x.dim() == 2 else x.flatten(0, -3) if x.dim() > 3 else x
            x, stride = _token_rows(flat, 1)
        self.x = x
        self.p = NormProblem(rows, D, dt, dt if res_dtype is None else _DT.get(res_dtype, -1),
                             _code(weight, "weight"), 0 if res_dtype is None else 1, _FORMATS[fmt],
                             int(group_size), float(eps), stride)
        self.ref = ctypes.byref(self.p)


def _norm_fwd(x, weight, eps, residual, fmt, group_size, need_rstd):
    c = _Norm(x, weight, eps, None if residual is None else residual.dtype, fmt, group_size)
    dev = x.device
    residual = _like("residual", residual, x.shape, (x.dtype, torch.float32), dev)
    D = x.shape[-1]
    h = None if residual is None else torch.empty_like(residual)
    y = _new(x, _QUANTISED.get(fmt))
    scale = None
    if fmt is not None:
        groups = 1 if group_size == 0 else -(-D // group_size)
        scale = x.new_empty(x.shape[:-1] + (groups,), dtype=torch.float32)
    rstd = x.new_empty(x.shape[:-1], dtype=torch.float32) if need_rstd else None
    _launch(x, lib.gdr_rms_norm_fwd, c.ref, _ptr(c.x), _ptr(residual), _ptr(c.weight), _ptr(y),
            _ptr(scale), _ptr(h), _ptr(rstd))
    return y, scale, h, rstd


def rms_norm_fwd(x, weight, eps=1e-6, residual=None):
    """:func:`rms_norm` without autograd: ``(y, h, rstd)``, ``h`` ``None``
    without a residual, ``rstd`` (fp32, one per row) for :func:`rms_norm_bwd`."""
    y, _, h, rstd = _norm_fwd(x, weight, eps, residual, None, 0, True)
    return y, h, rstd


def rms_norm_bwd(dy, h, weight, rstd, dh=None, has_residual=False):
    """The gradient of :func:`rms_norm`: ``(dx, dresidual, dweight)``.  ``h`` is
    what the forward normalised (its ``h`` with a residual, else x), ``dh``
    (optional, with a residual) the gradient of the ``h`` it returned.
    ``dresidual`` is ``None`` without a residual; of one dtype, x and the
    residual have the same gradient and get the same tensor."""
    if dh is not None and not has_residual:
        raise GdrError(10, "dh is the gradient of h, which only a residual brings")
    _need_gpu("h", h)
    if has_residual:
        c = _Norm(dy, weight, 0.0, h.dtype)
        stream, stride = h.contiguous(), h.shape[-1]
    else:
        c = _Norm(h, weight, 0.0, None)
        stream, stride = c.x, c.p.x_stride
    dev = dy.device
    c.p.x_stride = stride
    _expect("h", h, dy.shape, (dy.dtype, torch.float32) if has_residual else (dy.dtype,), dev)
    dy = dy.contiguous()
    rstd = _like("rstd", rstd, dy.shape[:-1], (torch.float32,), dev)
    dh = _like("dh", dh, dy.shape, (h.dtype,), dev)
    dx = torch.empty_like(dy)
    dres = None
    if has_residual and h.dtype != dy.dtype:
        dres = _new(dy, h.dtype)
    dw = torch.empty_like(c.weight)
    n = lib.gdr_rms_norm_bwd_workspace_size(c.ref)
    ws = _bytes(n, dev)
    _launch(dy, lib.gdr_rms_norm_bwd, c.ref, _ptr(dy), _ptr(stream), _ptr(c.weight), _ptr(rstd),
            _ptr(dh), _ptr(dx), _ptr(dres), _ptr(dw), _ptr(ws), n)
    if not has_residual:
        return dx, None, dw
    return dx, dx if dres is None else dres, dw


class _RmsNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, eps, residual):
        ctx.set_materialize_grads(False)
        y, h, rstd = rms_norm_fwd(x, weight, eps, residual)
        ctx.save_for_backward(x if h is None else h, weight, rstd)
        ctx.has_residual, ctx.dtype = h is not None, x.dtype
        return (y, h) if h is not None else y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh=None):
        h, weight, rstd = ctx.saved_tensors
        if dy is None:
            dy = torch.zeros(h.shape, dtype=ctx.dtype, device=h.device)
        dx, dres, dw = rms_norm_bwd(dy, h, weight, rstd, dh, ctx.has_residual)
        return dx, dw, None, dres


def rms_norm(x, weight, eps=1e-6, residual=None):
    """Root-mean-square norm over the last dimension, with autograd:
    ``weight * h / sqrt(mean(h^2) + eps)`` with ``h = x + residual``.

    Returns y in x's dtype, or ``(y, h)`` with a residual: ``h``, rounded to the
    residual's dtype (x's or fp32), is the stream that the next layer adds to,
    and it is this rounded stream that is normalised.  weight ``[D]`` in x's
    dtype or fp32; D up to 65536.  Gradients flow to x, weight and residual,
    also from ``h``."""
    return _RmsNorm.apply(x, weight, eps, residual)


def rms_norm_quant(x, weight, eps=1e-6, residual=None, format="fp8", group_size=0):
    """:func:`rms_norm` with its output in 8 bits, for a projection in 8 bits:
    ``(q, scale, h)``.  ``format`` ``"fp8"`` (e4m3, largest 448) or ``"int8"``;
    fp32 scales of shape ``x.shape[:-1] + (groups,)``, one per row (``group_size=0``,
    one group) or one per 128 columns (``group_size=128``, ``ceil(D / 128)``):
    ``scale = max(max|y| / top, 2**-126)`` and q the fp32 quotient ``y / scale``
    rounded to nearest even.  ``h`` is ``None`` without a residual.  No autograd."""
    if format is None:
        raise GdrError(10, "format must be 'fp8' or 'int8', got None")
    q, scale, h, _ = _norm_fwd(x, weight, eps, residual, format, group_size, False)
    return q, scale, h
