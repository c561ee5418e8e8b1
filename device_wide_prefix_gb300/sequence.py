"""Sequence operators of libdwp.so: the causal convolution, the selective
state space scan and the block norm (include/dwp.h, "Sequence operators").

Rows are tokens.  A tensor of rows is (batch, rows, channels), or (rows,
channels) for one packed stream: cut by CSR `offsets` into segments, or one
sequence without them.  Channels are contiguous; batch and row strides are
free, so views of a wider projection need no copy.

These helpers marshal arguments and allocate outputs and scratch, as the
others of the package do; allocations belong to the stream the call runs on.
Parameters (weight, bias, A, D, ...) and their gradients are described at
each function; gradients of parameters are float32.
"""
from __future__ import annotations

import ctypes
import struct

import torch

import device_wide_prefix_gb300 as _dwp

DWP_F32, DWP_BF16, DWP_F16 = 0, 1, 2
CHECKPOINT_ROWS = 16  # DWP_SCAN_CHECKPOINT_ROWS
NORM_MAX_GROUP = 16384  # DWP_NORM_MAX_GROUP

_DTYPES = {torch.float32: DWP_F32, torch.bfloat16: DWP_BF16, torch.float16: DWP_F16}
_NO_ROWS = (0, 0, 0)

# Every field of the argument structures is 8 bytes wide.
_CONV = "8q 3q 3q 5q"
_CONV_BACKWARD = _CONV + " 3q 3q 4q"
_CONV_STEP = "7q 3q 3q 5q"
_SCAN = "8q 18q 2q 3q 4q"
_SCAN_BACKWARD = _SCAN + " 3q 10q"
_SCAN_STEP = "7q 18q 2q 3q 3q"
_NORM = "7q d 15q 2q"
_NORM_BACKWARD = _NORM + " 15q 2q"
_PACK = {name: struct.Struct("=" + fmt.replace(" ", "")).pack for name, fmt in (
    ("dwp_causal_conv", _CONV), ("dwp_causal_conv_backward", _CONV_BACKWARD),
    ("dwp_causal_conv_step", _CONV_STEP), ("dwp_selective_scan", _SCAN),
    ("dwp_selective_scan_backward", _SCAN_BACKWARD), ("dwp_selective_scan_step", _SCAN_STEP),
    ("dwp_block_norm", _NORM), ("dwp_block_norm_backward", _NORM_BACKWARD))}
_WITH_SCRATCH = ("dwp_causal_conv_backward", "dwp_selective_scan", "dwp_selective_scan_backward",
                 "dwp_block_norm_backward")


_ENTRY = {}  # entry points by name, once the library is loaded


def _entry(name):
    f = _ENTRY.get(name)
    if f is None:
        f = _ENTRY[name] = getattr(_dwp.load(), name)
    return f


def scratch_bytes(name: str, packed: bytes) -> int:
    """Scratch a call needs, for its packed argument structure."""
    need = ctypes.c_size_t(0)
    _dwp._check(_entry(name)(packed, None, ctypes.byref(need), None), name)
    return need.value


def _launch(name, fields, x, stream, scratch=None):
    index = x.get_device()
    if index != torch._C._cuda_getDevice():
        with torch.cuda.device(index):
            return _launch(name, fields, x, stream, scratch)
    packed = _PACK[name](*fields)
    handle = torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream
    if name in _WITH_SCRATCH:
        size = ctypes.c_size_t(0)
        at = ctypes.byref(size)
        if scratch is None:
            st = _entry(name)(packed, None, at, None)
            if st:
                _dwp._check(st, name)
            scratch = _empty((size.value,), torch.uint8, x, stream)
        elif scratch.get_device() != index or not scratch.is_contiguous():
            _refuse("scratch must be a contiguous CUDA tensor on the inputs' device")
        size.value = scratch.numel() * scratch.element_size()
        st = _entry(name)(packed, scratch.data_ptr(), at, handle)
    else:
        st = _entry(name)(packed, handle)
    if st:
        _dwp._check(st, name)


def _empty(shape, dtype, x, stream):
    """Memory on x's device that belongs to the stream the call runs on."""
    if stream is None:  # torch.empty: half of new_empty's time on the host
        return torch.empty(shape, dtype=dtype, device=x.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=x.device)


def _refuse(what, *about):
    raise ValueError(what % about)


def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _main(x, what, ndims=(2, 3)):
    """Rows of the tensor that sets a call's type, device and row shape."""
    if not x.is_cuda or x.dtype not in _DTYPES or x.dim() not in ndims:
        _refuse("%s must be a CUDA tensor of float32, bfloat16 or float16 rows", what)
    return _rows(x, what)


def _rows(t, what):
    """(address, batch stride, row stride) of a tensor of rows."""
    s = t.stride()
    if s[-1] != 1 and t.shape[-1] > 1 and t.numel():
        _refuse("%s must have contiguous channels", what)
    return (t.data_ptr(), s[0], s[1]) if len(s) == 3 else (t.data_ptr(), 0, s[0])


def _like(t, x, what):
    """Rows of a tensor of the shape, type and device of x; zeros for None."""
    if t is None:
        return _NO_ROWS
    if t.shape != x.shape or t.dtype != x.dtype or t.get_device() != x.get_device():
        _refuse("%s must have the shape, type and device of the call's main input", what)
    return _rows(t, what)


def _dense(t, shape, dtype, x, what):
    """Address of a contiguous tensor on x's device; 0 for None."""
    if t is None:
        return 0
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous() or t.get_device() != x.get_device():
        _refuse("%s must be a contiguous %s tensor of shape %s on %s", what, dtype, tuple(shape), x.device)
    return t.data_ptr()


def _sequences(x, offsets):
    """(batch, rows, offsets' address, segments, sequences)."""
    if offsets is not None:
        if (x.dim() != 2 or offsets.get_device() != x.get_device() or offsets.dim() != 1 or offsets.numel() < 1
                or not offsets.is_contiguous() or offsets.element_size() != 4 or offsets.is_floating_point()):
            _refuse("offsets must be a contiguous CUDA tensor of 4-byte integers, for packed (rows, channels) inputs")
        n = offsets.numel() - 1
        return 1, x.shape[0], offsets.data_ptr(), n, n
    return (1, x.shape[0], 0, 0, 1) if x.dim() == 2 else (x.shape[0], x.shape[1], 0, 0, x.shape[0])


def _weight(weight, x, shape, what):
    if weight.dtype != x.dtype and weight.dtype != torch.float32:
        _refuse("%s must be float32 or of x's type", what)
    return _dense(weight, shape, weight.dtype, x, what)


def _output(out, x, stream, what="out"):
    if out is None:
        return _empty(x.shape, x.dtype, x, stream)
    _like(out, x, what)
    return out


# ---------------------------------------------------------------------------
# causal convolution


def _conv_fields(x, xr, out, weight, bias, offsets, initial_state, final_state, silu):
    _need(weight.dim() == 2 and weight.shape[0] == x.shape[-1], "weight must have shape (channels, width)")
    width, ch = weight.shape[1], x.shape[-1]
    batch, rows, off, nseg, seqs = _sequences(x, offsets)
    state = (seqs, width - 1, ch)
    return [_DTYPES[x.dtype], _DTYPES.get(weight.dtype, -1), 1 if silu else 0, width, ch, batch, rows, nseg, *xr, *out,
            _weight(weight, x, (ch, width), "weight"), _dense(bias, (ch,), weight.dtype, x, "bias"), off,
            _dense(initial_state, state, x.dtype, x, "initial_state"),
            _dense(final_state, state, x.dtype, x, "final_state")], state


def causal_conv(x, weight, bias=None, offsets=None, initial_state=None, silu=True, return_state=False, out=None,
                final_state=None, stream=None):
    """Causal depthwise convolution of rows `x` with `weight` (channels, width),
    through x * sigmoid(x) if `silu`.  `initial_state` (sequences, width - 1,
    channels) holds the inputs before each sequence's first row (None: zeros).
    Returns out, or (out, final_state) with `return_state` or a `final_state`
    to write."""
    xr = _main(x, "x")
    out = _output(out, x, stream)
    if return_state and final_state is None:
        _need(weight.dim() == 2, "weight must have shape (channels, width)")
        final_state = _empty((_sequences(x, offsets)[4], weight.shape[1] - 1, x.shape[-1]), x.dtype, x, stream)
    fields, _ = _conv_fields(x, xr, _rows(out, "out"), weight, bias, offsets, initial_state, final_state, silu)
    _launch("dwp_causal_conv", fields, x, stream)
    return out if final_state is None else (out, final_state)


def causal_conv_backward(grad_out, x, weight, bias=None, offsets=None, initial_state=None, silu=True,
                         grad_final_state=None, scratch=None, stream=None):
    """Gradients of causal_conv: a dict of "x", "weight" and, where given,
    "bias" and "initial_state" (the last also with a `grad_final_state`)."""
    xr = _main(x, "x")
    gr = _like(grad_out, x, "grad_out")
    fields, state = _conv_fields(x, xr, _NO_ROWS, weight, bias, offsets, initial_state, None, silu)
    f32 = torch.float32
    grads = {"x": _output(None, x, stream), "weight": _empty(weight.shape, f32, x, stream)}
    if bias is not None:
        grads["bias"] = _empty(bias.shape, f32, x, stream)
    if initial_state is not None or grad_final_state is not None:
        grads["initial_state"] = _empty(state, x.dtype, x, stream)
    at = lambda k: grads[k].data_ptr() if k in grads else 0  # noqa: E731
    fields += [*gr, *_rows(grads["x"], "grad_x"), _dense(grad_final_state, state, x.dtype, x, "grad_final_state"),
               at("weight"), at("bias"), at("initial_state")]
    _launch("dwp_causal_conv_backward", fields, x, stream, scratch)
    return grads


def _slots(slots, batch, x):
    if slots is None:
        return 0
    _need(slots.dtype == torch.int32, "slots must be int32")
    return _dense(slots, (batch,), torch.int32, x, "slots")


def _cache(state, shape, x):
    """Whether `state` is (slots, *shape) on x's device, each slot contiguous."""
    s = state.stride()
    return (len(s) == 3 and state.shape[1:] == shape and state.get_device() == x.get_device()
            and (state.numel() == 0 or ((s[2] == 1 or shape[1] == 1) and (s[1] == shape[1] or shape[0] == 1))))


def causal_conv_step(x, state, weight, bias=None, slots=None, silu=True, out=None, stream=None):
    """causal_conv of one new row of each of `batch` sequences: x (batch,
    channels), `state` (num_slots, width - 1, channels) updated in place.
    `slots` (int32, batch) names each row's state; a slot outside the cache
    marks a padding row (output 0).  None: row i has state i.  Returns out."""
    xr = _main(x, "x", (2,))
    out = _output(out, x, stream)
    batch, ch = x.shape
    _need(weight.dim() == 2 and weight.shape[0] == ch, "weight must have shape (channels, width)")
    width = weight.shape[1]
    _need(state.dtype == x.dtype and _cache(state, (width - 1, ch), x),
          "state must have shape (slots, width - 1, channels), each slot contiguous, and x's type and device")
    fields = [_DTYPES[x.dtype], _DTYPES.get(weight.dtype, -1), 1 if silu else 0, width, ch, batch, state.shape[0],
              *xr, *_rows(out, "out"), _weight(weight, x, (ch, width), "weight"),
              _dense(bias, (ch,), weight.dtype, x, "bias"), state.data_ptr(), state.stride(0),
              _slots(slots, batch, x)]
    _launch("dwp_causal_conv_step", fields, x, stream)
    return out


# ---------------------------------------------------------------------------
# selective scan


def _bc(t, u, what):
    """(rows triple, group stride, groups, states) of B or C: (..., groups, states) or (..., states)."""
    lead = u.dim() - 1
    s, shape = t.stride(), t.shape
    if (t.dtype != u.dtype or t.get_device() != u.get_device() or not lead + 1 <= len(s) <= lead + 2
            or shape[:lead] != u.shape[:lead]):
        _refuse("%s must have u's rows, type and device, and shape (..., groups, states)", what)
    if s[-1] != 1 and shape[-1] > 1 and t.numel():
        _refuse("%s must have contiguous states", what)
    batch, row = (s[0], s[1]) if lead == 2 else (0, s[0])
    if len(s) == lead + 2:
        return (t.data_ptr(), batch, row), s[-2], shape[-2], shape[-1]
    return (t.data_ptr(), batch, row), 0, 1, shape[-1]


def _scan_parts(u, dt, A, B, C, D, z, dt_bias, out):
    """The fields that the prompt and the token form share."""
    ch, f32 = u.shape[-1], torch.float32
    br, bg, groups, n = _bc(B, u, "B")
    cr, cg, cgroups, cn = _bc(C, u, "C")
    _need((groups, n) == (cgroups, cn), "B and C must have the same groups and states")
    rows = [*_main(u, "u"), *_like(dt, u, "dt"), *_like(z, u, "z"), *br, *cr, *out, bg, cg,
            _dense(A, (ch, n), f32, u, "A"), _dense(D, (ch,), f32, u, "D"),
            _dense(dt_bias, (ch,), f32, u, "dt_bias")]
    return rows, groups, n


def _scan_fields(u, dt, A, B, C, D, z, dt_bias, out, offsets, initial, final, checkpoints, dt_softplus):
    parts, groups, n = _scan_parts(u, dt, A, B, C, D, z, dt_bias, out)
    batch, rows, off, nseg, seqs = _sequences(u, offsets)
    ch, f32 = u.shape[-1], torch.float32
    state = (seqs, ch, n)
    points = (batch, -(-rows // CHECKPOINT_ROWS), ch, n)
    return [_DTYPES[u.dtype], 1 if dt_softplus else 0, ch, n, groups, batch, rows, nseg, *parts, off,
            _dense(initial, state, f32, u, "initial_state"), _dense(final, state, f32, u, "final_state"),
            _dense(checkpoints, points, f32, u, "checkpoints")], state


def selective_scan(u, dt, A, B, C, D=None, z=None, dt_bias=None, offsets=None, initial_state=None, dt_softplus=True,
                   return_state=False, return_checkpoints=False, out=None, final_state=None, checkpoints=None,
                   scratch=None, stream=None):
    """Selective state space scan.  u, dt, z: rows of channels; B, C: rows of
    (groups, states), or of states; A (channels, states), D, dt_bias
    (channels): float32.  `initial_state` (sequences, channels, states) is
    float32 (None: zeros).  Returns out, or a tuple of out and then, where
    asked for, the final state and the checkpoints that the gradient needs."""
    _main(u, "u")
    out = _output(out, u, stream)
    batch, rows, _, _, seqs = _sequences(u, offsets)
    ch, n = u.shape[-1], A.shape[-1]
    if return_state and final_state is None:
        final_state = _empty((seqs, ch, n), torch.float32, u, stream)
    if return_checkpoints and checkpoints is None:
        checkpoints = _empty((batch, -(-rows // CHECKPOINT_ROWS), ch, n), torch.float32, u, stream)
    fields, _ = _scan_fields(u, dt, A, B, C, D, z, dt_bias, _rows(out, "out"), offsets, initial_state, final_state,
                             checkpoints, dt_softplus)
    _launch("dwp_selective_scan", fields, u, stream, scratch)
    if final_state is None and checkpoints is None:
        return out
    return (out, *(t for t in (final_state, checkpoints) if t is not None))


def selective_scan_backward(grad_out, u, dt, A, B, C, checkpoints, D=None, z=None, dt_bias=None, offsets=None,
                            initial_state=None, dt_softplus=True, grad_final_state=None, scratch=None, stream=None):
    """Gradients of selective_scan: a dict of "u", "dt", "A", "B", "C" and,
    where given, "D", "z", "dt_bias" and "initial_state" (the last also with a
    `grad_final_state`).  `checkpoints` are the forward's."""
    _main(u, "u")
    gr = _like(grad_out, u, "grad_out")
    _need(checkpoints is not None, "the gradient needs the forward's checkpoints")
    fields, state = _scan_fields(u, dt, A, B, C, D, z, dt_bias, _NO_ROWS, offsets, initial_state, None, checkpoints,
                                 dt_softplus)
    f32 = torch.float32
    grads = {"u": _output(None, u, stream), "dt": _output(None, u, stream), "A": _empty(A.shape, f32, u, stream),
             "B": _empty(B.shape, u.dtype, u, stream), "C": _empty(C.shape, u.dtype, u, stream)}
    if D is not None:
        grads["D"] = _empty(D.shape, f32, u, stream)
    if z is not None:
        grads["z"] = _output(None, u, stream)
    if dt_bias is not None:
        grads["dt_bias"] = _empty(dt_bias.shape, f32, u, stream)
    if initial_state is not None or grad_final_state is not None:
        grads["initial_state"] = _empty(state, f32, u, stream)
    at = lambda k: grads[k].data_ptr() if k in grads else 0  # noqa: E731
    fields += [*gr, _dense(grad_final_state, state, f32, u, "grad_final_state"), at("u"), at("dt"), at("z"), at("B"),
               at("C"), at("A"), at("D"), at("dt_bias"), at("initial_state")]
    _launch("dwp_selective_scan_backward", fields, u, stream, scratch)
    return grads


def selective_scan_step(u, dt, A, B, C, state, D=None, z=None, dt_bias=None, slots=None, dt_softplus=True, out=None,
                        stream=None):
    """selective_scan of one new row of each of `batch` sequences: u, dt, z
    (batch, channels), B, C (batch, groups, states) or (batch, states),
    `state` float32 (num_slots, channels, states) updated in place; `slots` as
    for causal_conv_step.  Returns out."""
    _main(u, "u", (2,))
    out = _output(out, u, stream)
    parts, groups, n = _scan_parts(u, dt, A, B, C, D, z, dt_bias, _rows(out, "out"))
    batch, ch = u.shape
    _need(state.dtype == torch.float32 and _cache(state, (ch, n), u),
          "state must be float32 of shape (slots, channels, states), each slot contiguous, on u's device")
    fields = [_DTYPES[u.dtype], 1 if dt_softplus else 0, ch, n, groups, batch, state.shape[0], *parts,
              state.data_ptr(), state.stride(0), _slots(slots, batch, u)]
    _launch("dwp_selective_scan_step", fields, u, stream)
    return out


# ---------------------------------------------------------------------------
# block norm


def _norm_rows(t, x, what, f32=False):
    """(address, 0, row stride) of a tensor of x's shape, (rows, channels) or
    (batch, rows, channels) with evenly spaced rows; of x's type, or float32
    where `f32` allows it.  Zeros for None."""
    if t is None:
        return _NO_ROWS
    if t is not x and (t.shape != x.shape or (t.dtype != x.dtype and not (f32 and t.dtype == torch.float32))
                       or t.get_device() != x.get_device()):
        _refuse("%s must have the shape and device of the call's main input, and its type (a residual or sum: or float32)",
                what)
    s, shape = t.stride(), t.shape
    if s[-1] != 1 and shape[-1] > 1 and t.numel():
        _refuse("%s must have contiguous channels", what)
    if len(s) == 2:
        return t.data_ptr(), 0, s[0]
    if shape[0] > 1 and shape[1] > 1 and s[0] != shape[1] * s[1]:
        _refuse("%s must have evenly spaced rows", what)
    return t.data_ptr(), 0, s[1] if shape[1] > 1 else s[0]


def _norm_main(x, what):
    if not x.is_cuda or x.dtype not in _DTYPES or not 2 <= x.dim() <= 3:
        _refuse("%s must be a CUDA tensor of float32, bfloat16 or float16 rows", what)
    return _norm_rows(x, x, what)


def _norm_fields(x, weight, scale, rdtype, gate_after, groups, eps, *rows):
    ch = x.shape[-1]
    return [_DTYPES[x.dtype], _DTYPES.get(weight.dtype, -1), rdtype, 1 if gate_after else 0, ch, groups,
            x.numel() // ch if ch else 0, float(eps), *rows, _weight(weight, x, (ch,), "weight"),
            _dense(scale, (ch,), weight.dtype, x, "scale")]


def block_norm(x, weight, residual=None, scale=None, gate=None, gate_after=False, groups=1, eps=1e-5, out=None,
               sum_out=None, stream=None):
    """Root-mean-square norm over each of `groups` parts of a row, times
    `weight`: of x; of residual + scale * x with a `residual` (scale (channels)
    or None for 1), which is also returned; of x * silu(gate) with a `gate`, or
    times silu(gate) afterwards if `gate_after`.  `out` may be x and `sum_out`
    may be residual, in place.  Returns (out, sum), sum None without a residual."""
    xr = _norm_main(x, "x")
    if out is None:
        out = _empty(x.shape, x.dtype, x, stream)
    total, rr, tr, rdtype = None, _NO_ROWS, _NO_ROWS, _DTYPES[x.dtype]
    if residual is not None:
        rr, rdtype = _norm_rows(residual, x, "residual", True), _DTYPES[residual.dtype]
        total = _empty(x.shape, residual.dtype, x, stream) if sum_out is None else sum_out
        _need(total.dtype == residual.dtype, "sum_out must have residual's type")
        tr = _norm_rows(total, x, "sum_out", True)
    fields = _norm_fields(x, weight, scale, rdtype, gate_after, groups, eps, *xr, *rr, *_norm_rows(gate, x, "gate"), *tr,
                          *_norm_rows(out, x, "out"))
    _launch("dwp_block_norm", fields, x, stream)
    return out, total


def block_norm_backward(grad_out, v, weight, x=None, scale=None, gate=None, gate_after=False, grad_residual=None,
                        groups=1, eps=1e-5, residual=None, scratch=None, stream=None):
    """Gradients of block_norm.  `v` is what was normed: the returned sum where
    there was a residual, else x.  `residual` says whether there was one (None:
    there was if `scale`, `grad_residual` or v's type says so); `x` is needed
    with a `scale`; `grad_residual` is the returned sum's gradient.  A dict of
    "x", "weight" and, where they apply, "residual", "scale" and "gate"; "x"
    and "residual" are one tensor where they are equal."""
    gr = _norm_main(grad_out, "grad_out")
    if residual is None:
        residual = scale is not None or grad_residual is not None or v.dtype != grad_out.dtype
    _need(scale is None or (x is not None and residual), "the scale's gradient needs x, and a residual")
    _need(residual or v.dtype == grad_out.dtype, "v must have grad_out's type without a residual")
    _need(grad_residual is None or (residual and grad_residual.dtype == v.dtype),
          "grad_residual must have v's type, with a residual")
    vr = _norm_rows(v, grad_out, "v", True)
    shape, f32 = grad_out.shape, torch.float32
    grads = {"weight": _empty(weight.shape, f32, grad_out, stream), "x": _empty(shape, grad_out.dtype, grad_out, stream)}
    gx, gres, gz = _norm_rows(grads["x"], grad_out, "grad_x"), _NO_ROWS, _NO_ROWS
    if residual:
        if scale is None and v.dtype == grad_out.dtype:
            grads["residual"] = grads["x"]  # the same numbers
        else:
            grads["residual"] = _empty(shape, v.dtype, grad_out, stream)
            gres = _norm_rows(grads["residual"], grad_out, "grad_residual", True)
    if scale is not None:
        grads["scale"] = _empty(scale.shape, f32, grad_out, stream)
    if gate is not None:
        grads["gate"] = _empty(shape, grad_out.dtype, grad_out, stream)
        gz = _norm_rows(grads["gate"], grad_out, "grad_gate")
    xr = vr if not residual else _norm_rows(x, grad_out, "x") if scale is not None else _NO_ROWS
    fields = _norm_fields(grad_out, weight, scale, _DTYPES[v.dtype], gate_after, groups, eps, *xr, *_NO_ROWS,
                          *_norm_rows(gate, grad_out, "gate"), *(vr if residual else _NO_ROWS), *_NO_ROWS)
    fields += [*gr, *_norm_rows(grad_residual, grad_out, "grad_residual", True), *gx, *gres, *gz,
               grads["weight"].data_ptr(), grads["scale"].data_ptr() if scale is not None else 0]
    _launch("dwp_block_norm_backward", fields, grad_out, stream, scratch)
    return grads
