"""Retention: linear attention with a decay for each head, and the group norm
with an activation behind it.  Python binding of the ``ssd_linear_attn_*`` and
``ssd_group_norm_*`` entry points of include/ssd.h.

The functions carry the C names and only marshal arguments.  The runners hold
what a program keeps between calls (the dimensions and the workspace) and check
the tensors they are given; a runner's workspace belongs to one stream at a time.

A call runs on the runner's device, on ``stream`` (a stream, or its handle, which then has to outlive the runner)
or, without one, on the device's current stream.  What it allocates, outputs and a larger workspace, belongs to that stream as it would to a current one, and a workspace
that another stream used is kept for it.  That inputs are ready on the stream, and that they outlive the call
there, is the caller's affair, as it is under torch.cuda.stream.
"""
from __future__ import annotations

import ctypes

import torch

__all__ = [
    "SsdLinearAttnDims", "SsdLinearAttnInputs", "SsdLinearAttnGrads", "ssd_linear_attn_workspace_size",
    "ssd_linear_attn_forward", "ssd_linear_attn_backward", "ssd_linear_attn_step", "LinearAttnRunner",
    "SsdGroupNormDims", "SsdGroupNormInputs", "SsdGroupNormGrads", "ssd_group_norm_workspace_size",
    "ssd_group_norm_forward", "ssd_group_norm_backward", "GroupNormRunner",
    "SSD_ACT_NONE", "SSD_ACT_SILU", "SSD_ACT_GATE",
]

SSD_ACT_NONE, SSD_ACT_SILU, SSD_ACT_GATE = 0, 1, 2
_P, _I32, _I64, _F32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
_ACTS = {"none": SSD_ACT_NONE, "silu": SSD_ACT_SILU, "gate": SSD_ACT_GATE}
_DTYPES = {"bf16": (0, torch.bfloat16), "f32": (1, torch.float32)}


class SsdLinearAttnDims(ctypes.Structure):
    _fields_ = [(n, _I32) for n in ("nseq", "seqlen", "total_tokens", "packed", "nheads", "nheads_kv", "headdim_k",
                                    "headdim_v", "dtype")]


class SsdLinearAttnInputs(ctypes.Structure):
    _fields_ = [("q", _P), ("q_tok_stride", _I64), ("k", _P), ("k_tok_stride", _I64), ("v", _P),
                ("v_tok_stride", _I64), ("log_decay", _P), ("initial_states", _P), ("cu_seqlens", _P),
                ("scale", _F32)]


class SsdLinearAttnGrads(ctypes.Structure):
    _fields_ = [("dq", _P), ("dq_tok_stride", _I64), ("dk", _P), ("dk_tok_stride", _I64), ("dv", _P),
                ("dv_tok_stride", _I64), ("dinitial_states", _P)]


class SsdGroupNormDims(ctypes.Structure):
    _fields_ = [(n, _I32) for n in ("nsamples", "nrows", "channels", "groups", "dtype", "activation")]


class SsdGroupNormInputs(ctypes.Structure):
    _fields_ = [("x", _P), ("x_row_stride", _I64), ("z", _P), ("z_row_stride", _I64), ("weight", _P), ("bias", _P),
                ("eps", _F32)]


class SsdGroupNormGrads(ctypes.Structure):
    _fields_ = [("dx", _P), ("dx_row_stride", _I64), ("dz", _P), ("dz_row_stride", _I64), ("dweight", _P),
                ("dbias", _P)]


def declare(lib) -> None:
    """Argument types of this module's entry points (called once, when the library is loaded)."""
    size, ptr = ctypes.c_size_t, ctypes.POINTER
    D, I, G = ptr(SsdLinearAttnDims), ptr(SsdLinearAttnInputs), ptr(SsdLinearAttnGrads)
    lib.ssd_linear_attn_workspace_size.argtypes = [D, ctypes.c_int]
    lib.ssd_linear_attn_workspace_size.restype = size
    lib.ssd_linear_attn_forward.argtypes = [D, I, _P, _I64, _P, _P, size, _P]
    lib.ssd_linear_attn_forward.restype = ctypes.c_int
    lib.ssd_linear_attn_backward.argtypes = [D, I, _P, _I64, _P, G, _P, size, _P]
    lib.ssd_linear_attn_backward.restype = ctypes.c_int
    lib.ssd_linear_attn_step.argtypes = [D, I, _P, _I32, _P, _P, _I64, _P]
    lib.ssd_linear_attn_step.restype = ctypes.c_int
    D, I, G = ptr(SsdGroupNormDims), ptr(SsdGroupNormInputs), ptr(SsdGroupNormGrads)
    lib.ssd_group_norm_workspace_size.argtypes = [D, ctypes.c_int]
    lib.ssd_group_norm_workspace_size.restype = size
    lib.ssd_group_norm_forward.argtypes = [D, I, _P, _I64, _P, _P, _P, size, _P]
    lib.ssd_group_norm_forward.restype = ctypes.c_int
    lib.ssd_group_norm_backward.argtypes = [D, I, _P, _I64, _P, _P, G, _P, size, _P]
    lib.ssd_group_norm_backward.restype = ctypes.c_int


_loaded = None


def _lib():
    global _loaded
    if _loaded is None:
        from . import load

        _loaded = load()
    return _loaded


def _check(status: int, what: str) -> None:
    if status != 0:
        from . import SsdError

        raise SsdError(status, what)


def _ptr(t):
    return None if t is None else t if isinstance(t, int) else t.data_ptr()


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream if isinstance(stream, int) else stream.cuda_stream


def _bytes(ws, ws_bytes) -> int:
    return ws.numel() * ws.element_size() if ws_bytes is None else ws_bytes


# ---------------------------------------------------------------- the C entry points

def ssd_linear_attn_workspace_size(dims: SsdLinearAttnDims, backward: bool) -> int:
    return int(_lib().ssd_linear_attn_workspace_size(ctypes.byref(dims), int(bool(backward))))


def ssd_linear_attn_forward(dims, inputs, o, o_tok_stride, final_states, workspace, ws_bytes=None,
                            stream=None) -> None:
    _check(_lib().ssd_linear_attn_forward(ctypes.byref(dims), ctypes.byref(inputs), _ptr(o), o_tok_stride,
                                          _ptr(final_states), _ptr(workspace), _bytes(workspace, ws_bytes),
                                          _stream(stream)), "ssd_linear_attn_forward")


def ssd_linear_attn_backward(dims, inputs, dout, dout_tok_stride, dfinal_states, grads, workspace, ws_bytes=None,
                             stream=None) -> None:
    _check(_lib().ssd_linear_attn_backward(ctypes.byref(dims), ctypes.byref(inputs), _ptr(dout), dout_tok_stride,
                                           _ptr(dfinal_states), ctypes.byref(grads), _ptr(workspace),
                                           _bytes(workspace, ws_bytes), _stream(stream)), "ssd_linear_attn_backward")


def ssd_linear_attn_step(dims, inputs, states, nslots, slot_idx, o, o_tok_stride, stream=None) -> None:
    _check(_lib().ssd_linear_attn_step(ctypes.byref(dims), ctypes.byref(inputs), _ptr(states), nslots,
                                       _ptr(slot_idx), _ptr(o), o_tok_stride, _stream(stream)),
           "ssd_linear_attn_step")


def ssd_group_norm_workspace_size(dims: SsdGroupNormDims, backward: bool) -> int:
    return int(_lib().ssd_group_norm_workspace_size(ctypes.byref(dims), int(bool(backward))))


def ssd_group_norm_forward(dims, inputs, y, y_row_stride, mean, rstd, workspace, ws_bytes=None, stream=None) -> None:
    _check(_lib().ssd_group_norm_forward(ctypes.byref(dims), ctypes.byref(inputs), _ptr(y), y_row_stride, _ptr(mean),
                                         _ptr(rstd), _ptr(workspace), _bytes(workspace, ws_bytes), _stream(stream)),
           "ssd_group_norm_forward")


def ssd_group_norm_backward(dims, inputs, dy, dy_row_stride, mean, rstd, grads, workspace, ws_bytes=None,
                            stream=None) -> None:
    _check(_lib().ssd_group_norm_backward(ctypes.byref(dims), ctypes.byref(inputs), _ptr(dy), dy_row_stride,
                                          _ptr(mean), _ptr(rstd), ctypes.byref(grads), _ptr(workspace),
                                          _bytes(workspace, ws_bytes), _stream(stream)), "ssd_group_norm_backward")


# ---------------------------------------------------------------- runners

def _rows(x, name: str, rows: int, width: int, dtype, device) -> tuple[int, int]:
    """(address, row stride) of a (..., width) tensor whose leading dimensions flatten to `rows` evenly spaced rows."""
    strides = x.stride()
    # the usual case first: a small call's time is mostly spent on the host
    if (len(strides) == 2 and strides[1] == 1 and x.dtype is dtype and x.shape == (rows, width)
            and x.get_device() == device.index and x.is_cuda):
        return x.data_ptr(), strides[0] if rows > 1 else max(width, strides[0])
    shape = x.shape
    if x.dtype != dtype or x.device != device:
        raise ValueError(f"{name}: expected {dtype} on {device}, got {x.dtype} on {x.device}")
    if x.dim() < 2 or shape[-1] != width or x.numel() != rows * width:
        raise ValueError(f"{name}: expected {rows} rows of {width} channels, got {tuple(shape)}")
    if width > 1 and strides[-1] != 1:
        raise ValueError(f"{name}: channels must be contiguous")
    step, count = 0, 1  # rows seen so far, innermost first, and their spacing
    for size, stride in zip(reversed(shape[:-1]), reversed(strides[:-1])):
        if size == 1:
            continue
        if count == 1:
            step = stride
        elif stride != step * count:
            raise ValueError(f"{name}: rows must be evenly spaced")
        count *= size
    return x.data_ptr(), step if count > 1 else width


def _exact(x, name: str, shape: tuple, dtype, device):
    if x is None:
        return None
    if x.dtype is not dtype or x.shape != shape or x.device != device or not x.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous {dtype} tensor of shape {shape} on {device}, "
                         f"got {x.dtype} {tuple(x.shape)} on {x.device}")
    return x.data_ptr()


def _current(runner):
    """Handle of the current stream, for which the runner's workspace is kept from now on."""
    handle = torch._C._cuda_getCurrentRawStream(runner.device.index)
    if handle != runner._stream:
        runner.workspace.record_stream(torch.cuda.current_stream(runner.device))
        runner._stream = handle
    return handle


def _elsewhere(runner, stream):
    """What makes the runner's device and the given stream the current ones, so that a call is launched there and what it
    allocates belongs to the stream it is written on; None where they are current already."""
    index = runner.device.index
    if stream is None:
        return None if index is None or index == torch._C._cuda_getDevice() else torch.cuda.device(runner.device)
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=runner.device)
    if stream.device != runner.device:
        raise ValueError(f"stream: expected one of {runner.device}, got one of {stream.device}")
    return torch.cuda.stream(stream)


def _device(device) -> torch.device:
    device = torch.device(device)
    if device.type == "cuda" and device.index is None:
        device = torch.device("cuda", torch.cuda.current_device())
    return device


def _grow(runner, workspace_size) -> None:
    """The workspace that backward passes need, from the first one on.  The forward pass's stays alive: a stream that
    is not the allocator's may still be using it."""
    if runner._forward_workspace is None:
        size = workspace_size(runner.dims, True)
        runner._forward_workspace = runner.workspace
        if runner.workspace.numel() < size:
            runner.workspace = torch.empty(size, dtype=torch.uint8, device=runner.device)


class LinearAttnRunner:
    """Linear attention of one shape: S_t = lam S_(t-1) + k_t^T v_t, o_t = scale q_t S_t per head.

    ``tokens`` is each sequence's length, or with ``packed=True`` the rows of all ``nseq`` sequences together, whose
    bounds every call then takes as ``cu_seqlens``.  q, k, v and gradients are (rows, heads * headdim) or
    (nseq, tokens, heads * headdim), possibly strided views of one projection output.  ``scale`` defaults to
    headdim_k ** -0.5."""

    def __init__(self, nseq: int, tokens: int, nheads: int, headdim_k: int, headdim_v: int, *, nheads_kv=None,
                 dtype: str = "bf16", packed: bool = False, device="cuda"):
        self.nseq, self.nheads, self.nheads_kv = nseq, nheads, nheads if nheads_kv is None else nheads_kv
        self.headdim_k, self.headdim_v, self.packed = headdim_k, headdim_v, bool(packed)
        self.rows = tokens if packed else nseq * tokens
        self.device = _device(device)
        code, self.tdtype = _DTYPES[dtype]
        self.dims = SsdLinearAttnDims(nseq, 0 if packed else tokens, tokens if packed else 0, int(self.packed),
                                      nheads, self.nheads_kv, headdim_k, headdim_v, code)
        size = ssd_linear_attn_workspace_size(self.dims, False)
        if size == 0:
            raise ValueError("invalid dims for libssd")
        self.state_shape = (nseq, nheads, headdim_k, headdim_v)
        self.workspace = torch.empty(size, dtype=torch.uint8, device=self.device)
        self._stream = None  # the last one that used the workspace
        self._widths = (nheads * headdim_k, self.nheads_kv * headdim_k, self.nheads_kv * headdim_v,
                        nheads * headdim_v)
        self._scale = headdim_k ** -0.5
        self._heads, self._bounds = (nheads,), (nseq + 1,)
        self._forward_workspace = None

    def _grow(self):
        _grow(self, ssd_linear_attn_workspace_size)

    def _inputs(self, q, k, v, log_decay, scale, init, cu) -> SsdLinearAttnInputs:
        wq, wk, wv, _ = self._widths
        rows, tdtype, device = self.rows, self.tdtype, self.device
        qp, qs = _rows(q, "q", rows, wq, tdtype, device)
        kp, ks = _rows(k, "k", rows, wk, tdtype, device)
        vp, vs = _rows(v, "v", rows, wv, tdtype, device)
        if (cu is not None) != self.packed:
            raise ValueError("cu_seqlens goes with packed=True")
        f32 = torch.float32
        return SsdLinearAttnInputs(qp, qs, kp, ks, vp, vs, _exact(log_decay, "log_decay", self._heads, f32, device),
                                   _exact(init, "initial_state", self.state_shape, f32, device),
                                   _exact(cu, "cu_seqlens", self._bounds, torch.int32, device),
                                   self._scale if scale is None else scale)

    def forward(self, q, k, v, log_decay, *, scale=None, initial_state=None, cu_seqlens=None, final_state=True,
                out=None, stream=None):
        """(o, final_state): o (rows, nheads * headdim_v); final_state (nseq, nheads, headdim_k, headdim_v) fp32, or
        None with final_state=False.  ``out``: a tensor for o."""
        there = _elsewhere(self, stream)
        if there is not None:
            with there:
                return self.forward(q, k, v, log_decay, scale=scale, initial_state=initial_state,
                                    cu_seqlens=cu_seqlens, final_state=final_state, out=out)
        wo = self._widths[3]
        inputs = self._inputs(q, k, v, log_decay, scale, initial_state, cu_seqlens)
        if out is None:
            o = torch.empty(self.rows, wo, dtype=self.tdtype, device=self.device)
            op, os = o.data_ptr(), wo
        else:
            o = out
            op, os = _rows(o, "out", self.rows, wo, self.tdtype, self.device)
        fin = torch.empty(self.state_shape, dtype=torch.float32, device=self.device) if final_state else None
        ssd_linear_attn_forward(self.dims, inputs, op, os, fin, self.workspace, stream=_current(self))
        return o, fin

    def backward(self, q, k, v, log_decay, do, *, scale=None, initial_state=None, dfinal_state=None, cu_seqlens=None,
                 stream=None) -> dict:
        """Gradients of <do, o> + <dfinal_state, final_state>: dq, dk, dv, and dinitial_state (None without an
        initial state)."""
        there = _elsewhere(self, stream)
        if there is not None:
            with there:
                return self.backward(q, k, v, log_decay, do, scale=scale, initial_state=initial_state,
                                     dfinal_state=dfinal_state, cu_seqlens=cu_seqlens)
        wq, wk, wv, wo = self._widths
        rows, tdtype, device = self.rows, self.tdtype, self.device
        inputs = self._inputs(q, k, v, log_decay, scale, initial_state, cu_seqlens)
        dop, dos = _rows(do, "do", rows, wo, tdtype, device)
        dfin = _exact(dfinal_state, "dfinal_state", self.state_shape, torch.float32, device)
        self._grow()
        g = {"dq": torch.empty(rows, wq, dtype=tdtype, device=device),
             "dk": torch.empty(rows, wk, dtype=tdtype, device=device),
             "dv": torch.empty(rows, wv, dtype=tdtype, device=device),
             "dinitial_state": None if initial_state is None else torch.empty(self.state_shape, dtype=torch.float32,
                                                                              device=device)}
        grads = SsdLinearAttnGrads(g["dq"].data_ptr(), wq, g["dk"].data_ptr(), wk, g["dv"].data_ptr(), wv,
                                   _ptr(g["dinitial_state"]))
        ssd_linear_attn_backward(self.dims, inputs, dop, dos, dfin, grads, self.workspace, stream=_current(self))
        return g

    def step(self, q, k, v, log_decay, states, *, slot_idx=None, scale=None, out=None, stream=None):
        """One token of each of ``nseq`` rows (a runner with tokens=1): updates ``states`` (slots, nheads, headdim_k,
        headdim_v) in place at ``slot_idx`` (int32; None: row r uses slot r; a negative one leaves the cache alone and
        gives zeros) and returns o (rows, nheads * headdim_v)."""
        there = _elsewhere(self, stream)
        if there is not None:
            with there:
                return self.step(q, k, v, log_decay, states, slot_idx=slot_idx, scale=scale, out=out)
        wo = self._widths[3]
        inputs = self._inputs(q, k, v, log_decay, scale, None, None)
        _exact(states, "states", (states.shape[0],) + self.state_shape[1:], torch.float32, self.device)
        idx = _exact(slot_idx, "slot_idx", (self.nseq,), torch.int32, self.device)
        if out is None:
            o = torch.empty(self.rows, wo, dtype=self.tdtype, device=self.device)
            op, os = o.data_ptr(), wo
        else:
            o = out
            op, os = _rows(o, "out", self.rows, wo, self.tdtype, self.device)
        ssd_linear_attn_step(self.dims, inputs, states, states.shape[0], idx, op, os, _current(self))
        return o


class GroupNormRunner:
    """Group norm with an activation ("none", "silu", or "gate": times silu of a tensor z), channels last.

    x is (nsamples, nrows, channels), or nsamples * nrows rows; statistics are over the rows and the channels of a
    group of each sample (nrows=1: each head of each token)."""

    def __init__(self, nsamples: int, nrows: int, channels: int, groups: int, activation: str = "none",
                 dtype: str = "bf16", device="cuda"):
        self.rows, self.channels, self.stat_shape = nsamples * nrows, channels, (nsamples, groups)
        self.activation, self.device = activation, _device(device)
        code, self.tdtype = _DTYPES[dtype]
        self.dims = SsdGroupNormDims(nsamples, nrows, channels, groups, code, _ACTS[activation])
        size = ssd_group_norm_workspace_size(self.dims, False)
        if size == 0:
            raise ValueError("invalid dims for libssd")
        self.workspace = torch.empty(size, dtype=torch.uint8, device=self.device)
        self._stream = None  # the last one that used the workspace
        self._forward_workspace = None

    def _grow(self):
        _grow(self, ssd_group_norm_workspace_size)

    def _row(self, x, name):
        return _rows(x, name, self.rows, self.channels, self.tdtype, self.device)

    def _inputs(self, x, weight, bias, z, eps) -> SsdGroupNormInputs:
        xp, xs = self._row(x, "x")
        if (z is not None) != (self.activation == "gate"):
            raise ValueError('z goes with activation="gate"')
        zp, zs = (None, 0) if z is None else self._row(z, "z")
        shape = (self.channels,)
        return SsdGroupNormInputs(xp, xs, zp, zs, _exact(weight, "weight", shape, torch.float32, self.device),
                                  _exact(bias, "bias", shape, torch.float32, self.device), eps)

    def forward(self, x, weight=None, bias=None, *, z=None, eps: float = 1e-5, out=None, stream=None):
        """(y, mean, rstd): y shaped like x; mean and rstd (nsamples, groups) fp32, for backward."""
        there = _elsewhere(self, stream)
        if there is not None:
            with there:
                return self.forward(x, weight, bias, z=z, eps=eps, out=out)
        inputs = self._inputs(x, weight, bias, z, eps)
        y = torch.empty(x.shape, dtype=self.tdtype, device=self.device) if out is None else out
        yp, ys = self._row(y, "out")
        stats = torch.empty((2,) + self.stat_shape, dtype=torch.float32, device=self.device)
        mean, rstd = stats[0], stats[1]
        ssd_group_norm_forward(self.dims, inputs, yp, ys, mean, rstd, self.workspace, stream=_current(self))
        return y, mean, rstd

    def backward(self, dy, x, weight, bias, mean, rstd, *, z=None, stream=None) -> dict:
        """dx, dweight, dbias, and dz with the gate (else None).  dweight and dbias are also given for the constant 1
        and 0 that stand for an absent weight and bias."""
        there = _elsewhere(self, stream)
        if there is not None:
            with there:
                return self.backward(dy, x, weight, bias, mean, rstd, z=z)
        device = self.device
        inputs = self._inputs(x, weight, bias, z, 0.0)
        dyp, dys = self._row(dy, "dy")
        mp = _exact(mean, "mean", self.stat_shape, torch.float32, device)
        rp = _exact(rstd, "rstd", self.stat_shape, torch.float32, device)
        self._grow()
        g = {"dx": torch.empty(x.shape, dtype=self.tdtype, device=device),
             "dz": None if z is None else torch.empty(x.shape, dtype=self.tdtype, device=device),
             "dweight": torch.empty(self.channels, dtype=torch.float32, device=device),
             "dbias": torch.empty(self.channels, dtype=torch.float32, device=device)}
        grads = SsdGroupNormGrads(g["dx"].data_ptr(), self.channels, _ptr(g["dz"]), self.channels,
                                  g["dweight"].data_ptr(), g["dbias"].data_ptr())
        ssd_group_norm_backward(self.dims, inputs, dyp, dys, mp, rp, grads, self.workspace, stream=_current(self))
        return g
