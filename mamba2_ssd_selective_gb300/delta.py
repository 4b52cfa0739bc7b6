"""The gated delta rule, and the norms around a block joined with its gate, its scale and the residual stream.
Python binding of the ``ssd_delta_rule_*`` and ``ssd_block_norm_*`` entry points of include/ssd.h.

The functions carry the C names and only marshal arguments.  The runners hold what a program keeps between calls and
check the tensors they are given; streams, devices and workspaces are treated as by the runners of retention.py.
"""
from __future__ import annotations

import ctypes

import torch

from .retention import (_DTYPES, _bytes, _check, _current, _device, _elsewhere, _exact, _grow, _lib, _ptr, _rows,
                        _stream)

__all__ = [
    "SsdDeltaRuleDims", "SsdDeltaRuleInputs", "SsdDeltaRuleGrads", "ssd_delta_rule_workspace_size",
    "ssd_delta_rule_forward", "ssd_delta_rule_backward", "ssd_delta_rule_step", "DeltaRuleRunner",
    "SsdBlockNormDims", "SsdBlockNormInputs", "SsdBlockNormSaved", "SsdBlockNormGrads",
    "ssd_block_norm_workspace_size", "ssd_block_norm_forward", "ssd_block_norm_backward", "BlockNormRunner",
]

_P, _I32, _I64, _F32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float


def _tensors(*names: str, stride: str):
    return [f for n in names for f in ((n, _P), (f"{n}_{stride}", _I64))]


class SsdDeltaRuleDims(ctypes.Structure):
    _fields_ = [(n, _I32) for n in ("nseq", "seqlen", "total_tokens", "packed", "nheads", "nheads_qk", "headdim_k",
                                    "headdim_v", "dtype", "qk_norm")]


class SsdDeltaRuleInputs(ctypes.Structure):
    _fields_ = _tensors("q", "k", "v", "log_decay", "beta", stride="tok_stride") + [
        ("initial_states", _P), ("cu_seqlens", _P), ("scale", _F32), ("norm_eps", _F32)]


class SsdDeltaRuleGrads(ctypes.Structure):
    _fields_ = _tensors("dq", "dk", "dv", "dlog_decay", "dbeta", stride="tok_stride") + [("dinitial_states", _P)]


class SsdBlockNormDims(ctypes.Structure):
    _fields_ = [(n, _I32) for n in ("rows", "channels", "dtype", "residual_dtype", "post_norm", "gate", "residual",
                                    "pre_norm")]


class SsdBlockNormInputs(ctypes.Structure):
    _fields_ = _tensors("x", "z", "residual", stride="row_stride") + [
        ("post_weight", _P), ("branch_scale", _P), ("pre_weight", _P), ("eps", _F32)]


class SsdBlockNormSaved(ctypes.Structure):
    _fields_ = _tensors("h", "dh", "dy", stride="row_stride") + [("rstd_post", _P), ("rstd_pre", _P)]


class SsdBlockNormGrads(ctypes.Structure):
    _fields_ = _tensors("dx", "dz", "dresidual", stride="row_stride") + [
        ("dpost_weight", _P), ("dbranch_scale", _P), ("dpre_weight", _P)]


def declare(lib) -> None:
    """Argument types of this module's entry points (called once, when the library is loaded)."""
    size, ptr = ctypes.c_size_t, ctypes.POINTER
    D, I, G = ptr(SsdDeltaRuleDims), ptr(SsdDeltaRuleInputs), ptr(SsdDeltaRuleGrads)
    lib.ssd_delta_rule_workspace_size.argtypes = [D, ctypes.c_int]
    lib.ssd_delta_rule_workspace_size.restype = size
    lib.ssd_delta_rule_forward.argtypes = [D, I, _P, _I64, _P, _P, size, _P]
    lib.ssd_delta_rule_forward.restype = ctypes.c_int
    lib.ssd_delta_rule_backward.argtypes = [D, I, _P, _I64, _P, G, _P, size, _P]
    lib.ssd_delta_rule_backward.restype = ctypes.c_int
    lib.ssd_delta_rule_step.argtypes = [D, I, _P, _I32, _P, _P, _I64, _P]
    lib.ssd_delta_rule_step.restype = ctypes.c_int
    D, I, S, G = ptr(SsdBlockNormDims), ptr(SsdBlockNormInputs), ptr(SsdBlockNormSaved), ptr(SsdBlockNormGrads)
    lib.ssd_block_norm_workspace_size.argtypes = [D]
    lib.ssd_block_norm_workspace_size.restype = size
    lib.ssd_block_norm_forward.argtypes = [D, I, _P, _I64, _P, _I64, _P, _P, _P]
    lib.ssd_block_norm_forward.restype = ctypes.c_int
    lib.ssd_block_norm_backward.argtypes = [D, I, S, G, _P, size, _P]
    lib.ssd_block_norm_backward.restype = ctypes.c_int


# ---------------------------------------------------------------- the C entry points

def ssd_delta_rule_workspace_size(dims: SsdDeltaRuleDims, backward: bool) -> int:
    return int(_lib().ssd_delta_rule_workspace_size(ctypes.byref(dims), int(bool(backward))))


def ssd_delta_rule_forward(dims, inputs, o, o_tok_stride, final_states, workspace, ws_bytes=None, stream=None) -> None:
    _check(_lib().ssd_delta_rule_forward(ctypes.byref(dims), ctypes.byref(inputs), _ptr(o), o_tok_stride,
                                         _ptr(final_states), _ptr(workspace), _bytes(workspace, ws_bytes),
                                         _stream(stream)), "ssd_delta_rule_forward")


def ssd_delta_rule_backward(dims, inputs, dout, dout_tok_stride, dfinal_states, grads, workspace, ws_bytes=None,
                            stream=None) -> None:
    _check(_lib().ssd_delta_rule_backward(ctypes.byref(dims), ctypes.byref(inputs), _ptr(dout), dout_tok_stride,
                                          _ptr(dfinal_states), ctypes.byref(grads), _ptr(workspace),
                                          _bytes(workspace, ws_bytes), _stream(stream)), "ssd_delta_rule_backward")


def ssd_delta_rule_step(dims, inputs, states, nslots, slot_idx, o, o_tok_stride, stream=None) -> None:
    _check(_lib().ssd_delta_rule_step(ctypes.byref(dims), ctypes.byref(inputs), _ptr(states), nslots, _ptr(slot_idx),
                                      _ptr(o), o_tok_stride, _stream(stream)), "ssd_delta_rule_step")


def ssd_block_norm_workspace_size(dims: SsdBlockNormDims) -> int:
    return int(_lib().ssd_block_norm_workspace_size(ctypes.byref(dims)))


def ssd_block_norm_forward(dims, inputs, h, h_row_stride, y, y_row_stride, rstd_post, rstd_pre, stream=None) -> None:
    _check(_lib().ssd_block_norm_forward(ctypes.byref(dims), ctypes.byref(inputs), _ptr(h), h_row_stride, _ptr(y),
                                         y_row_stride, _ptr(rstd_post), _ptr(rstd_pre), _stream(stream)),
           "ssd_block_norm_forward")


def ssd_block_norm_backward(dims, inputs, saved, grads, workspace, ws_bytes=None, stream=None) -> None:
    _check(_lib().ssd_block_norm_backward(ctypes.byref(dims), ctypes.byref(inputs), ctypes.byref(saved),
                                          ctypes.byref(grads), _ptr(workspace), _bytes(workspace, ws_bytes),
                                          _stream(stream)), "ssd_block_norm_backward")


# ---------------------------------------------------------------- runners

class DeltaRuleRunner:
    """The gated delta rule of one shape: S' = a_t S_(t-1), S_t = S' + beta_t k_t^T (v_t - k_t S'), o_t = scale q_t S_t
    per head, a_t = exp(log_decay_t).

    ``tokens`` is each sequence's length, or with ``packed=True`` the rows of all ``nseq`` sequences together, whose
    bounds every call then takes as ``cu_seqlens``.  q and k are (rows, nheads_qk * headdim_k), v and do
    (rows, nheads * headdim_v), log_decay and beta (rows, nheads), each possibly (nseq, tokens, ...) and a strided
    view, all of ``dtype``.  ``qk_norm``: q and k are divided by their length, sqrt(|.|^2 + norm_eps).  ``scale``
    defaults to headdim_k ** -0.5."""

    def __init__(self, nseq: int, tokens: int, nheads: int, headdim_k: int, headdim_v: int, *, nheads_qk=None,
                 qk_norm: bool = False, norm_eps: float = 1e-6, dtype: str = "bf16", packed: bool = False,
                 device="cuda"):
        self.nseq, self.nheads, self.nheads_qk = nseq, nheads, nheads if nheads_qk is None else nheads_qk
        self.headdim_k, self.headdim_v, self.packed = headdim_k, headdim_v, bool(packed)
        self.rows = tokens if packed else nseq * tokens
        self.qk_norm, self.norm_eps = bool(qk_norm), norm_eps
        self.device = _device(device)
        code, self.tdtype = _DTYPES[dtype]
        self.dims = SsdDeltaRuleDims(nseq, 0 if packed else tokens, tokens if packed else 0, int(self.packed), nheads,
                                     self.nheads_qk, headdim_k, headdim_v, code, int(self.qk_norm))
        size = ssd_delta_rule_workspace_size(self.dims, False)
        if size == 0:
            raise ValueError("invalid dims for libssd")
        self.state_shape = (nseq, nheads, headdim_k, headdim_v)
        # a runner of single tokens needs none
        self.workspace = torch.empty(0 if tokens == 1 and not packed else size, dtype=torch.uint8, device=self.device)
        self._size = size
        self._stream = None  # the last one that used the workspace
        self._widths = (self.nheads_qk * headdim_k, nheads * headdim_v)
        self._scale = headdim_k ** -0.5
        self._forward_workspace = None

    def _inputs(self, q, k, v, log_decay, beta, scale, init, cu) -> SsdDeltaRuleInputs:
        wk, wv = self._widths
        rows, tdtype, device, nheads = self.rows, self.tdtype, self.device, self.nheads
        qp, qs = _rows(q, "q", rows, wk, tdtype, device)
        kp, ks = _rows(k, "k", rows, wk, tdtype, device)
        vp, vs = _rows(v, "v", rows, wv, tdtype, device)
        gp, gs = _rows(log_decay, "log_decay", rows, nheads, tdtype, device)
        bp, bs = _rows(beta, "beta", rows, nheads, tdtype, device)
        if (cu is not None) != self.packed:
            raise ValueError("cu_seqlens goes with packed=True")
        return SsdDeltaRuleInputs(qp, qs, kp, ks, vp, vs, gp, gs, bp, bs,
                                  _exact(init, "initial_state", self.state_shape, torch.float32, device),
                                  _exact(cu, "cu_seqlens", (self.nseq + 1,), torch.int32, device),
                                  self._scale if scale is None else scale, self.norm_eps)

    def forward(self, q, k, v, log_decay, beta, *, scale=None, initial_state=None, cu_seqlens=None, final_state=True,
                out=None, stream=None):
        """(o, final_state): o (rows, nheads * headdim_v); final_state (nseq, nheads, headdim_k, headdim_v) fp32, or
        None with final_state=False.  ``out``: a tensor for o."""
        there = _elsewhere(self, stream)
        if there is not None:
            with there:
                return self.forward(q, k, v, log_decay, beta, scale=scale, initial_state=initial_state,
                                    cu_seqlens=cu_seqlens, final_state=final_state, out=out)
        wv = self._widths[1]
        inputs = self._inputs(q, k, v, log_decay, beta, scale, initial_state, cu_seqlens)
        if out is None:
            o = torch.empty(self.rows, wv, dtype=self.tdtype, device=self.device)
            op, os = o.data_ptr(), wv
        else:
            o = out
            op, os = _rows(o, "out", self.rows, wv, self.tdtype, self.device)
        fin = torch.empty(self.state_shape, dtype=torch.float32, device=self.device) if final_state else None
        if self.workspace.numel() < self._size:  # a single token taken as a prompt
            self.workspace = torch.empty(self._size, dtype=torch.uint8, device=self.device)
        ssd_delta_rule_forward(self.dims, inputs, op, os, fin, self.workspace, stream=_current(self))
        return o, fin

    def backward(self, q, k, v, log_decay, beta, do, *, scale=None, initial_state=None, dfinal_state=None,
                 cu_seqlens=None, stream=None) -> dict:
        """Gradients of <do, o> + <dfinal_state, final_state>: dq, dk, dv, dlog_decay, dbeta, and dinitial_state (None
        without an initial state)."""
        there = _elsewhere(self, stream)
        if there is not None:
            with there:
                return self.backward(q, k, v, log_decay, beta, do, scale=scale, initial_state=initial_state,
                                     dfinal_state=dfinal_state, cu_seqlens=cu_seqlens)
        wk, wv = self._widths
        rows, tdtype, device, nheads = self.rows, self.tdtype, self.device, self.nheads
        inputs = self._inputs(q, k, v, log_decay, beta, scale, initial_state, cu_seqlens)
        dop, dos = _rows(do, "do", rows, wv, tdtype, device)
        dfin = _exact(dfinal_state, "dfinal_state", self.state_shape, torch.float32, device)
        _grow(self, ssd_delta_rule_workspace_size)
        g = {"dq": torch.empty(rows, wk, dtype=tdtype, device=device),
             "dk": torch.empty(rows, wk, dtype=tdtype, device=device),
             "dv": torch.empty(rows, wv, dtype=tdtype, device=device),
             "dlog_decay": torch.empty(rows, nheads, dtype=tdtype, device=device),
             "dbeta": torch.empty(rows, nheads, dtype=tdtype, device=device),
             "dinitial_state": None if initial_state is None else torch.empty(self.state_shape, dtype=torch.float32,
                                                                              device=device)}
        grads = SsdDeltaRuleGrads(g["dq"].data_ptr(), wk, g["dk"].data_ptr(), wk, g["dv"].data_ptr(), wv,
                                  g["dlog_decay"].data_ptr(), nheads, g["dbeta"].data_ptr(), nheads,
                                  _ptr(g["dinitial_state"]))
        ssd_delta_rule_backward(self.dims, inputs, dop, dos, dfin, grads, self.workspace, stream=_current(self))
        return g

    def step(self, q, k, v, log_decay, beta, states, *, slot_idx=None, scale=None, out=None, stream=None):
        """One token of each of ``nseq`` rows (a runner with tokens=1): updates ``states`` (slots, nheads, headdim_k,
        headdim_v) in place at ``slot_idx`` (int32; None: row r uses slot r; a negative one leaves the cache alone and
        gives zeros) and returns o (rows, nheads * headdim_v)."""
        there = _elsewhere(self, stream)
        if there is not None:
            with there:
                return self.step(q, k, v, log_decay, beta, states, slot_idx=slot_idx, scale=scale, out=out)
        wv = self._widths[1]
        inputs = self._inputs(q, k, v, log_decay, beta, scale, None, None)
        _exact(states, "states", (states.shape[0],) + self.state_shape[1:], torch.float32, self.device)
        idx = _exact(slot_idx, "slot_idx", (self.nseq,), torch.int32, self.device)
        if out is None:
            o = torch.empty(self.rows, wv, dtype=self.tdtype, device=self.device)
            op, os = o.data_ptr(), wv
        else:
            o = out
            op, os = _rows(o, "out", self.rows, wv, self.tdtype, self.device)
        ssd_delta_rule_step(self.dims, inputs, states, states.shape[0], idx, op, os,
                            torch._C._cuda_getCurrentRawStream(self.device.index))
        return o


class BlockNormRunner:
    """The norms behind and before a block, joined with its gate, its scale and the residual stream, of one shape:

        h = residual + branch_scale * (x / rms(x) * post_weight) * silu(z),   y = h / rms(h) * pre_weight

    where post_norm, gate, residual and pre_norm say which parts there are; rms(v) = sqrt(mean(v^2) + eps) of a row.  x,
    z and y are (rows, channels) of ``dtype``, residual and h of ``residual_dtype`` ("f32" with either, default: dtype),
    rows possibly strided; weights and branch_scale (channels) fp32, each may be None (1)."""

    def __init__(self, rows: int, channels: int, *, post_norm: bool = False, gate: bool = False,
                 residual: bool = True, pre_norm: bool = True, dtype: str = "bf16", residual_dtype=None,
                 device="cuda"):
        self.rows, self.channels, self.device = rows, channels, _device(device)
        self.post_norm, self.gate, self.residual, self.pre_norm = bool(post_norm), bool(gate), bool(residual), bool(pre_norm)
        code, self.tdtype = _DTYPES[dtype]
        rcode, self.rdtype = _DTYPES[dtype if residual_dtype is None else residual_dtype]
        self.dims = SsdBlockNormDims(rows, channels, code, rcode, int(self.post_norm), int(self.gate),
                                     int(self.residual), int(self.pre_norm))
        self._size = ssd_block_norm_workspace_size(self.dims)
        if self._size == 0:
            raise ValueError("invalid dims for libssd")
        self.workspace = torch.empty(0, dtype=torch.uint8, device=self.device)  # of backward passes, from the first on
        self._stream = None  # the last one that used the workspace

    def _with(self, x, name, there: bool, dtype):
        """(address, row stride) of a tensor that goes with a part of the runner."""
        if (x is not None) != there:
            raise ValueError(f"{name}: {'needed' if there else 'not taken'} by this runner")
        return (None, 0) if x is None else _rows(x, name, self.rows, self.channels, dtype, self.device)

    def _inputs(self, x, z, residual, residual_there, post_weight, branch_scale, pre_weight, eps) -> SsdBlockNormInputs:
        device = self.device
        xp, xs = _rows(x, "x", self.rows, self.channels, self.tdtype, device)
        zp, zs = self._with(z, "z", self.gate, self.tdtype)
        rp, rs = self._with(residual, "residual", residual_there, self.rdtype)
        if (post_weight is not None and not self.post_norm) or (pre_weight is not None and not self.pre_norm):
            raise ValueError("post_weight goes with post_norm, pre_weight with pre_norm")
        shape, f32 = (self.channels,), torch.float32
        return SsdBlockNormInputs(xp, xs, zp, zs, rp, rs, _exact(post_weight, "post_weight", shape, f32, device),
                                  _exact(branch_scale, "branch_scale", shape, f32, device),
                                  _exact(pre_weight, "pre_weight", shape, f32, device), eps)

    def forward(self, x, *, residual=None, z=None, post_weight=None, branch_scale=None, pre_weight=None,
                eps: float = 1e-6, h_out=None, stream=None) -> dict:
        """h, y, rstd_post, rstd_pre (None where the runner has no such part); ``h_out``: a tensor for h, possibly the
        residual itself.  What backward needs besides the inputs: h, rstd_post, rstd_pre."""
        there = _elsewhere(self, stream)
        if there is not None:
            with there:
                return self.forward(x, residual=residual, z=z, post_weight=post_weight, branch_scale=branch_scale,
                                    pre_weight=pre_weight, eps=eps, h_out=h_out)
        inputs = self._inputs(x, z, residual, self.residual, post_weight, branch_scale, pre_weight, eps)
        empty, device = torch.empty, self.device
        if h_out is None:
            h = empty(x.shape, dtype=self.rdtype, device=device)
            hp, hs = h.data_ptr(), self.channels
        else:
            h = h_out
            hp, hs = _rows(h, "h_out", self.rows, self.channels, self.rdtype, device)
        y = empty(x.shape, dtype=self.tdtype, device=device) if self.pre_norm else None
        post = empty(self.rows, dtype=torch.float32, device=device) if self.post_norm else None
        pre = empty(self.rows, dtype=torch.float32, device=device) if self.pre_norm else None
        ssd_block_norm_forward(self.dims, inputs, hp, hs, y, self.channels, post, pre,
                               torch._C._cuda_getCurrentRawStream(device.index))
        return {"h": h, "y": y, "rstd_post": post, "rstd_pre": pre}

    def backward(self, x, h=None, *, dh=None, dy=None, z=None, post_weight=None, branch_scale=None, pre_weight=None,
                 rstd_post=None, rstd_pre=None, stream=None) -> dict:
        """Gradients of <dh, h> + <dy, y> (dh None: zero): dx, dz, dresidual, dpost_weight, dbranch_scale, dpre_weight,
        None where there is no such input (a weight that is None stands for a constant 1 and has no gradient)."""
        there = _elsewhere(self, stream)
        if there is not None:
            with there:
                return self.backward(x, h, dh=dh, dy=dy, z=z, post_weight=post_weight, branch_scale=branch_scale,
                                     pre_weight=pre_weight, rstd_post=rstd_post, rstd_pre=rstd_pre)
        inputs = self._inputs(x, z, None, False, post_weight, branch_scale, pre_weight, 0.0)
        hp, hs = self._with(h if self.pre_norm else None, "h", self.pre_norm, self.rdtype)
        dhp, dhs = self._with(dh, "dh", dh is not None, self.rdtype)
        dyp, dys = self._with(dy, "dy", self.pre_norm, self.tdtype)
        stat = (self.rows,)
        if (rstd_post is not None) != self.post_norm or (rstd_pre is not None) != self.pre_norm:
            raise ValueError("rstd_post goes with post_norm, rstd_pre with pre_norm")
        saved = SsdBlockNormSaved(hp, hs, dhp, dhs, dyp, dys,
                                  _exact(rstd_post, "rstd_post", stat, torch.float32, self.device),
                                  _exact(rstd_pre, "rstd_pre", stat, torch.float32, self.device))
        if self.workspace.numel() < self._size:
            self.workspace = torch.empty(self._size, dtype=torch.uint8, device=self.device)

        def rows(there, dtype):
            return torch.empty(x.shape, dtype=dtype, device=self.device) if there else None

        def weight(w):
            return None if w is None else torch.empty(self.channels, dtype=torch.float32, device=self.device)

        g = {"dx": rows(True, self.tdtype), "dz": rows(self.gate, self.tdtype),
             "dresidual": rows(self.residual, self.rdtype), "dpost_weight": weight(post_weight),
             "dbranch_scale": weight(branch_scale), "dpre_weight": weight(pre_weight)}
        c = self.channels
        grads = SsdBlockNormGrads(g["dx"].data_ptr(), c, _ptr(g["dz"]), c, _ptr(g["dresidual"]), c,
                                  _ptr(g["dpost_weight"]), _ptr(g["dbranch_scale"]), _ptr(g["dpre_weight"]))
        ssd_block_norm_backward(self.dims, inputs, saved, grads, self.workspace, stream=_current(self))
        return g
