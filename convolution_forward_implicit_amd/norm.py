"""The group norm with an activation, channels innermost (conv_gnorm_*), and its
gradient.  Argument marshalling only; the computation and its definition are in
include/convfwd.h.
"""
from ctypes import byref

from . import capi
from .sequence import _dtype, _given, _Plan, _with_workspace


class GroupNorm(_Plan):
    """A plan of the group norm.  `problem` is a dict {"N", "L", "G", "C"}: samples,
    pixels or tokens of a sample, groups, channels of a group.  act: "none", "silu"
    or "gelu", of the result or, with gated=True, of the gate that it is multiplied
    by; center=False leaves the mean in (a norm by the root of the mean square);
    per_token=True takes the statistics of each token by itself."""

    _describe = staticmethod(capi.conv_gnorm_describe)
    _destroy = staticmethod(capi.conv_gnorm_destroy)

    def __init__(self, problem, dtype, act="none", has_bias=False, gated=False, center=True, per_token=False, eps=1e-5):
        self.problem = dict(problem)
        self.dtype, dt = _dtype(dtype)
        if act not in capi.NORM_ACTS:
            raise ValueError("act must be one of %s, got %r" % (", ".join(capi.NORM_ACTS), act))
        self.act, self.eps = act, float(eps)
        self.has_bias, self.gated, self.center, self.per_token = bool(has_bias), bool(gated), bool(center), bool(per_token)
        N, L, G, C = (int(self.problem[k]) for k in ("N", "L", "G", "C"))
        self._plan = capi.conv_gnorm_create(capi.conv_gnorm_desc_t(
            dt, capi.NORM_ACTS[act], self.has_bias, self.gated, self.center, self.per_token, N, L, G, C, self.eps))
        self.x_shape = (N, L, G, C)
        self.w_shape = (G, C)
        self.workspace_bytes = capi.conv_gnorm_workspace_bytes(self._plan)
        self.bwd_workspace_bytes = capi.conv_gnorm_bwd_workspace_bytes(self._plan)

    def _weights(self, w, bias, t, dev):
        if self.has_bias != (bias is not None):
            raise ValueError("this plan has a bias" if self.has_bias else "this plan has no bias")
        return (self._dense(w, self.w_shape, t, dev, "w"),
                self._dense(bias, self.w_shape, t, dev, "bias") if self.has_bias else None)

    def _gate(self, gate, t, dev):
        if self.gated != (gate is not None):
            raise ValueError("this plan has a gate" if self.gated else "this plan has no gate")
        return self._rows(gate, self.x_shape[:2], self.x_shape[2:], t, dev, "gate") if self.gated else (None, 0)

    def __call__(self, x, w, bias=None, gate=None, lengths=None, out=None, stream=None):
        """y (N, L, G, C) of x; w and bias (G, C); gate like x; lengths: int32 (N,).
        x, gate and out may be column ranges of wider tensors."""
        import torch
        t, dev = self._type(torch), x.device
        stream, away = self._on(torch, dev, stream)
        if out is None:
            out = self._new(torch, x, self.x_shape, away)
        lead, inner = self.x_shape[:2], self.x_shape[2:]
        xp, x_ld = self._rows(x, lead, inner, t, dev, "x")
        yp, y_ld = self._rows(out, lead, inner, t, dev, "out")
        gp, gate_ld = self._gate(gate, t, dev)
        args = capi.conv_gnorm_args_t(
            xp, *self._weights(w, bias, t, dev), gp,
            None if lengths is None else self._dense(lengths, self.x_shape[:1], torch.int32, dev, "lengths"), yp, x_ld,
            gate_ld, y_ld)
        _with_workspace(torch, self.workspace_bytes, dev, away, lambda ws, n: capi.conv_gnorm_run(
            self._plan, byref(args), ws, n, stream))
        return out

    def backward(self, dy, x, w, bias=None, gate=None, lengths=None, out=None, stream=None):
        """Gradients of <y, dy> as a dict of "dx", "dw", "dbias" and "dgate" (None
        without a bias or a gate).  out: a dict of tensors to write some of them
        into; "dx" and "dgate" may be column ranges."""
        import torch
        t, dev = self._type(torch), x.device
        stream, away = self._on(torch, dev, stream)
        shapes = {"dx": self.x_shape, "dw": self.w_shape, "dbias": self.w_shape if self.has_bias else None,
                  "dgate": self.x_shape if self.gated else None}
        got = dict.fromkeys(shapes)
        _given(got, out, shapes)
        for k, shape in shapes.items():
            if shape is not None and got[k] is None:
                got[k] = self._new(torch, x, shape, away)
        lead, inner = self.x_shape[:2], self.x_shape[2:]
        dyp, dy_ld = self._rows(dy, lead, inner, t, dev, "dy")
        xp, x_ld = self._rows(x, lead, inner, t, dev, "x")
        gp, gate_ld = self._gate(gate, t, dev)
        dxp, dx_ld = self._rows(got["dx"], lead, inner, t, dev, "dx")
        dgp, dgate_ld = self._rows(got["dgate"], lead, inner, t, dev, "dgate") if self.gated else (None, 0)
        args = capi.conv_gnorm_bwd_args_t(
            dyp, xp, *self._weights(w, bias, t, dev), gp,
            None if lengths is None else self._dense(lengths, self.x_shape[:1], torch.int32, dev, "lengths"), dxp,
            self._dense(got["dw"], self.w_shape, t, dev, "dw"),
            self._dense(got["dbias"], self.w_shape, t, dev, "dbias") if self.has_bias else None, dgp,
            dy_ld, x_ld, gate_ld, dx_ld, dgate_ld)
        _with_workspace(torch, self.bwd_workspace_bytes, dev, away, lambda ws, n: capi.conv_gnorm_bwd_run(
            self._plan, byref(args), ws, n, stream))
        return got
