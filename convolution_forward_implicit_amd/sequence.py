"""The sequence operators: the short causal depthwise convolution
(conv_causal_*) and the selective state space scan (conv_scan_*), each over
prompts, token by token, and with its gradient.  Argument marshalling only; the
computation and its definitions are in include/convfwd.h.
"""
from ctypes import byref

from . import capi


class _Plan:
    """What both operators share: the plan's life, tensor checks, the device."""

    _plan = None

    def describe(self):
        return self._describe(self._plan)

    def close(self):
        if self._plan:
            self._destroy(self._plan)
            self._plan = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _type(self, torch):
        return torch.float32 if self.dtype == "f32" else torch.bfloat16

    @staticmethod
    def _dense(t, shape, dtype, dev, name):
        """Address of a contiguous tensor of this shape and type on `dev`."""
        if t.dtype is dtype and t.get_device() == dev.index and t.shape == shape and t.is_contiguous():
            return t.data_ptr()
        if t.device != dev or dev.type != "cuda":
            raise ValueError("%s must be on the cuda device of the other tensors (%s), got %s" % (name, dev, t.device))
        if t.dtype != dtype:
            raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
        if t.shape != shape:
            raise ValueError("%s has shape %r, expected %r" % (name, tuple(t.shape), shape))
        raise ValueError("%s must be contiguous" % name)

    def _rows(self, t, lead, inner, dtype, dev, name):
        """(address, elements from token to token) of a tensor lead + inner
        whose rows are packed and evenly spaced: contiguous, or a range of the
        last dimensions of a contiguous one."""
        if t.is_contiguous():
            if t.dtype is dtype and t.get_device() == dev.index and t.shape == lead + inner:
                return t.data_ptr(), 0
            return self._dense(t, lead + inner, dtype, dev, name), 0
        if t.device != dev or dev.type != "cuda":
            raise ValueError("%s must be on the cuda device of the other tensors (%s), got %s" % (name, dev, t.device))
        if t.dtype != dtype:
            raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
        if t.shape != lead + inner:
            raise ValueError("%s has shape %r, expected %r" % (name, tuple(t.shape), lead + inner))
        st = t.stride()
        width = 1
        for d in range(len(inner) - 1, -1, -1):
            if inner[d] != 1 and st[len(lead) + d] != width:
                raise ValueError("%s: the elements of a token must be contiguous" % name)
            width *= inner[d]
        # the spacing of the rows, from the last leading dimension that has more than one
        ld, step = 0, 1
        for d in range(len(lead) - 1, -1, -1):
            if lead[d] != 1:
                if ld == 0:
                    ld = st[d] if step == 1 else 0
                if st[d] != ld * step or ld < width:
                    raise ValueError("%s: tokens must be evenly spaced rows (stride %r)" % (name, st))
            step *= lead[d]
        return t.data_ptr(), ld

    @staticmethod
    def _on(torch, dev, stream):
        """(stream handle, context): the stream to use, and, where it is not the
        current one of the current device, the context to allocate and launch in:
        memory that is released when a call returns belongs to the stream that
        used it."""
        if dev.type != "cuda":
            raise ValueError("tensors must be on a cuda device, got %s" % dev)
        if stream is None:
            if torch._C._cuda_getDevice() == dev.index:
                # the handle alone: building the Stream object takes as long as a launch
                return torch._C._cuda_getCurrentRawStream(dev.index), None
            stream = torch.cuda.current_stream(dev)
        elif stream.device != dev:
            raise ValueError("stream is of %s, the tensors are on %s" % (stream.device, dev))
        return stream.cuda_stream, torch.cuda.stream(stream)       # also makes its device the current one

    @staticmethod
    def _new(torch, like, shape, away):
        """An output: of the stream that writes it, whose earlier work alone may
        still hold its memory, and known to the caller's, which will read it."""
        if away is None:
            return like.new_empty(*shape)
        with away:
            t = like.new_empty(*shape)
        t.record_stream(torch.cuda.current_stream(like.device))
        return t


class CausalConv(_Plan):
    """A plan of the causal depthwise convolution.  `problem` is a dict {"N",
    "L", "C", "F"}: sequences, tokens, channels, taps (2 to 8)."""

    _describe = staticmethod(capi.conv_causal_describe)
    _destroy = staticmethod(capi.conv_causal_destroy)

    def __init__(self, problem, dtype, has_bias=False, silu=False):
        self.problem = dict(problem)
        self.dtype, dt = _dtype(dtype)
        self.has_bias, self.silu = bool(has_bias), bool(silu)
        N, L, C, F = (int(self.problem[k]) for k in ("N", "L", "C", "F"))
        self._plan = capi.conv_causal_create(capi.conv_causal_desc_t(dt, self.has_bias, self.silu, 0, N, L, C, F))
        self.x_shape = (N, L, C)
        self.w_shape = (C, F)
        self.b_shape = (C,)
        self.state_shape = (N, F - 1, C)
        self.bwd_workspace_bytes = capi.conv_causal_bwd_workspace_bytes(self._plan)

    def _bias(self, bias, t, dev):
        if self.has_bias != (bias is not None):
            raise ValueError("this plan has a bias" if self.has_bias else "this plan has no bias")
        return self._dense(bias, self.b_shape, t, dev, "bias") if self.has_bias else None

    def __call__(self, x, w, bias=None, state=None, lengths=None, out=None, state_out=None, stream=None):
        """y (N, L, C).  state (N, F - 1, C): the tokens before the first;
        lengths: int32 (N,); state_out: a tensor like state that receives the
        last F - 1 tokens.  x and out may be column ranges of wider tensors."""
        import torch
        t, dev = self._type(torch), x.device
        stream, away = self._on(torch, dev, stream)
        if out is None:
            out = self._new(torch, x, self.x_shape, away)
        lead, inner = self.x_shape[:2], self.x_shape[2:]
        xp, x_ld = self._rows(x, lead, inner, t, dev, "x")
        yp, y_ld = self._rows(out, lead, inner, t, dev, "out")
        args = capi.conv_causal_args_t(
            xp, self._dense(w, self.w_shape, t, dev, "w"), self._bias(bias, t, dev),
            None if state is None else self._dense(state, self.state_shape, t, dev, "state"),
            None if lengths is None else self._dense(lengths, self.x_shape[:1], torch.int32, dev, "lengths"), yp,
            None if state_out is None else self._dense(state_out, self.state_shape, t, dev, "state_out"), x_ld, y_ld)
        if away is None:
            capi.conv_causal_run(self._plan, byref(args), stream)
        else:
            with away:
                capi.conv_causal_run(self._plan, byref(args), stream)
        return out

    def step(self, x, w, state, bias=None, out=None, stream=None):
        """One token of every sequence: x and the returned y are (N, C); state
        (N, F - 1, C) moves on by one token, in place."""
        import torch
        t, dev = self._type(torch), x.device
        stream, away = self._on(torch, dev, stream)
        lead, inner = self.x_shape[:1], self.x_shape[2:]
        if out is None:
            out = self._new(torch, x, lead + inner, away)
        xp, x_ld = self._rows(x, lead, inner, t, dev, "x")
        yp, y_ld = self._rows(out, lead, inner, t, dev, "out")
        sp = self._dense(state, self.state_shape, t, dev, "state")
        args = capi.conv_causal_args_t(xp, self._dense(w, self.w_shape, t, dev, "w"), self._bias(bias, t, dev), sp, None,
                                       yp, sp, x_ld, y_ld)
        if away is None:
            capi.conv_causal_step(self._plan, byref(args), stream)
        else:
            with away:
                capi.conv_causal_step(self._plan, byref(args), stream)
        return out

    def backward(self, dy, x, w, bias=None, state=None, lengths=None, dstate_out=None, out=None, stream=None):
        """Gradients of <y, dy> + <state_out, dstate_out> as a dict of "dx",
        "dw", "dbias" and "dstate" (None without a bias or a state).  out: a
        dict of tensors to write some of them into."""
        import torch
        t, dev = self._type(torch), x.device
        stream, away = self._on(torch, dev, stream)
        got = {"dx": None, "dw": None, "dbias": None, "dstate": None}
        shapes = {"dx": self.x_shape, "dw": self.w_shape, "dbias": self.b_shape if self.has_bias else None,
                  "dstate": None if state is None else self.state_shape}
        _given(got, out, shapes)
        for k, shape in shapes.items():
            if shape is not None and got[k] is None:
                got[k] = self._new(torch, x, shape, away)
        lead, inner = self.x_shape[:2], self.x_shape[2:]
        dyp, dy_ld = self._rows(dy, lead, inner, t, dev, "dy")
        xp, x_ld = self._rows(x, lead, inner, t, dev, "x")
        dxp, dx_ld = self._rows(got["dx"], lead, inner, t, dev, "dx")
        like = lambda v, shape, name: None if v is None else self._dense(v, shape, t, dev, name)
        args = capi.conv_causal_bwd_args_t(
            dyp, xp, self._dense(w, self.w_shape, t, dev, "w"), self._bias(bias, t, dev),
            like(state, self.state_shape, "state"),
            None if lengths is None else self._dense(lengths, self.x_shape[:1], torch.int32, dev, "lengths"),
            like(dstate_out, self.state_shape, "dstate_out"), dxp, like(got["dw"], self.w_shape, "dw"),
            like(got["dbias"], self.b_shape, "dbias"), like(got["dstate"], self.state_shape, "dstate"), dy_ld, x_ld, dx_ld)
        _with_workspace(torch, self.bwd_workspace_bytes, dev, away, lambda ws, n: capi.conv_causal_bwd_run(
            self._plan, byref(args), ws, n, stream))
        return got


class SelectiveScan(_Plan):
    """A plan of the selective state space scan.  `problem` is a dict {"N", "L",
    "H", "P", "G", "S"}: sequences, tokens, heads, channels of a head, groups of
    heads with B and C in common, states of a channel (up to 128)."""

    _describe = staticmethod(capi.conv_scan_describe)
    _destroy = staticmethod(capi.conv_scan_destroy)

    def __init__(self, problem, dtype, softplus=True):
        self.problem = dict(problem)
        self.dtype, dt = _dtype(dtype)
        self.softplus = bool(softplus)
        N, L, H, P, G, S = (int(self.problem[k]) for k in ("N", "L", "H", "P", "G", "S"))
        self._plan = capi.conv_scan_create(capi.conv_scan_desc_t(dt, self.softplus, N, L, H, P, G, S))
        self.x_shape = (N, L, H, P)
        self.dt_shape = (N, L, H)
        self.b_shape = (N, L, G, S)
        self.a_shape = (H,)
        self.state_shape = (N, H, P, S)
        self.workspace_bytes = capi.conv_scan_workspace_bytes(self._plan)
        self.bwd_workspace_bytes = capi.conv_scan_bwd_workspace_bytes(self._plan)

    def _heads(self, v, name, torch, dev):
        return None if v is None else self._dense(v, self.a_shape, torch.float32, dev, name)

    def _state(self, v, name, torch, dev):
        return None if v is None else self._dense(v, self.state_shape, torch.float32, dev, name)

    def __call__(self, x, dt, A, B, C, D=None, dt_bias=None, state=None, lengths=None, out=None, state_out=None,
                 stream=None):
        """y (N, L, H, P) of x (N, L, H, P), dt (N, L, H), B and C (N, L, G, S)
        in the plan's dtype and A, D, dt_bias (H,) in float32.  state and
        state_out: float32 (N, H, P, S), before the first token and, written,
        behind the last; lengths: int32 (N,).  x, dt, B, C and out may be column
        ranges of wider tensors."""
        import torch
        t, dev = self._type(torch), x.device
        stream, away = self._on(torch, dev, stream)
        if out is None:
            out = self._new(torch, x, self.x_shape, away)
        lead = self.x_shape[:2]
        xp, x_ld = self._rows(x, lead, self.x_shape[2:], t, dev, "x")
        dp, dt_ld = self._rows(dt, lead, self.dt_shape[2:], t, dev, "dt")
        bp, b_ld = self._rows(B, lead, self.b_shape[2:], t, dev, "B")
        cp, c_ld = self._rows(C, lead, self.b_shape[2:], t, dev, "C")
        yp, y_ld = self._rows(out, lead, self.x_shape[2:], t, dev, "out")
        args = capi.conv_scan_args_t(
            xp, dp, self._dense(A, self.a_shape, torch.float32, dev, "A"), bp, cp, self._heads(D, "D", torch, dev),
            self._heads(dt_bias, "dt_bias", torch, dev), self._state(state, "state", torch, dev),
            None if lengths is None else self._dense(lengths, self.x_shape[:1], torch.int32, dev, "lengths"), yp,
            self._state(state_out, "state_out", torch, dev), x_ld, dt_ld, b_ld, c_ld, y_ld)
        _with_workspace(torch, self.workspace_bytes, dev, away, lambda ws, n: capi.conv_scan_run(
            self._plan, byref(args), ws, n, stream))
        return out

    def step(self, x, dt, A, B, C, state, D=None, dt_bias=None, out=None, stream=None):
        """One token of every sequence: x and the returned y (N, H, P), dt
        (N, H), B and C (N, G, S); state (N, H, P, S) is updated in place."""
        import torch
        t, dev = self._type(torch), x.device
        stream, away = self._on(torch, dev, stream)
        lead, hp, gs = self.x_shape[:1], self.x_shape[2:], self.b_shape[2:]
        if out is None:
            out = self._new(torch, x, lead + hp, away)
        xp, x_ld = self._rows(x, lead, hp, t, dev, "x")
        dp, dt_ld = self._rows(dt, lead, self.a_shape, t, dev, "dt")
        bp, b_ld = self._rows(B, lead, gs, t, dev, "B")
        cp, c_ld = self._rows(C, lead, gs, t, dev, "C")
        yp, y_ld = self._rows(out, lead, hp, t, dev, "out")
        sp = self._state(state, "state", torch, dev)
        args = capi.conv_scan_args_t(xp, dp, self._dense(A, self.a_shape, torch.float32, dev, "A"), bp, cp,
                                     self._heads(D, "D", torch, dev), self._heads(dt_bias, "dt_bias", torch, dev), sp,
                                     None, yp, sp, x_ld, dt_ld, b_ld, c_ld, y_ld)
        if away is None:
            capi.conv_scan_step(self._plan, byref(args), stream)
        else:
            with away:
                capi.conv_scan_step(self._plan, byref(args), stream)
        return out

    def backward(self, dy, x, dt, A, B, C, D=None, dt_bias=None, state=None, lengths=None, dstate_out=None, out=None,
                 stream=None):
        """Gradients of <y, dy> + <state_out, dstate_out> as a dict of "dx",
        "ddt", "dA", "dB", "dC", "dD", "ddt_bias" and "dstate" (None for inputs
        that are not given).  out: a dict of tensors to write some of them into;
        "dx", "dB" and "dC" may be column ranges of one tensor, the gradient of
        the convolution's output."""
        import torch
        t, dev, f32 = self._type(torch), x.device, torch.float32
        stream, away = self._on(torch, dev, stream)
        shapes = {"dx": self.x_shape, "ddt": self.dt_shape, "dA": self.a_shape, "dB": self.b_shape, "dC": self.b_shape,
                  "dD": None if D is None else self.a_shape, "ddt_bias": None if dt_bias is None else self.a_shape,
                  "dstate": None if state is None else self.state_shape}
        got = dict.fromkeys(shapes)
        _given(got, out, shapes)
        for k, shape in shapes.items():
            if shape is not None and got[k] is None:
                got[k] = self._new(torch, x if k in ("dx", "ddt", "dB", "dC") else A, shape, away)
        lead, hp, gs, hh = self.x_shape[:2], self.x_shape[2:], self.b_shape[2:], self.dt_shape[2:]
        rows = [self._rows(v, lead, inner, t, dev, name) for v, inner, name in (
            (dy, hp, "dy"), (x, hp, "x"), (dt, hh, "dt"), (B, gs, "B"), (C, gs, "C"),
            (got["dx"], hp, "dx"), (got["ddt"], hh, "ddt"), (got["dB"], gs, "dB"), (got["dC"], gs, "dC"))]
        (dyp, _), (xp, _), (dp, _), (bp, _), (cp, _), (dxp, _), (ddp, _), (dbp, _), (dcp, _) = rows
        args = capi.conv_scan_bwd_args_t(
            dyp, xp, dp, self._dense(A, self.a_shape, f32, dev, "A"), bp, cp, self._heads(D, "D", torch, dev),
            self._heads(dt_bias, "dt_bias", torch, dev), self._state(state, "state", torch, dev),
            None if lengths is None else self._dense(lengths, self.x_shape[:1], torch.int32, dev, "lengths"),
            self._state(dstate_out, "dstate_out", torch, dev), dxp, ddp, self._heads(got["dA"], "dA", torch, dev), dbp, dcp,
            self._heads(got["dD"], "dD", torch, dev), self._heads(got["ddt_bias"], "ddt_bias", torch, dev),
            self._state(got["dstate"], "dstate", torch, dev), *(ld for _, ld in rows))
        _with_workspace(torch, self.bwd_workspace_bytes, dev, away, lambda ws, n: capi.conv_scan_bwd_run(
            self._plan, byref(args), ws, n, stream))
        return got


def _dtype(dtype):
    """The name and the number of a type given by either; the library refuses a number it does not know."""
    number = capi.DTYPES[dtype] if isinstance(dtype, str) else int(dtype)
    return next((k for k, v in capi.DTYPES.items() if v == number), dtype), number


def _given(got, out, shapes):
    """Takes the caller's output tensors, which must be outputs of this call."""
    for k, v in (out or {}).items():
        if shapes.get(k) is None:
            raise ValueError("%r is not an output of this call" % (k,))
        got[k] = v


def _with_workspace(torch, nbytes, dev, away, run):
    """Runs `run(workspace, bytes)` with a workspace of this call's own, from
    torch's allocator on the stream that uses it (under graph capture from the
    graph's pool), so that calls on other streams or graphs share none."""
    if away is None:
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
        run(ws.data_ptr() if nbytes else None, nbytes)
    else:
        with away:
            ws = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
            run(ws.data_ptr() if nbytes else None, nbytes)
