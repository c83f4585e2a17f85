"""Rows in microscaled (MX) form and the experts that work on them (moe_mx_*,
moe_mx4_* and moe_experts_*_checkpoint in ``include/moe.h``).

Serving with 4-bit weights::

    gate, up, down = (moe_mx_quantize(w, "mxfp4") for w in (gate, up, down))
    experts = Mx4SwiGluExperts(gate, up, down, dtype=torch.bfloat16)
    y = experts.forward(x, logits, top_k=8, renormalize=True)

Training with activations kept in 8 bits::

    d = moe_dispatch(idx, num_experts=E, x=x)
    out, ckpt = experts.forward_checkpoint(d.x_disp, d.offsets)
    x_mx = moe_mx_quantize(x, "mxfp8")          # x, x_disp and out may go now
    ...
    dinput, dgate, dup, ddown = experts.backward_checkpoint(x_mx, d.perm, d.offsets, ckpt, dout, top_k)

All tensors of a call are contiguous and on one CUDA device, which need not be
the current one.  A call works on ``stream``, or on the current stream of that
device; what it allocates belongs to that stream.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass

import torch

from . import _lib
from ._lib import MoeError, check as _check
from .router_losses import _CODES, _I32, _buffer, _code, _load, _on, _p, _ws

_FORMATS = {"mxfp4": 0, "mxfp8": 1}
_U8 = (torch.uint8,)


def _format(name: str) -> int:
    code = _FORMATS.get(name)
    if code is None:
        raise MoeError(3, f"format must be 'mxfp4' or 'mxfp8' (got {name!r})")
    return code


def _shapes(shape, fmt: str):
    """Shapes of the values and the scales of rows of ``shape``."""
    *rows, cols = shape
    return (*rows, (cols + 1) // 2 if fmt == "mxfp4" else cols), (*rows, (cols + 31) // 32)


def _dense(t, what: str, device=None):
    if not t.is_cuda:
        raise ValueError(f"{what}: expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{what}: expected a contiguous tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{what} is on {t.device}, expected {device}")
    return t.data_ptr()


@dataclass
class MxRows:
    """Rows of ``cols`` values in blocks of 32 that share a power-of-two scale.
    ``format`` "mxfp4": two e2m1 elements a byte, the first in the low half;
    "mxfp8": e4m3 elements.  Scale bytes are exponents with a bias of 127."""
    values: torch.Tensor  # uint8 [..., ceil(cols/2)] or [..., cols]
    scales: torch.Tensor  # uint8 [..., ceil(cols/32)]
    format: str
    cols: int

    @classmethod
    def empty(cls, shape, format: str, device="cuda") -> "MxRows":
        _format(format)
        v, s = _shapes(shape, format)
        return cls(torch.empty(v, dtype=torch.uint8, device=device),
                   torch.empty(s, dtype=torch.uint8, device=device), format, shape[-1])

    @property
    def shape(self) -> tuple:
        return (*self.values.shape[:-1], self.cols)

    def _checked(self, what: str, shape=None, format=None, device=None):
        """Pointers of values and scales; ``shape`` and ``format`` as the call needs them.
        A call's rows are mostly like those of the call before: what was checked
        of them is remembered (not the tensors) and compared with what they are now."""
        v, s, d = self.values, self.scales, self.__dict__
        known = d.get("_known")
        if known is not None:
            fmt, cols, whole, vs, ss, index = known
            if (fmt == self.format and cols == self.cols
                    and (shape is None or whole == shape) and (format is None or fmt == format)
                    and v.shape == vs and s.shape == ss and v.dtype is torch.uint8 and s.dtype is torch.uint8
                    and v.is_contiguous() and s.is_contiguous() and v.get_device() == index
                    and s.get_device() == index and (device is None or device.index == index)):
                return v.data_ptr(), s.data_ptr()
        if format is not None and self.format != format:
            raise MoeError(3, f"{what} must be {format} (got {self.format})")
        _format(self.format)
        whole = torch.Size(self.shape)
        if shape is not None and whole != tuple(shape):
            raise MoeError(2, f"{what} must have shape {tuple(shape)} (got {tuple(whole)})")
        device = v.device if device is None else device
        if not v.is_cuda:
            raise ValueError(f"{what}.values: expected a CUDA tensor")
        vs, ss = _shapes(whole, self.format)
        got = (_p(v, f"{what}.values", _U8, vs, device), _p(s, f"{what}.scales", _U8, ss, device))
        d["_known"] = (self.format, self.cols, whole, v.shape, s.shape, v.get_device())
        return got


def moe_mx_quantize(x: torch.Tensor, format: str, out: MxRows | None = None, stream=None) -> MxRows:
    """Rows of x [..., C] (F32/F16/BF16) in "mxfp4" or "mxfp8" form."""
    lib = _load()
    fmt = _format(format)
    shape = x.shape
    if len(shape) < 1:
        raise MoeError(2, "x must have at least one dimension")
    code, xp, dev = _code(x, "x"), _dense(x, "x"), x.device
    C = shape[-1]
    R = x.numel() // C if C else 0
    current, raw = _on(dev, stream)
    with current:
        if out is None:
            out = MxRows.empty(shape, format, dev)
        v, s = out._checked("out", shape, format, dev)
        _check(lib.moe_mx_quantize(xp, code, R, C, fmt, v, s, raw))
    return out


def moe_mx_dequantize(mx: MxRows, dtype: torch.dtype, perm: torch.Tensor | None = None, top_k: int = 1,
                      out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The values of ``mx`` [..., C] in ``dtype``; with ``perm`` [N] (int32) rows
    in dispatch order [N, C], row r the token perm[r] // top_k of mx [T, C]."""
    lib = _load()
    fmt = _format(mx.format)
    v, s = mx._checked("mx")
    shape = mx.__dict__["_known"][2]
    dev, C = mx.values.device, mx.cols
    R = shape[:-1].numel()
    code = _CODES.get(dtype)
    if code is None:
        raise MoeError(3, f"dtype {dtype} is not F32/F16/BF16")
    if perm is None:
        n, pp = R, None
    else:
        if len(shape) != 2 or perm.dim() != 1:
            raise MoeError(2, "perm [N] needs rows [T, C]")
        n = perm.shape[0]
        shape, pp = torch.Size((n, C)), _p(perm, "perm", _I32, (n,), dev)
    current, raw = _on(dev, stream)
    with current:
        if out is None:
            out = torch.empty(shape, dtype=dtype, device=dev)
        _check(lib.moe_mx_dequantize(v, s, fmt, R, C, pp, top_k, n, _p(out, "out", (dtype,), shape, dev),
                                     code, raw))
    return out


class Mx4SwiGluExperts:
    """Bias-free SwiGLU experts on 4-bit operands: gate and up [E,I,H], down
    [E,H,I] in "mxfp4" form; rows x and the outputs in ``dtype`` (float16 or
    bfloat16), rounded to 4 bits on the way in and between the products.  The
    object keeps the weights' values and its own re-ordered copy of the scales
    alive; the scales it was given may go.  The re-ordering is enqueued on
    ``stream`` (or the current one): calls on other streams have to be ordered
    behind it.  When the object goes, its memory is handed out again only after
    what its calls have enqueued by then, on whichever streams; a graph that was
    captured needs the object for as long as it is replayed."""

    def __init__(self, gate: MxRows, up: MxRows, down: MxRows, dtype: torch.dtype = torch.bfloat16, stream=None):
        self.handle = None
        self._lib = lib = _load()
        if gate.values.dim() != 3:
            raise MoeError(2, "4-bit expert weights must be rank-three rows")
        E, I, H = gate.shape
        dev = gate.values.device
        ptrs = (*gate._checked("gate", (E, I, H), "mxfp4", dev), *up._checked("up", (E, I, H), "mxfp4", dev),
                *down._checked("down", (E, H, I), "mxfp4", dev))
        if dtype not in _CODES:
            raise MoeError(3, f"dtype {dtype} is not F16/BF16")
        self.E, self.I, self.H, self.dtype, self.device = E, I, H, dtype, dev
        h = ctypes.c_void_p()
        current, raw = _on(dev, stream)
        with current:
            scales = _buffer(lib.moe_mx4_experts_scale_bytes(E, I, H), dev)
            _check(lib.moe_mx4_experts_create(*ptrs, _CODES[dtype], E, I, H, scales.data_ptr(), scales.nbytes, raw,
                                              ctypes.byref(h)))
        self._keep = (gate.values, up.values, down.values, scales)
        self._streams = set()
        self._read_on(stream, raw)
        for m in (gate, up, down):  # read by the re-ordering
            m.scales.record_stream(stream or torch.cuda.current_stream(dev))
        self.handle = h

    def __del__(self):
        if getattr(self, "handle", None) is not None:
            self._lib.moe_mx4_experts_destroy(self.handle)
            self.handle = None

    def _read_on(self, stream, raw):
        """Notes a stream that a call reads the weights on: what that stream holds when
        they are freed comes before another use of their memory."""
        if raw not in self._streams:
            self._streams.add(raw)
            for t in self._keep:
                t.record_stream(stream or torch.cuda.current_stream(self.device))

    def workspace(self, N: int) -> torch.Tensor:
        """A workspace for forward_dispatched of up to N rows."""
        return _buffer(self._lib.moe_mx4_experts_workspace_size(self.handle, N), self.device)

    def forward_workspace(self, T: int, top_k: int, logits_dtype=torch.bfloat16) -> torch.Tensor:
        return _buffer(self._lib.moe_mx4_forward_workspace_size(self.handle, T, top_k, _CODES[logits_dtype]),
                       self.device)

    def forward_dispatched(self, x_disp: torch.Tensor, offsets: torch.Tensor, out=None, workspace=None,
                           stream=None) -> torch.Tensor:
        """Expert outputs [N,H] of dispatched rows x_disp [N,H]."""
        dev, dt = self.device, (self.dtype,)
        if x_disp.dim() != 2:
            raise MoeError(2, "x_disp must be [N, H]")
        N = x_disp.shape[0]
        args = (_p(x_disp, "x_disp", dt, (N, self.H), dev), N, _p(offsets, "offsets", _I32, (self.E + 1,), dev))
        current, raw = _on(dev, stream)
        with current:
            if out is None:
                out = torch.empty((N, self.H), dtype=self.dtype, device=dev)
            if workspace is None:
                workspace = self.workspace(N)
            self._read_on(stream, raw)
            _check(self._lib.moe_mx4_experts_forward(self.handle, *args, _p(out, "out", dt, (N, self.H), dev),
                                                     *_ws(workspace, dev), raw))
        return out

    def _forward(self, call, x, logits, top_k, route, y, workspace, stream):
        dev, dt = self.device, (self.dtype,)
        if x.dim() != 2:
            raise MoeError(2, "x must be [T, H]")
        T = x.shape[0]
        code = _code(logits, "logits")
        xp = _p(x, "x", dt, (T, self.H), dev)
        lp = _p(logits, "logits", (logits.dtype,), (T, self.E), dev)
        current, raw = _on(dev, stream)
        with current:
            if y is None:
                y = torch.empty((T, self.H), dtype=self.dtype, device=dev)
            if workspace is None:
                workspace = self.forward_workspace(T, top_k, logits.dtype)
            self._read_on(stream, raw)
            _check(call(self.handle, xp, lp, code, T, *route, _p(y, "y", dt, (T, self.H), dev),
                        *_ws(workspace, dev), raw))
        return y

    def forward(self, x: torch.Tensor, logits: torch.Tensor, top_k: int, renormalize: bool, y=None,
                workspace=None, stream=None) -> torch.Tensor:
        """Fused route -> dispatch -> 4-bit experts -> combine, as SwiGluExperts.forward."""
        return self._forward(self._lib.moe_mx4_forward, x, logits, top_k, (top_k, int(bool(renormalize))), y,
                             workspace, stream)

    def forward_sigmoid_grouped(self, x: torch.Tensor, logits: torch.Tensor, top_k: int, groups: int,
                                selected_groups: int, group_top_two: bool, renormalize: bool, scale: float = 1.0,
                                bias: torch.Tensor | None = None, y=None, workspace=None,
                                stream=None) -> torch.Tensor:
        """The fused forward with sigmoid group-limited routing, as
        SwiGluExperts.forward_sigmoid_grouped."""
        opt = _lib.GroupRoutingOptions(top_k, groups, selected_groups, int(bool(group_top_two)),
                                       int(bool(renormalize)), float(scale))
        bp = _p(bias, "bias", (torch.float32,), (self.E,), self.device)
        return self._forward(self._lib.moe_mx4_forward_sigmoid_grouped, x, logits, top_k, (bp, ctypes.byref(opt)),
                             y, workspace, stream)


@dataclass
class ExpertCheckpoint:
    """What the experts' backward needs of the forward, in 8 bits: the gate and
    up projections [N,I] of the dispatched rows."""
    gate: MxRows
    up: MxRows

    @classmethod
    def empty(cls, N: int, I: int, device="cuda") -> "ExpertCheckpoint":
        return cls(MxRows.empty((N, I), "mxfp8", device), MxRows.empty((N, I), "mxfp8", device))

    def _checked(self, N, I, dev):
        return (*self.gate._checked("checkpoint.gate", (N, I), "mxfp8", dev),
                *self.up._checked("checkpoint.up", (N, I), "mxfp8", dev))
