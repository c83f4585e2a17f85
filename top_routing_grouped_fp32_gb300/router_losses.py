"""Training losses of the router: balance loss with expert counts and z-loss,
and distillation from a teacher's top logits (moe_balance_loss*,
moe_distill_* in ``include/moe.h``).

A router's training step, next to the gradient of the routing weights::

    idx, w = moe_route(logits, top_k=6, renormalize=False)
    bal = moe_balance_loss(logits, idx, z_loss=True)             # bal.loss [S], bal.counts [S,E]
    tgt = moe_distill_targets(teacher_logits, top_m=8)
    dis = moe_distill_loss(logits, tgt)                          # dis.loss [S], dis.row_loss [T]
    ...
    dl = moe_router_backward(logits, idx, dweights, "softmax", False)
    moe_balance_loss_backward(logits, bal, 6, dloss, dz_loss=dz, base=dl, dlogits=dl)
    moe_distill_loss_backward(logits, tgt, dis, ddistill, base=dl, dlogits=dl)

All tensors of a call are contiguous and on one CUDA device, which need not be
the current one.  A call works on ``stream``, or on the current stream of that
device; what it allocates belongs to that stream.  ``out`` is a result of an
earlier call of the same sizes to write into; ``workspace`` a buffer from the
``*_workspace`` function to work in (calls that may overlap need one each).
"""
from __future__ import annotations

import contextlib
import ctypes
from dataclasses import dataclass

import torch

from . import _lib
from ._lib import MoeError, check as _check

_CODES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
_SCORING = {"softmax": 0, "sigmoid": 1}
_F32, _I32 = (torch.float32,), (torch.int32,)
_MASK = (torch.bool, torch.uint8)
_NOTHING = contextlib.nullcontext()
# what the backwards read of a forward's results
_BALANCE_READS = ("counts", "tokens", "row_stats")
_DISTILL_READS = ("tokens", "row_stats")
_LIST_READS = ("idx", "logits")


def _code(t: torch.Tensor, what: str) -> int:
    code = _CODES.get(t.dtype)
    if code is None:
        raise MoeError(3, f"{what} dtype {t.dtype} is not F32/F16/BF16")
    return code


def _scoring(name: str) -> int:
    code = _SCORING.get(name)
    if code is None:
        raise MoeError(1, f"scoring must be 'softmax' or 'sigmoid' (got {name!r})")
    return code


def _rows_of(logits: torch.Tensor, what: str):
    """T, E, type code, data pointer and device of the rows of a call, which its
    other tensors are checked against."""
    shape = logits.shape
    if len(shape) != 2:
        raise MoeError(2, f"{what} must have rank two (got {len(shape)})")
    if not logits.is_cuda:
        raise ValueError(f"{what}: expected a CUDA tensor")
    code = _code(logits, what)
    if not logits.is_contiguous():
        raise ValueError(f"{what}: expected a contiguous tensor")
    return (*shape, code, logits.data_ptr(), logits.device)


def _p(t, what: str, dtypes, shape, device):
    """Data pointer of a checked tensor (None passes)."""
    if t is None:
        return None
    if t.dtype in dtypes and t.shape == shape and t.device == device and t.is_contiguous():
        return t.data_ptr()
    if t.dtype not in dtypes:
        raise MoeError(3, f"{what} dtype {t.dtype} is not one of {', '.join(str(d) for d in dtypes)}")
    if t.shape != shape:
        raise MoeError(2, f"{what} must have shape {tuple(shape)} (got {tuple(t.shape)})")
    if t.device != device:
        raise ValueError(f"{what} is on {t.device}, the call's other tensors are on {device}")
    raise ValueError(f"{what}: expected a contiguous tensor")


class _Checked:
    """Tensors that a call writes or hands on; a training step passes them call
    after call.  What was checked of each is remembered, and each call compares
    it with what the tensor is then (its memory can be exchanged behind it, by
    ``.data``, ``set_`` or an in-place transpose): a difference is checked anew."""

    def __setattr__(self, name, value):
        self.__dict__[name] = value
        if name != "workspace":
            self.__dict__["_checked"] = {}

    def _pointers(self, device, *sizes, of=None):
        """Data pointers of _tensors(*sizes) in their order (of those named in `of`)."""
        d = self.__dict__
        known = d["_checked"].get(of)
        if known is not None and known[0] == sizes and known[1] == device:
            out = []
            for t, dtype, flat, size, index in known[2]:
                if t is None:
                    out.append(None)
                elif (t.dtype is dtype and (t.nbytes if flat else t.shape) == size and t.get_device() == index
                        and t.is_contiguous()):
                    out.append(t.data_ptr())
                else:
                    break
            else:
                return out
        named = [x for x in self._tensors(*sizes) if of is None or x[0] in of]
        out = [_p(d[n], n, dtypes, shape, device) for n, dtypes, shape in named]
        # (a vector's bytes in a row are the same vector in every shape)
        d["_checked"][of] = (sizes, device, [
            (None,) * 5 if t is None else
            (t, t.dtype, t.dim() == 1, t.nbytes if t.dim() == 1 else t.shape, t.get_device())
            for t in (d[n] for n, _, _ in named)])
        return out


def _ws(t, device):
    if t.device != device or not t.is_contiguous():
        raise ValueError(f"workspace: expected a contiguous tensor on {device}")
    return t.data_ptr(), t.nbytes


def _same_temperature(kept, temperature, what: str) -> None:
    """`kept`: the temperature that `what` was made at (None: not known)."""
    if kept is not None and ctypes.c_float(kept).value != ctypes.c_float(temperature).value:  # what the library gets
        raise MoeError(1, f"temperature is {temperature}, {what} was made at {kept}")


def _num_seqs(seq_offsets) -> int:
    if seq_offsets.dim() != 1 or seq_offsets.shape[0] < 2:
        raise MoeError(2, "seq_offsets must be [num_seqs + 1] with num_seqs >= 1")
    return seq_offsets.shape[0] - 1


# the current device, and the current stream's handle without a Stream object around
# it, where torch offers them (CUDA is initialised: the tensors are on a device)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                              lambda index: torch.cuda.current_stream(index).cuda_stream)


def _on(device: torch.device, stream):
    """A context in which `device` and `stream` (None: the device's current one)
    are current, and the stream's handle."""
    if stream is not None:
        if stream.device != device:
            raise ValueError(f"stream is on {stream.device}, the call's tensors are on {device}")
        return torch.cuda.stream(stream), stream.cuda_stream
    index = device.index
    return _NOTHING if _current_device() == index else torch.cuda.device(device), _current_raw_stream(index)


_lib_handle = None


def _load():
    global _lib_handle
    if _lib_handle is None:
        _lib_handle = _lib.load()
    return _lib_handle


def _buffer(nbytes: int, device) -> torch.Tensor:
    # torch allocations are 512-byte aligned, above the ABI's 256-byte rule
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


@dataclass
class BalanceLoss(_Checked):
    """What moe_balance_loss gives and moe_balance_loss_backward takes (it reads
    counts, tokens and row_stats)."""
    loss: torch.Tensor                # float32 [S]
    z_loss: torch.Tensor | None       # float32 [S]
    mean_scores: torch.Tensor | None  # float32 [S,E]
    counts: torch.Tensor              # int32 [S,E]
    tokens: torch.Tensor              # int32 [S]
    row_stats: torch.Tensor           # float32 [T,2]
    workspace: torch.Tensor | None = None  # holds the device status word

    @classmethod
    def empty(cls, T: int, E: int, num_seqs: int, device, z_loss: bool = False) -> "BalanceLoss":
        def f32(*shape):
            return torch.empty(shape, dtype=torch.float32, device=device)

        def i32(*shape):
            return torch.empty(shape, dtype=torch.int32, device=device)
        S = num_seqs
        return cls(f32(S), f32(S) if z_loss else None, f32(S, E), i32(S, E), i32(S), f32(T, 2))

    @staticmethod
    def _tensors(T, E, S):
        return (("loss", _F32, (S,)), ("z_loss", _F32, (S,)), ("mean_scores", _F32, (S, E)),
                ("counts", _I32, (S, E)), ("tokens", _I32, (S,)), ("row_stats", _F32, (T, 2)))


def moe_balance_loss_workspace(T: int, E: int, num_seqs: int = 1, device="cuda") -> torch.Tensor:
    return _buffer(_load().moe_balance_loss_workspace_size(T, E, num_seqs), device)


def moe_balance_loss(logits: torch.Tensor, idx: torch.Tensor, scoring: str = "softmax",
                     token_mask: torch.Tensor | None = None, seq_offsets: torch.Tensor | None = None,
                     z_loss: bool = False, out: BalanceLoss | None = None,
                     workspace: torch.Tensor | None = None, stream=None) -> BalanceLoss:
    """Balance loss, per-expert counts, mean scores and (``z_loss``) the z-loss
    of router logits [T,E] and their routed experts idx [T,k] (int32)."""
    lib = _load()
    T, E, code, rows, dev = _rows_of(logits, "logits")
    sc = _scoring(scoring)
    if idx.dim() != 2:
        raise MoeError(2, "idx must be [T, top_k]")
    k, S = idx.shape[1], 1 if seq_offsets is None else _num_seqs(seq_offsets)
    args = (rows, code, _p(idx, "idx", _I32, (T, k), dev),
            _p(token_mask, "token_mask", _MASK, (T,), dev), _p(seq_offsets, "seq_offsets", _I32, (S + 1,), dev),
            T, E, k, S, sc)
    current, raw = _on(dev, stream)
    with current:
        if out is None:
            out = BalanceLoss.empty(T, E, S, dev, z_loss)
        elif (out.z_loss is not None) != z_loss:
            raise MoeError(1, "out was made with another z_loss")
        if workspace is None:
            workspace = moe_balance_loss_workspace(T, E, S, dev)
        out.__dict__["workspace"] = workspace
        ws, nbytes = _ws(workspace, dev)
        _check(lib.moe_balance_loss(*args, *out._pointers(dev, T, E, S), ws, nbytes, raw))
    return out


def moe_balance_loss_backward(logits: torch.Tensor, forward: BalanceLoss, top_k: int, dloss: torch.Tensor,
                              scoring: str = "softmax", seq_offsets: torch.Tensor | None = None,
                              dz_loss: torch.Tensor | None = None, base: torch.Tensor | None = None,
                              dlogits: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """dlogits [T,E] = base + gradient of sum(dloss * loss) (+ sum(dz_loss *
    z_loss)), dloss and dz_loss float32 [S].  ``dlogits`` is written if given
    (it may be ``base``)."""
    lib = _load()
    T, E, code, rows, dev = _rows_of(logits, "logits")
    sc, S, dt = _scoring(scoring), 1 if seq_offsets is None else _num_seqs(seq_offsets), (logits.dtype,)
    counts, tokens, row_stats = forward._pointers(dev, T, E, S, of=_BALANCE_READS)
    args = (rows, code, row_stats, counts, tokens,
            _p(seq_offsets, "seq_offsets", _I32, (S + 1,), dev), T, E, top_k, S, sc,
            _p(dloss, "dloss", _F32, (S,), dev), _p(dz_loss, "dz_loss", _F32, (S,), dev),
            _p(base, "base", dt, (T, E), dev))
    current, raw = _on(dev, stream)
    with current:
        if dlogits is None:
            dlogits = torch.empty((T, E), dtype=logits.dtype, device=dev)
        _check(lib.moe_balance_loss_backward(*args, _p(dlogits, "dlogits", dt, (T, E), dev),
                                             raw))
    return dlogits


@dataclass
class DistillTargets(_Checked):
    """A teacher's top logits: what moe_distill_targets gives and the
    distillation loss takes.  ``rest`` may be None: no mass outside the list.  A
    rest belongs to the temperature that it was summed at, which moe_distill_targets
    notes here (another ``rest`` in its place: not known)."""
    idx: torch.Tensor           # int32 [T,m]
    logits: torch.Tensor        # [T,m] in the teacher's dtype
    rest: torch.Tensor | None   # float32 [T]
    temperature: float | None = None

    def __setattr__(self, name, value):
        super().__setattr__(name, value)
        if name == "rest":
            self.__dict__["temperature"] = None

    @classmethod
    def empty(cls, T: int, top_m: int, dtype, device) -> "DistillTargets":
        return cls(torch.empty((T, top_m), dtype=torch.int32, device=device),
                   torch.empty((T, top_m), dtype=dtype, device=device),
                   torch.empty((T,), dtype=torch.float32, device=device))

    def _tensors(self, T, m):
        return ("idx", _I32, (T, m)), ("logits", (self.logits.dtype,), (T, m)), ("rest", _F32, (T,))


def moe_distill_targets(teacher_logits: torch.Tensor, top_m: int, temperature: float = 1.0,
                        out: DistillTargets | None = None, stream=None) -> DistillTargets:
    """The top_m largest of each row of a teacher's logits [T,E] and the logit of
    all its other experts together at ``temperature``."""
    lib = _load()
    T, E, code, rows, dev = _rows_of(teacher_logits, "teacher_logits")
    dt = teacher_logits.dtype
    if out is None and not 1 <= top_m <= E:
        raise MoeError(1, f"top_m must satisfy 1 <= top_m <= E (top_m={top_m}, E={E})")
    current, raw = _on(dev, stream)
    with current:
        if out is None:
            out = DistillTargets.empty(T, top_m, dt, dev)
        if out.rest is None:
            raise MoeError(1, "out has no rest")
        if out.logits.dtype != dt:
            raise MoeError(3, f"out.logits dtype {out.logits.dtype} is not the teacher logits' {dt}")
        _check(lib.moe_distill_targets(rows, code, T, E, top_m,
                                       temperature, *out._pointers(dev, T, top_m), raw))
    out.__dict__["temperature"] = temperature
    return out


@dataclass
class DistillLoss(_Checked):
    """What moe_distill_loss gives and moe_distill_loss_backward takes (it reads
    tokens and row_stats, which belong to a temperature as a teacher's rest does)."""
    loss: torch.Tensor       # float32 [S]
    tokens: torch.Tensor     # int32 [S]
    row_loss: torch.Tensor   # float32 [T]
    row_stats: torch.Tensor  # float32 [5,T]
    workspace: torch.Tensor | None = None  # holds the device status word
    temperature: float | None = None

    def __setattr__(self, name, value):
        super().__setattr__(name, value)
        if name == "row_stats":
            self.__dict__["temperature"] = None

    @classmethod
    def empty(cls, T: int, num_seqs: int, device) -> "DistillLoss":
        def f32(*shape):
            return torch.empty(shape, dtype=torch.float32, device=device)
        return cls(f32(num_seqs), torch.empty((num_seqs,), dtype=torch.int32, device=device), f32(T), f32(5, T))

    @staticmethod
    def _tensors(T, S):
        return ("loss", _F32, (S,)), ("tokens", _I32, (S,)), ("row_loss", _F32, (T,)), ("row_stats", _F32, (5, T))


def _list_args(targets: DistillTargets, T: int, dev, of=None):
    shape = targets.idx.shape
    if len(shape) != 2:
        raise MoeError(2, "targets.idx must be [T, top_m]")
    m = shape[1]
    idx, logits, *rest = targets._pointers(dev, T, m, of=of)
    return m, (idx, logits, _code(targets.logits, "targets.logits")), *rest


def moe_distill_loss_workspace(T: int, num_seqs: int = 1, device="cuda") -> torch.Tensor:
    return _buffer(_load().moe_distill_loss_workspace_size(T, num_seqs), device)


def moe_distill_loss(logits: torch.Tensor, targets: DistillTargets, temperature: float = 1.0,
                     token_mask: torch.Tensor | None = None, seq_offsets: torch.Tensor | None = None,
                     out: DistillLoss | None = None, workspace: torch.Tensor | None = None,
                     stream=None) -> DistillLoss:
    """Mean KL divergence of student logits [T,E] from a teacher's lists, at the
    temperature of their rest."""
    lib = _load()
    T, E, code, rows, dev = _rows_of(logits, "logits")
    kept = targets.temperature
    if kept is not None and kept != temperature and targets.rest is not None:
        _same_temperature(kept, temperature, "the teacher's rest")
    S = 1 if seq_offsets is None else _num_seqs(seq_offsets)
    m, lists, rest = _list_args(targets, T, dev)
    args = (rows, code, *lists, rest, _p(token_mask, "token_mask", _MASK, (T,), dev),
            _p(seq_offsets, "seq_offsets", _I32, (S + 1,), dev), T, E, m, S, temperature)
    current, raw = _on(dev, stream)
    with current:
        if out is None:
            out = DistillLoss.empty(T, S, dev)
        if workspace is None:
            workspace = moe_distill_loss_workspace(T, S, dev)
        out.__dict__["workspace"] = workspace
        ws, nbytes = _ws(workspace, dev)
        _check(lib.moe_distill_loss(*args, *out._pointers(dev, T, S), ws, nbytes, raw))
    out.__dict__["temperature"] = temperature
    return out


def moe_distill_loss_backward(logits: torch.Tensor, targets: DistillTargets, forward: DistillLoss,
                              dloss: torch.Tensor, temperature: float = 1.0,
                              seq_offsets: torch.Tensor | None = None, base: torch.Tensor | None = None,
                              dlogits: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """dlogits [T,E] = base + gradient of sum(dloss * loss), dloss float32 [S], at
    the forward's temperature.  ``dlogits`` is written if given (it may be ``base``)."""
    lib = _load()
    T, E, code, rows, dev = _rows_of(logits, "logits")
    kept = forward.temperature
    if kept is not None and kept != temperature:
        _same_temperature(kept, temperature, "the forward")
    S, dt = 1 if seq_offsets is None else _num_seqs(seq_offsets), (logits.dtype,)
    m, lists = _list_args(targets, T, dev, of=_LIST_READS)
    tokens, row_stats = forward._pointers(dev, T, S, of=_DISTILL_READS)
    args = (rows, code, *lists, row_stats, tokens,
            _p(seq_offsets, "seq_offsets", _I32, (S + 1,), dev), T, E, m, S, temperature,
            _p(dloss, "dloss", _F32, (S,), dev), _p(base, "base", dt, (T, E), dev))
    current, raw = _on(dev, stream)
    with current:
        if dlogits is None:
            dlogits = torch.empty((T, E), dtype=logits.dtype, device=dev)
        _check(lib.moe_distill_loss_backward(*args, _p(dlogits, "dlogits", dt, (T, E), dev),
                                             raw))
    return dlogits
