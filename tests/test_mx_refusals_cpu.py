"""Each refusal of the microscaled calls by itself, as far as no device is
needed: the call is right but for one argument, and the message names it."""
import ctypes

import pytest
import torch

OK, INVALID_ARG, SHAPE, DTYPE, UNSUPPORTED = 0, 1, 2, 3, 4
BF16, MXFP4, MXFP8 = 2, 0, 1
R, C, N = 8, 96, 16


def _at(n, off=0):
    """The n-th buffer: none is dereferenced, since every call below is refused."""
    return ctypes.c_void_p(0x10000000 + (n << 20) + off)


@pytest.fixture(scope="module")
def lib():
    from top_routing_grouped_fp32_gb300 import build as native_build
    from top_routing_grouped_fp32_gb300 import _lib
    native_build.build()
    return _lib.load()


QUANTIZE = dict(x=_at(0), dt=BF16, R=R, C=C, fmt=MXFP4, values=_at(1), scales=_at(2), stream=None)
DEQUANTIZE = dict(values=_at(1), scales=_at(2), fmt=MXFP8, R=R, C=C, perm=_at(3), k=2, n=N, out=_at(4), dt=BF16,
                  stream=None)
CREATE = dict(gate=_at(0), gs=_at(1), up=_at(2), us=_at(3), down=_at(4), ds=_at(5), dt=BF16, E=4, I=64, H=96,
              buffer=_at(6), nbytes=1 << 30, stream=None)
CALLS = {"moe_mx_quantize": QUANTIZE, "moe_mx_dequantize": DEQUANTIZE, "moe_mx4_experts_create": CREATE}
CASES = [
    ("moe_mx_quantize", dict(dt=3), DTYPE, "x dtype"), ("moe_mx_quantize", dict(dt=-1), DTYPE, "x dtype"),
    ("moe_mx_quantize", dict(fmt=2), DTYPE, "format"), ("moe_mx_quantize", dict(fmt=-1), DTYPE, "format"),
    ("moe_mx_quantize", dict(R=-1), SHAPE, "R must"), ("moe_mx_quantize", dict(R=2 ** 31), UNSUPPORTED, "R="),
    ("moe_mx_quantize", dict(C=0), SHAPE, "C must"), ("moe_mx_quantize", dict(C=2 ** 20 + 1), UNSUPPORTED, "C="),
    ("moe_mx_quantize", dict(x=None), INVALID_ARG, "non-NULL"),
    ("moe_mx_quantize", dict(values=None), INVALID_ARG, "non-NULL"),
    ("moe_mx_quantize", dict(scales=None), INVALID_ARG, "non-NULL"),
    ("moe_mx_quantize", dict(x=_at(0, 1)), INVALID_ARG, "misaligned"),
    ("moe_mx_quantize", dict(values=_at(0, R * C * 2 - 1)), INVALID_ARG, "overlap"),
    ("moe_mx_quantize", dict(scales=_at(0)), INVALID_ARG, "overlap"),
    ("moe_mx_quantize", dict(scales=_at(1, R * C // 2 - 1)), INVALID_ARG, "overlap"),
    ("moe_mx_dequantize", dict(dt=5), DTYPE, "out dtype"), ("moe_mx_dequantize", dict(fmt=9), DTYPE, "format"),
    ("moe_mx_dequantize", dict(R=-1), SHAPE, "R must"), ("moe_mx_dequantize", dict(n=-1), SHAPE, "n must"),
    ("moe_mx_dequantize", dict(n=2 ** 31), UNSUPPORTED, "n="), ("moe_mx_dequantize", dict(C=0), SHAPE, "C must"),
    ("moe_mx_dequantize", dict(k=0), INVALID_ARG, "top_k"),
    ("moe_mx_dequantize", dict(perm=None, k=1), SHAPE, "without perm"),
    ("moe_mx_dequantize", dict(perm=None, n=R), INVALID_ARG, "needs perm"),
    ("moe_mx_dequantize", dict(out=None), INVALID_ARG, "non-NULL"),
    ("moe_mx_dequantize", dict(values=None), INVALID_ARG, "non-NULL"),
    ("moe_mx_dequantize", dict(scales=None), INVALID_ARG, "non-NULL"),
    ("moe_mx_dequantize", dict(out=_at(4, 1)), INVALID_ARG, "misaligned"),
    ("moe_mx_dequantize", dict(perm=_at(3, 2)), INVALID_ARG, "misaligned"),
    ("moe_mx_dequantize", dict(out=_at(1, R * C - 2)), INVALID_ARG, "overlap"),
    ("moe_mx_dequantize", dict(out=_at(2)), INVALID_ARG, "overlap"),
    ("moe_mx_dequantize", dict(out=_at(3)), INVALID_ARG, "overlap"),
    ("moe_mx4_experts_create", dict(dt=0), DTYPE, "F16 or BF16"),
    ("moe_mx4_experts_create", dict(E=0), SHAPE, "E must"),
    ("moe_mx4_experts_create", dict(E=1025), UNSUPPORTED, "E=1025"),
    ("moe_mx4_experts_create", dict(I=0), SHAPE, "I must"), ("moe_mx4_experts_create", dict(H=0), SHAPE, "H must"),
    ("moe_mx4_experts_create", dict(I=2 ** 20 + 32), UNSUPPORTED, "I="),
    ("moe_mx4_experts_create", dict(I=40), UNSUPPORTED, "blocks of 32"),
    ("moe_mx4_experts_create", dict(H=48), UNSUPPORTED, "blocks of 32"),
    ("moe_mx4_experts_create", dict(buffer=None), INVALID_ARG, "scale_buffer"),
    ("moe_mx4_experts_create", dict(buffer=_at(6, 16)), INVALID_ARG, "scale_buffer"),
    ("moe_mx4_experts_create", dict(nbytes=1), INVALID_ARG, "scale_buffer too small"),
] + [("moe_mx4_experts_create", {a: None}, INVALID_ARG, "non-NULL") for a in ("gate", "gs", "up", "us", "down", "ds")] \
  + [("moe_mx4_experts_create", {a: _at(9, 8)}, INVALID_ARG, "16-byte aligned") for a in ("gate", "up", "down")]


@pytest.mark.parametrize("name,change,status,words", CASES)
def test_refusal(lib, name, change, status, words):
    args = {**CALLS[name], **change}
    values = list(args.values())
    handle = ctypes.c_void_p(1)
    if name == "moe_mx4_experts_create":
        values.append(ctypes.byref(handle))
    assert getattr(lib, name)(*values) == status, lib.moe_last_error().decode()
    assert words in lib.moe_last_error().decode()
    if name == "moe_mx4_experts_create":
        assert not handle.value


@pytest.mark.parametrize("name,empty", [("moe_mx_quantize", dict(R=0)), ("moe_mx_dequantize", dict(n=0))])
def test_the_unchanged_call_is_right(lib, name, empty):
    assert getattr(lib, name)(*{**CALLS[name], **empty}.values()) == OK


def test_calls_without_a_handle(lib):
    z = ctypes.c_void_p()
    assert lib.moe_mx4_experts_forward(z, _at(0), 1, _at(1), _at(2), _at(3), 1 << 20, None) == INVALID_ARG
    assert lib.moe_mx4_forward(z, _at(0), _at(1), BF16, 1, 1, 1, _at(2), _at(3), 1 << 20, None) == INVALID_ARG
    assert lib.moe_experts_forward_checkpoint(z, _at(0), 1, *[_at(i) for i in range(1, 8)], 1 << 20, None) == INVALID_ARG
    assert lib.moe_experts_backward_checkpoint(z, _at(0), _at(1), 1, 1, *[_at(i) for i in range(2, 14)], 1 << 20,
                                               None) == INVALID_ARG
    assert lib.moe_mx4_experts_create(*CREATE.values(), None) == INVALID_ARG
    assert lib.moe_mx4_experts_workspace_size(z, 8) == lib.moe_mx4_forward_workspace_size(z, 8, 2, BF16) == 0
    assert lib.moe_experts_backward_checkpoint_workspace_size(z, 8) == 0
    assert lib.moe_mx4_experts_scale_bytes(0, 64, 64) == lib.moe_mx4_experts_scale_bytes(4, 2 ** 21, 64) == 0
    lib.moe_mx4_experts_destroy(z)


# ---- the binding ---------------------------------------------------------------------------------
def test_rows_have_the_shapes_of_their_format():
    import top_routing_grouped_fp32_gb300 as moe
    for fmt, cols, values, scales in (("mxfp4", 33, 17, 2), ("mxfp4", 64, 32, 2), ("mxfp8", 33, 33, 2),
                                      ("mxfp8", 1, 1, 1)):
        m = moe.MxRows.empty((2, 3, cols), fmt, "cpu")
        assert m.values.shape == (2, 3, values) and m.scales.shape == (2, 3, scales) and m.shape == (2, 3, cols)


def test_binding_refusals():
    import top_routing_grouped_fp32_gb300 as moe
    m = moe.MxRows.empty((4, 64), "mxfp8", "cpu")
    for call, status in ((lambda: moe.moe_mx_quantize(torch.zeros(4, 64), "mxfp6"), 3),
                         (lambda: moe.MxRows.empty((4, 64), "e4m3", "cpu"), 3),
                         (lambda: moe.moe_mx_quantize(torch.zeros(4, 64, dtype=torch.float64), "mxfp4"), 3),
                         (lambda: moe.moe_mx_quantize(torch.zeros(()), "mxfp4"), 2),
                         (lambda: m._checked("m", (4, 65)), 2), (lambda: m._checked("m", format="mxfp4"), 3),
                         (lambda: moe.Mx4SwiGluExperts(m, m, m), 2)):
        with pytest.raises(moe.MoeError) as e:
            call()
        assert e.value.status == status
    with pytest.raises(ValueError, match="CUDA"):
        moe.moe_mx_quantize(torch.zeros(4, 64), "mxfp4")
    with pytest.raises(ValueError, match="CUDA"):
        moe.moe_mx_dequantize(m, torch.float32)
