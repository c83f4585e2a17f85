"""The buffer for the re-ordered scales of 4-bit experts lies over none of the weights,
by a byte on either side; nothing is dereferenced."""
import ctypes

import pytest

INVALID_ARG, BF16 = 1, 2
E, I, H = 4, 64, 96
VALUES, SCALES, DOWN_SCALES = E * I * H // 2, E * I * (H // 32), E * H * (I // 32)


@pytest.fixture(scope="module")
def lib():
    from top_routing_grouped_fp32_gb300 import build as native_build
    from top_routing_grouped_fp32_gb300 import _lib
    native_build.build()
    return _lib.load()


def at(n, off=0):
    return 0x10000000 + (n << 20) + off


def create(lib, args, buffer):
    out = ctypes.c_void_p(1)
    P = ctypes.c_void_p
    st = lib.moe_mx4_experts_create(*(P(args[n]) for n in ("gate", "gs", "up", "us", "down", "ds")), BF16, E, I, H,
                                    P(buffer), 1 << 30, None, ctypes.byref(out))
    assert not out.value
    return st, lib.moe_last_error().decode()


@pytest.mark.parametrize("name,size", [("gate", VALUES), ("up", VALUES), ("down", VALUES), ("gs", SCALES), ("us", SCALES),
                                       ("ds", DOWN_SCALES)])
def test_over_the_weights(lib, name, size):
    names = ("gate", "gs", "up", "us", "down", "ds")
    args = {n: at(i) for i, n in enumerate(names)}
    need, buffer = lib.moe_mx4_experts_scale_bytes(E, I, H), at(9)
    unit = 1 if name.endswith("s") else 16
    # from the first byte of the buffer, up to the last, and reaching into it from below
    for place in (buffer, buffer + (need - 1) // unit * unit, buffer - (size - 1) // unit * unit):
        st, words = create(lib, {**args, name: place}, buffer)
        assert st == INVALID_ARG and "overlap" in words, (name, place - buffer)
    # next to it: past this check (what comes then needs a device)
    for place in (buffer + (need + unit - 1) // unit * unit, buffer - (size + unit - 1) // unit * unit):
        st, words = create(lib, {**args, name: place}, buffer)
        assert st != 0 and "overlap" not in words
