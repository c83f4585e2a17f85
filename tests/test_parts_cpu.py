"""How the checkpointed backward cuts its sums (csrc/parts.h), compiled for the host:
the room for the parts' outputs holds them and does not fall as batches grow."""
import ctypes
import os
import random
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "top_routing_grouped_fp32_gb300", "csrc")
SOURCE = """
#include "parts.h"
extern "C" {
int weight_gradient(int64_t N, int64_t E, int64_t m, int64_t n, int64_t sms) {
  return moe::parts::weight_gradient(N, E, m, n, sms);
}
int dinput(int64_t N, int64_t E, int64_t H, int64_t I, int64_t sms) { return moe::parts::dinput(N, E, H, I, sms); }
int64_t room(int64_t N, int64_t E, int64_t H, int64_t I, int64_t sms) { return moe::parts::room(N, E, H, I, sms); }
}
"""
I64 = ctypes.c_int64
SMS = 152


@pytest.fixture(scope="module")
def parts(tmp_path_factory):
    d = tmp_path_factory.mktemp("parts")
    (d / "parts.cc").write_text(SOURCE)
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, "-o", str(d / "parts.so"),
                    str(d / "parts.cc")], check=True)
    lib = ctypes.CDLL(str(d / "parts.so"))
    for f, res in ((lib.weight_gradient, ctypes.c_int), (lib.dinput, ctypes.c_int), (lib.room, I64)):
        f.argtypes, f.restype = [I64] * 5, res
    return lib


def shapes():
    rng = random.Random(3)
    out = [(2, 2048, 1408), (4, 1024, 1024), (1, 8, 8), (1, 8, 1 << 20), (1024, 8, 2056), (64, 2048, 1408), (5, 3688, 696)]
    for _ in range(60):
        out.append((int(2 ** rng.uniform(0, 8)), 8 * int(2 ** rng.uniform(0, 10)), 8 * int(2 ** rng.uniform(0, 11))))
    return out


def taken(parts, N, E, H, I, sms=SMS):
    """FP32 values that a batch of N rows writes."""
    gate_up, down = parts.weight_gradient(N, E, 2 * I, H, sms), parts.weight_gradient(N, E, H, I, sms)
    x = parts.dinput(N, E, H, I, sms)
    assert min(gate_up, down, x) >= 1
    return max(gate_up * E * 2 * I * H if gate_up > 1 else 0, down * E * I * H if down > 1 else 0, x * N * H if x > 1 else 0)


def test_the_room_holds_the_parts_and_does_not_fall(parts):
    cut = 0
    for E, H, I in shapes():
        last = 0
        for N in [*range(0, 700), *range(700, 40000, 61), 1 << 20, (1 << 31) - 1]:
            room, need = parts.room(N, E, H, I, SMS), taken(parts, N, E, H, I)
            assert need <= room and last <= room, (N, E, H, I)
            last, cut = room, cut + (need > 0)
    assert cut > 10000


def test_where_the_parts_of_dinput_become_fewer(parts):
    """The cases that a workspace of exactly the parts' size would refuse."""
    for E, H, I, N in ((2, 2048, 1408, 767), (4, 1024, 1024, 1535)):
        assert parts.dinput(N, E, H, I, SMS) > 1 == parts.dinput(N + 1, E, H, I, SMS)
        assert parts.room(N, E, H, I, SMS) == parts.room(N + 1, E, H, I, SMS) >= taken(parts, N, E, H, I)


@pytest.mark.parametrize("sms", [2, 20, 76, 132, 148, 152, 160])
def test_parts_fill_the_sms_of_the_device(parts, sms):
    """Never a second wave for parts alone, and no room left for another part of every tile
    unless the parts are short."""
    for E, H, I in shapes():
        for N in (1, 3, 30, 100, 127, 128, 700, 5000, 20560, 98304):
            pair = N >= 128 * E
            x, places = parts.dinput(N, E, H, I, sms), sms // 2 if pair else sms
            tiles = (N // (256 if pair else 128) + min(E, N)) * -(-H // 256)
            deepest = 2 * -(-I // 64) // 8
            assert x == 1 or x * tiles <= places
            assert (x + 1) * tiles > places or x >= deepest
            for m, n in ((2 * I, H), (H, I)):
                w, tiles = parts.weight_gradient(N, E, m, n, sms), E * -(-m // 256) * -(-n // 256)
                assert w == 1 or w * tiles <= sms // 2
                assert (w + 1) * tiles > sms // 2 or w >= N // (E * 256)
            assert taken(parts, N, E, H, I, sms) <= parts.room(N, E, H, I, sms)
