"""A number that belongs to a device (csrc/per_device.h), compiled for the host: each
device is asked for its own, once."""
import ctypes
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "top_routing_grouped_fp32_gb300", "csrc")
SOURCE = """
#include "per_device.h"
static moe::PerDevice known;
extern "C" int get(int device, int answer, int error, int* out, int* asked) {
  return known.get(device, out, [&](int* n) { ++*asked; *n = answer; return error; });
}
"""


@pytest.fixture
def get(tmp_path):
    (tmp_path / "p.cc").write_text(SOURCE)
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, "-o", str(tmp_path / "p.so"),
                    str(tmp_path / "p.cc")], check=True)
    lib = ctypes.CDLL(str(tmp_path / "p.so"))

    def call(device, answer, error=0):
        out, asked = ctypes.c_int(-1), ctypes.c_int(0)
        return lib.get(device, answer, error, ctypes.byref(out), ctypes.byref(asked)), out.value, asked.value
    return call


def test_each_device_is_asked_once(get):
    assert get(0, 152) == (0, 152, 1) and get(0, 99) == (0, 152, 0)
    assert get(1, 148) == (0, 148, 1) and get(1, 99) == (0, 148, 0) and get(0, 99) == (0, 152, 0)
    assert get(63, 7) == (0, 7, 1) and get(63, 8) == (0, 7, 0)


def test_errors_and_nothing_are_not_kept(get):
    assert get(2, 5, error=3)[0::2] == (3, 1)
    assert get(2, 0) == (0, 0, 1)
    assert get(2, 6) == (0, 6, 1) and get(2, 7, error=3) == (0, 6, 0)


def test_devices_beyond_the_table_are_asked_every_time(get):
    for n in (11, 12):
        assert get(64, n) == (0, n, 1) and get(1000, n) == (0, n, 1)
    assert get(0, 13) == (0, 13, 1)
