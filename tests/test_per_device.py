"""What the library keeps for each device: asked once on each, and again after a failure (host code, no GPU)."""
import ctypes
import os
import subprocess

import pytest

from helpers import ROOT

SOURCE = r"""
#include "perdevice.h"
static fp4moe::PerDevice kept;
static int asked[fp4moe::kMaxDevices];
extern "C" int get(int device, int answer) {
  return kept.get(device, [=] { ++asked[device]; return answer; });
}
extern "C" int times(int device) { return asked[device]; }
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("per_device")
    src, out = d / "t.cpp", d / "t.so"
    src.write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "block_scaled_fp4_top_gb300", "csrc"), str(src), "-o", str(out)], check=True)
    return ctypes.CDLL(str(out))


def test_each_device_is_asked_once(lib):
    assert lib.get(0, 7) == 7 and lib.get(0, 8) == 7 and lib.times(0) == 1
    assert lib.get(1, 9) == 9 and lib.get(1, 9) == 9 and lib.times(1) == 1      # the first device's does not stand for it
    assert lib.get(0, 1) == 7


def test_a_failure_is_not_kept(lib):
    assert lib.get(2, 0) == 0 and lib.get(2, 0) == 0 and lib.times(2) == 2
    assert lib.get(2, 5) == 5 and lib.get(2, 0) == 5 and lib.times(2) == 3


def test_devices_out_of_range(lib):
    assert lib.get(-1, 3) == 0 and lib.get(64, 3) == 0
