"""Which phase of an mbarrier a thread that gives up has to wait for, so that no load of its own is in flight when its block
ends (host code, no GPU): the barrier is modelled as its phases."""
import ctypes
import os
import subprocess

import pytest

from helpers import ROOT

SOURCE = r"""
#include "inflight.h"
extern "C" int any_after(int n) { fp4moe::InFlight f; for (int i = 0; i < n; ++i) f.issue(); return f.any(); }
extern "C" unsigned last_after(int n) { fp4moe::InFlight f; for (int i = 0; i < n; ++i) f.issue(); return f.last(); }
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("in_flight")
    src, out = d / "t.cpp", d / "t.so"
    src.write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "block_scaled_fp4_top_gb300", "csrc"), str(src), "-o", str(out)], check=True)
    return ctypes.CDLL(str(out))


class Barrier:
    """mbarrier of one arrival a phase: a wait for a parity is over when the phase under way has the other one."""

    def __init__(self):
        self.completed = 0

    def waits(self, parity):
        return self.completed & 1 == parity


def test_nothing_was_issued(lib):
    assert not lib.any_after(0)


@pytest.mark.parametrize("n", range(1, 9))
def test_the_wait_is_for_the_last_load(lib, n):
    assert lib.any_after(n)
    b = Barrier()
    b.completed = n - 1                       # all before it have landed: nothing is issued on a phase that is not over
    assert b.waits(lib.last_after(n)), "over while the last load is in flight"
    b.completed = n
    assert not b.waits(lib.last_after(n)), "waits for a load that was never issued"


def test_loader_counts_its_loads_of_q():
    """The loader gives up inside a unit (its q is issued) and in front of one (it is not): units say neither."""
    with open(os.path.join(ROOT, "block_scaled_fp4_top_gb300", "csrc", "attntile.cu")) as f:
        text = f.read()
    issue = text.index("q_boxes.issue();")
    assert text.rindex("mbar_arrive_expect_tx(bar.q_full()", 0, issue) < issue < text.index("tma_load_3d(sm32", issue)
    assert "drain_wait(bar.q_full(), q_boxes.last())" in text and text.count("drain_wait(bar.q_full()") == 1
