"""CPU test of when a decode launch goes without programmatic dependent launch: the rule is host code,
compiled here with nothing around it."""
import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CUDA = os.environ.get("CUDA_HOME", "/usr/local/cuda")

SOURCE = """
#include "pkv_internal.h"
extern "C" {
pkv_pool *made() { return new pkv_pool(); }
void gone(pkv_pool *p) { delete p; }
void wrote(pkv_pool *p, uintptr_t s) { pkv::pages_written(p, reinterpret_cast<cudaStream_t>(s)); }
int may(pkv_pool *p, uintptr_t s, int wanted)
{
    return pkv::take_pdl_permission(p, reinterpret_cast<cudaStream_t>(s), wanted != 0);
}
}
"""


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    d = tmp_path_factory.mktemp("fence")
    (d / "fence.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", f"{CUDA}/include", "-I",
                    os.path.join(ROOT, "paged_kv_decode_12_gb300", "csrc"), "-o", str(d / "fence.so"), str(d / "fence.cpp")],
                   check=True)
    L = ctypes.CDLL(str(d / "fence.so"))
    L.made.restype = ctypes.c_void_p
    L.gone.argtypes = [ctypes.c_void_p]
    L.wrote.argtypes = [ctypes.c_void_p, ctypes.c_size_t]
    L.may.argtypes = [ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int]
    return L


A, B, C = 0, 0x1000, 0x2000                      # streams (0: the default one)


def test_the_next_launch_waits_wherever_it_is(rule):
    p = rule.made()
    assert rule.may(p, A, 1) == 1 and rule.may(p, A, 0) == 0
    rule.wrote(p, A)
    assert rule.may(p, A, 1) == 0 and rule.may(p, A, 1) == 1
    rule.wrote(p, A)
    assert rule.may(p, B, 1) == 0                # as before: the next launch on the pool
    rule.gone(p)


@pytest.mark.parametrize("wanted", [0, 1])
def test_a_launch_on_another_stream_does_not_use_the_wait_up(rule, wanted):
    """Pages written on A, a launch on B, then one on A right behind the writes."""
    p = rule.made()
    rule.wrote(p, A)
    rule.may(p, B, wanted)
    assert rule.may(p, A, 1) == 0 and rule.may(p, A, 1) == 1
    # two streams that have written, and one that has not
    rule.wrote(p, A)
    rule.wrote(p, B)
    rule.wrote(p, B)
    assert rule.may(p, C, 1) == 0 and rule.may(p, C, 1) == 1
    assert rule.may(p, B, 1) == 0 and rule.may(p, B, 1) == 1
    assert rule.may(p, A, 0) == 0 and rule.may(p, A, 1) == 1      # one that never overlaps has waited too
    rule.gone(p)


def test_many_streams(rule):
    p = rule.made()
    for s in range(1, 3001):
        rule.wrote(p, s * 64)
    rule.may(p, A, 1)
    for s in range(3000, 0, -1):
        assert rule.may(p, s * 64, 1) == 0
    assert all(rule.may(p, s * 64, 1) == 1 for s in range(1, 3001))
    rule.gone(p)
