"""What the library does once per device (a kernel's shared-memory limit is an
attribute of a function on a device): host code, compiled here by itself."""
import glob
import os
import shutil
import subprocess

import pytest

from combine_moedc_layout_gb300 import build as mbuild

PROGRAM = r"""
#include "per_device.cuh"
#include <cstdio>
#define CHECK(c) do { if (!(c)) { std::printf("line %d\n", __LINE__); return 1; } } while (0)
int main()
{
    moedc_host::PerDevice first, second;
    int calls = 0;
    bool works = true;
    auto act = [&] { ++calls; return works; };
    CHECK(first.once(0, act) && calls == 1);
    CHECK(first.once(0, act) && calls == 1);       // done there
    CHECK(first.once(1, act) && calls == 2);       // another device has its own
    CHECK(second.once(0, act) && calls == 3);      // and so has another function
    works = false;
    CHECK(!first.once(2, act) && calls == 4);
    CHECK(!first.once(2, act) && calls == 5);      // a failure is tried again
    works = true;
    CHECK(first.once(2, act) && calls == 6);
    CHECK(first.once(2, act) && calls == 6);
    CHECK(first.once(64, act) && first.once(64, act) && calls == 8);   // past the table: each time
    CHECK(first.once(-1, act) && calls == 9);
    return 0;
}
"""


def test_once_on_each_device_and_never_a_failure_kept(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host compiler")
    src, exe = tmp_path / "once.cpp", tmp_path / "once"
    src.write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-I", mbuild.CSRC, str(src), "-o", str(exe), "-pthread"],
                   check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


def test_no_function_attribute_is_set_once_per_process():
    for path in glob.glob(os.path.join(mbuild.CSRC, "*.cu*")):
        with open(path) as f:
            text = f.read()
        assert "cudaFuncSetAttribute" not in text or "call_once" not in text, path
