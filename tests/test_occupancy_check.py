"""The library keeps what the driver says of a kernel's resident blocks
(tests/occupancy_check.cpp): every kernel is asked about once, however many forms and
devices a process uses, and a full table still gives the right answers."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "combine_moe_dispatch_gb300", "csrc")


@pytest.fixture(scope="module")
def exe(tmp_path_factory):
    out = tmp_path_factory.mktemp("occupancy") / "occupancy_check"
    subprocess.run([shutil.which("g++") or "g++", "-O2", "-std=c++17", "-I", CSRC,
                    os.path.join(HERE, "occupancy_check.cpp"), "-o", str(out)], check=True)
    return str(out)


def _run(exe, kernels, devices):
    out = subprocess.run([exe, str(kernels), str(devices)], check=True, capture_output=True, text=True,
                         timeout=60).stdout.split()
    return {out[i]: int(out[i + 1]) for i in range(0, len(out), 2)}


@pytest.mark.parametrize("kernels,devices", [(1, 1), (64, 1), (150, 1), (150, 4), (180, 4)])
def test_each_kernel_is_asked_about_once(exe, kernels, devices):
    assert _run(exe, kernels, devices) == {"first": 2 * kernels * devices, "again": 0, "wrong": 0}


def test_a_full_table(exe):
    r = _run(exe, 2000, 2)
    assert r["wrong"] == 0 and r["first"] == 8000 and r["again"] == 3 * (8000 - 1536)
