"""The tiles of an expert's tokens (tests/tiles_check.cpp), for up to 2^31 - 1 of
them: the sums that round up pass 31 bits there, and a tile whose first token came
out negative would have been read and written before its arrays."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "combine_moe_dispatch_gb300", "csrc")


@pytest.fixture(scope="module")
def exe(tmp_path_factory):
    out = tmp_path_factory.mktemp("tiles") / "tiles_check"
    subprocess.run([shutil.which("g++") or "g++", "-O1", "-std=c++17", "-fwrapv", "-I", CSRC,
                    os.path.join(HERE, "tiles_check.cpp"), "-o", str(out)], check=True)
    return str(out)


@pytest.mark.parametrize("step", ["32", "64"])
def test_tiles(exe, step):
    out = subprocess.run([exe, step], check=True, capture_output=True, text=True).stdout.split()
    r = {out[i]: int(out[i + 1]) for i in range(0, len(out), 2)}
    assert r["bad"] == 0 and r["rows"] > 10000 and r["tiles"] > r["rows"], r
