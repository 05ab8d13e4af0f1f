"""The library's table of workspaces, compiled with the host compiler against a CUDA
runtime that fails where it is told to (workspace_host.cpp)."""
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("workspace") / "workspace_host")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", os.path.join(HERE, "workspace_host.cpp"), "-o", out],
                   check=True, timeout=300)
    return out


@pytest.mark.parametrize("what", ["reuse_and_growth", "an_allocation_fails", "zeroing_fails", "a_stream_that_is_captured",
                                  "growth_after_a_capture"])
def test_workspaces(program, what):
    r = subprocess.run([program, what], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout
