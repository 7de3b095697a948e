"""Which rows and columns the tiles of the experts' products take (CPU): the kernels' arithmetic, compiled for the
host, on whole plans, on dense groups and on plan workspaces of any content."""
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)


def test_tiles_stay_inside_their_buffers(tmp_path):
    exe = str(tmp_path / "tile_line_check")
    r = subprocess.run(["g++", "-std=c++17", "-O2", "-fsanitize=undefined", "-fno-sanitize-recover=undefined",
                        "-D__HIP_PLATFORM_AMD__", "-I", "/opt/rocm/include", "-I", os.path.join(ROOT, "include"), "-I",
                        os.path.join(ROOT, "combine_ep_plan_amd", "csrc"), "-o", exe,
                        os.path.join(HERE, "native", "tile_line_check.cpp")], capture_output=True, text=True)
    if r.returncode != 0:
        pytest.fail("could not build the check: " + r.stderr[-2000:])
    out = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stdout + out.stderr
    assert int(out.stdout.split()[1]) > 1_000_000
