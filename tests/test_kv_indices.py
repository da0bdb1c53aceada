"""The K/V cache kernels' index arithmetic, compiled for the host: whatever the
device's index arrays hold, rows, positions and pages stay inside the caller's
buffers; the tiles of a call's blocks cover every key that a row sees."""
import os
import subprocess

import pytest

from error_compensated_bit_amd import binding as B
from error_compensated_bit_amd import build as eb

HIPCC = "/opt/rocm/bin/hipcc"


def test_indices_stay_inside_and_tiles_cover_every_key(tmp_path):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not installed")
    B.load_library()
    exe = tmp_path / "check_indices"
    src = os.path.join(os.path.dirname(os.path.abspath(__file__)), "kv_host", "check_indices.cpp")
    subprocess.run([HIPCC, "-x", "hip", "--offload-host-only", "-std=c++17", "-O1", "-I", eb.CSRC, src, "-o", str(exe),
                    "-x", "none", eb.library_path()], check=True, capture_output=True, text=True)
    run = subprocess.run([str(exe)], capture_output=True, text=True, env={**os.environ,
                         "LD_LIBRARY_PATH": os.path.dirname(eb.library_path()) + ":" + os.environ.get("LD_LIBRARY_PATH", "")})
    assert run.returncode == 0 and run.stdout == "ok\n", run.stdout + run.stderr
