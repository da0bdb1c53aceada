"""Positions of query rows, compiled for the host: attention puts each row of a
sequence where the write puts it, also where max_len or the page table end
before the sequence does, and covers the keys that such rows see."""
import os
import subprocess

import pytest

from error_compensated_bit_amd import binding as B
from error_compensated_bit_amd import build as eb

HIPCC = "/opt/rocm/bin/hipcc"


def test_rows_are_attended_at_the_positions_they_are_written_to(tmp_path):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not installed")
    B.load_library()
    exe = tmp_path / "check_positions"
    src = os.path.join(os.path.dirname(os.path.abspath(__file__)), "kv_host", "check_positions.cpp")
    subprocess.run([HIPCC, "-x", "hip", "--offload-host-only", "-std=c++17", "-O1", "-I", eb.CSRC, src, "-o", str(exe),
                    "-x", "none", eb.library_path()], check=True, capture_output=True, text=True)
    run = subprocess.run([str(exe)], capture_output=True, text=True, env={**os.environ,
                         "LD_LIBRARY_PATH": os.path.dirname(eb.library_path()) + ":" + os.environ.get("LD_LIBRARY_PATH", "")})
    assert run.returncode == 0 and run.stdout == "ok\n", run.stdout + run.stderr
