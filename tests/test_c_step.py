"""The step operators used from plain C (tests/native/c_step_check.c): no
Python on the path, results compared with loops in double."""
import os
import subprocess

import pytest

EXE = os.path.join(os.path.dirname(os.path.abspath(__file__)), "native", "c_step_check")


def test_c_program_links_against_the_header():
    """Built by __graft_entry__.build()."""
    assert os.path.exists(EXE), "run __graft_entry__.build() (builds tests/native/c_step_check)"
    out = subprocess.run(["ldd", EXE], capture_output=True, text=True).stdout
    assert "libzpq.so" in out and "not found" not in out, out


@pytest.mark.gpu
def test_c_program_matches_loops_in_double():
    print("c_step_check", flush=True)
    r = subprocess.run([EXE], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "c_step_check: ok" in r.stdout, r.stdout + r.stderr
