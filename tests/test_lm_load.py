"""The library as the package hands it out, in a process that has called nothing yet."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "linear_recurrence_scan_diagonal_amd", "liblrs.so")


@pytest.mark.skipif(not os.path.exists(LIB), reason="liblrs.so not built")
def test_load_sets_the_prototypes_of_every_function():
    """A workspace of more than 2 GiB, asked for before any other call (an int would be
    negative), and a status string."""
    code = ("import linear_recurrence_scan_diagonal_amd as lrs\n"
            "lib = lrs.load()\n"
            "print(lib.lrs_linear_ce_workspace_bytes(65536, 131072, 1024, 1, 1))\n"
            "print(lib.lrs_status_string(0).decode())\n"
            "from linear_recurrence_scan_diagonal_amd import binding, lm\n"
            "print(all(getattr(lib, n).argtypes is not None for n in binding.EXPORTS + lm.EXPORTS))\n")
    out = subprocess.run([sys.executable, "-c", code], cwd=ROOT, check=True, capture_output=True, text=True)
    nbytes, status, prototypes = out.stdout.splitlines()
    assert 2 ** 31 < int(nbytes) < 2 ** 32 and status and prototypes == "True"
