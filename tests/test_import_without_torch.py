"""The package's names with and without torch, which only the decoder-layer operators need."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("torch_there", [False, True])
def test_star_import(torch_there):
    import __graft_entry__

    __graft_entry__.build()
    code = ("import sys\n" + ("" if torch_there else "sys.modules['torch'] = None\n") +
            "from moe_decode_host_gb300 import *\n"
            "print(Layer.__name__, moe_route.__name__, 'moe_linear' in globals(), 'KvCache' in globals())\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    assert r.stdout.split() == ["Layer", "moe_route", str(torch_there), str(torch_there)]
