"""A compiled module built for another torch is not loaded."""
import os
import subprocess
import sys
import sysconfig

import torch

import bit_quantized_all_gb300 as qr

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(qr.__file__)))

CALL = """
import sys, warnings
sys.path.insert(0, sys.argv[1])
import torch
torch.__version__ = "0.0.0"
from bit_quantized_all_gb300 import layer
with warnings.catch_warnings(record=True) as seen:
    warnings.simplefilter("always")
    layer._fast()
assert "_qr_fast" in str(seen[0].message) and "bit_quantized_all_gb300._qr_fast" not in sys.modules
print("not loaded")
"""


def test_another_torch():
    from bit_quantized_all_gb300 import build
    build.build()
    p = subprocess.run([sys.executable, "-c", CALL, ROOT], capture_output=True, text=True)
    assert p.returncode == 0 and "not loaded" in p.stdout, p.stderr


def test_the_name():
    from bit_quantized_all_gb300 import build, layer
    build.build()
    assert torch.__version__ in build.FAST_PATH and sysconfig.get_config_var("SOABI") in build.FAST_PATH
    assert layer._fast().__file__ == build.FAST_PATH
