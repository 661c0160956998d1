"""Without the compiled module the calls of layer.py run in their interpreted form."""
import os
import subprocess
import sys

import bit_quantized_all_gb300 as qr

PACKAGE = os.path.dirname(os.path.abspath(qr.__file__))

CALLS = """
import sys, warnings
sys.path.insert(0, sys.argv[1])
import torch
import bit_quantized_all_gb300 as qr
x = torch.zeros((4, 64), dtype=torch.float16)
rope = qr.Rope([1.0], device="cpu")
with warnings.catch_warnings(record=True) as seen:
    warnings.simplefilter("always")
    for call in (lambda: qr.qr_q8_quantize(x), lambda: qr.qr_rms_norm(x, x[0]), lambda: qr.qr_rms_norm_q8(x, x[0]),
                 lambda: qr.qr_rope(x[:, None], None, rope, torch.zeros(4, dtype=torch.int32))):
        try:
            call()
        except ValueError as e:  # what the interpreted form says of a tensor on the CPU
            assert "CUDA tensor" in str(e), e
        else:
            raise AssertionError("not refused")
assert len([w for w in seen if "_qr_fast" in str(w.message)]) == 1, seen
print("interpreted")
"""


def test_calls_without_the_compiled_module(tmp_path):
    from bit_quantized_all_gb300 import build
    build.build()
    copy = tmp_path / "bit_quantized_all_gb300"
    copy.mkdir()
    for name in os.listdir(PACKAGE):
        if not name.startswith(("_qr_fast", "__pycache__")):
            os.symlink(os.path.join(PACKAGE, name), copy / name)
    p = subprocess.run([sys.executable, "-c", CALLS, str(tmp_path)], capture_output=True, text=True, cwd=tmp_path)
    assert p.returncode == 0 and "interpreted" in p.stdout, p.stderr
