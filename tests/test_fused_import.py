"""The package without the extension module of the fused calls: everything else stays, and
each of those calls says what is missing."""
import os
import subprocess
import sys

import pytest

import quantized_int8_gemm_amd as q

HERE = os.path.dirname(os.path.abspath(q.__file__))
PROGRAM = """
import torch
import quantized_int8_gemm_amd as q
x = torch.zeros(2, 32)
for call in (lambda: q.qgemm_a8w8_linear(x, x, x, x), lambda: q.qgemm_a8w8_gated(x, x, x, x, x, x), lambda: q.qgemm_a8w8_linear_grad(x, x, x),
             lambda: q.qgemm_a8w8_gated_grad(x, x, x, x, x, (x, x)), lambda: q.int8_quantize(x), lambda: q.int8_dequantize(x, x)):
    try:
        call()
    except ImportError as e:
        assert "_fused_binding.so" in str(e) and "build()" in str(e) and "WHY" in str(e), str(e)
    else:
        raise SystemExit("no error")
try:
    q.mx_quantize(x)
except ValueError:   # the module is there: the tensor is on the CPU
    print("fine")
"""


@pytest.mark.parametrize("kind,why", [("missing", "_fused_binding"), ("not a library", "invalid ELF header")])
def test_the_rest_without_the_extension(tmp_path, kind, why):
    pkg = tmp_path / os.path.basename(HERE)
    pkg.mkdir()
    for name in os.listdir(HERE):
        if name.endswith(".py") or name in ("libqgemm.so", "_mx_binding.so"):
            os.symlink(os.path.join(HERE, name), pkg / name)
    if kind != "missing":
        (pkg / "_fused_binding.so").write_bytes(b"not a shared library, but long enough for the loader to read a header of it " * 4)
    r = subprocess.run([sys.executable, "-c", PROGRAM.replace("WHY", why)], cwd=tmp_path, capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "fine", r.stderr
