"""The package without its extension module: the integer products stay, and the
norm and MX calls say what is missing."""
import os
import subprocess
import sys

import pytest

import quantized_int8_gemm_amd as q
from quantized_int8_gemm_amd import build

HERE = os.path.dirname(os.path.abspath(q.__file__))
PROGRAM = """
import torch
import quantized_int8_gemm_amd as q
assert q.version().startswith("qgemm") and q.workspace_bytes is not None
x = torch.zeros(2, 32)
for call in (lambda: q.rms_norm(x, x[0]), lambda: q.rms_norm_quantize(x, x[0]), lambda: q.rms_norm_grad(x, x, x[0], x[:, 0]),
             lambda: q.mx_quantize(x), lambda: q.mx_dequantize(x, x), lambda: q.mx_matmul(x, x, x, x)):
    try:
        call()
    except ImportError as e:
        assert "_mx_binding.so" in str(e) and "build()" in str(e) and "WHY" in str(e), str(e)
    else:
        raise SystemExit("no error")
print("fine")
"""


@pytest.mark.parametrize("kind,why", [("missing", "_mx_binding"), ("not a library", "invalid ELF header")])
def test_integer_products_without_the_extension(tmp_path, kind, why):
    pkg = tmp_path / os.path.basename(HERE)
    pkg.mkdir()
    for name in os.listdir(HERE):
        if name.endswith(".py") or name == "libqgemm.so":
            os.symlink(os.path.join(HERE, name), pkg / name)
    if kind != "missing":
        (pkg / "_mx_binding.so").write_bytes(b"not a shared library, but long enough for the loader to read a header of it " * 4)
    r = subprocess.run([sys.executable, "-c", PROGRAM.replace("WHY", why)], cwd=tmp_path, capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "fine", r.stderr


def test_the_library_is_built_where_the_extension_cannot_be(tmp_path, monkeypatch):
    def link(cmd, check):
        open(cmd[cmd.index("-o") + 1], "w").close()

    def fails(verbose):
        raise RuntimeError("no host compiler")

    monkeypatch.setattr(build, "LIB", str(tmp_path / "libqgemm.so"))
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "objects"))
    monkeypatch.setattr(build, "_compile", lambda source, verbose: source)
    monkeypatch.setattr(build, "build_binding", fails)
    monkeypatch.setattr(build.subprocess, "run", link)
    with pytest.raises(RuntimeError, match="no host compiler"):
        build.build_library()
    assert (tmp_path / "libqgemm.so").exists()
