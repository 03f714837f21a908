"""The module that makes the calls of the microscaled operators, where it is not there or was
built for another interpreter (no GPU needed)."""
import os
import shutil
import subprocess
import sys
import sysconfig
import types

import pytest

import bit_group_quantized_qgemv_gb300 as q
from bit_group_quantized_qgemv_gb300 import build


def test_the_module_is_the_interpreters_own():
    assert os.path.basename(build.CALLS) == "_mx_calls" + sysconfig.get_config_var("EXT_SUFFIX")
    assert os.path.exists(build.CALLS)


def test_all_else_works_without_the_module(tmp_path):
    package = os.path.dirname(q.__file__)
    shutil.copytree(package, tmp_path / os.path.basename(package), ignore=shutil.ignore_patterns("*.o", "_mx_calls*", "__pycache__"))
    # (a module without the interpreter's suffix is not its own)
    (tmp_path / os.path.basename(package) / "_build" / "_mx_calls.so").write_bytes(b"for another interpreter")
    code = """
import torch, bit_group_quantized_qgemv_gb300 as q
assert q.lib.qgemv_version() and q.strerror(0)
x, w = torch.zeros(2, 64).half(), (torch.zeros(8, 8, dtype=torch.int32), torch.zeros(8, 2, dtype=torch.uint8))
c = torch.zeros(2, 64, dtype=torch.uint8), torch.zeros(2, 2, dtype=torch.uint8)
for call in (lambda: q.mx_quantize(x), lambda: q.mx_dequantize(*c), lambda: q.residual_rmsnorm_mxfp8(x, x[0]),
             lambda: q.qgemv_mxfp4(w, x), lambda: q.mx_gemm(w, c), lambda: q.mx_swiglu(w, w, c)):
    try:
        call()
    except ImportError as e:
        assert "_mx_calls" in str(e)
    else:
        assert False
print("done")
"""
    env = {**os.environ, "PYTHONPATH": str(tmp_path)}
    env.pop("QGEMV_LIB", None)
    r = subprocess.run([sys.executable, "-c", code], cwd=tmp_path, env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout == "done\n", r.stderr[-2000:]


@pytest.mark.parametrize("how", ["no compiler", "no headers"])
def test_the_library_is_built_without_the_module(tmp_path, monkeypatch, how):
    def run(cmd, **kw):
        if cmd[0] == "gcc":
            if how == "no compiler":
                raise FileNotFoundError("gcc")
            return types.SimpleNamespace(returncode=1, stderr="Python.h: No such file or directory")
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("new")
        return types.SimpleNamespace(returncode=0, stderr="")

    monkeypatch.setattr(build, "subprocess", types.SimpleNamespace(run=run))
    for name, file in (("BUILD", ""), ("LIB", "libqgemv.so"), ("CALLS", "_mx_calls.x.so")):
        monkeypatch.setattr(build, name, str(tmp_path / file))
    (tmp_path / "_mx_calls.x.so").write_text("of an older library")
    with pytest.raises(RuntimeError, match="gcc"):
        build.build(force=True)
    assert (tmp_path / "libqgemv.so").read_text() == "new"
    assert not (tmp_path / "_mx_calls.x.so").exists() and not build.up_to_date()
