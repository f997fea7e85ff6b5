"""The package without its native tensor calls: they are a faster way to the same calls, so a host on
which they were not built, or not for this torch, still has everything.  CPU only."""
import importlib.util
import os
import subprocess
import sys

import pytest

from test_abi_host import moe  # noqa: F401  (the built library)

PKG = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "moe_expert_layer_fp32_gb300")
USE = """
import warnings, torch
with warnings.catch_warnings(record=True) as seen:
    warnings.simplefilter("always")
    import moe_expert_layer_fp32_gb300 as moe
assert [w for w in seen if "tensor calls" in str(w.message)], seen
assert not moe.NATIVE_TENSOR_CALLS and moe.moe_mx4_packed_bytes(2, 256, 128) == 2 * 17408
for call in (lambda: moe.route_select(torch.zeros(4, 8), 2), lambda: moe.mx4_quantize(torch.zeros(4, 64))):
    try:
        call()
    except ValueError as e:
        assert "CUDA device" in str(e)
    else:
        raise AssertionError("no refusal")
"""


def build_script():
    spec = importlib.util.spec_from_file_location("moe_build_script", os.path.join(PKG, "build.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("extension", [None, "garbage", "other torch"])
def test_import_without_native_calls(moe, tmp_path, extension):  # noqa: F811
    pkg = tmp_path / "moe_expert_layer_fp32_gb300"
    pkg.mkdir()
    for f in ("__init__.py", "libmoe_gb300.so"):
        os.symlink(os.path.join(PKG, f), pkg / f)
    if extension == "garbage":
        (pkg / "_tensor_calls.so").write_bytes(b"\x7fELF and nothing more")
    elif extension == "other torch":
        (pkg / "_tensor_calls.py").write_text("torch_version = '1.0'\ndef bind(path): pass\n")
    r = subprocess.run([sys.executable, "-c", USE], cwd=tmp_path, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr


def test_native_calls_are_used_where_they_are_built(moe):  # noqa: F811
    b = build_script()
    assert moe.NATIVE_TENSOR_CALLS == (b.calls_missing() is None)


def test_build_says_what_is_missing(monkeypatch):
    b = build_script()
    monkeypatch.setenv("CXX", "/nonexistent/compiler")
    assert "/nonexistent/compiler" in b.calls_missing()
    monkeypatch.setattr(b, "CALLS", "/nonexistent/calls.so")
    assert b.up_to_date() == (b.built_for_this_machine(b.LIB) and b.newest_source() <= os.path.getmtime(b.LIB))
