"""What is built when: the library alone for the verification, the cache's binding
for the versions of Python and torch that load it."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture()
def build():
    from speculative_decoding_verification_69_gb300 import _build
    return _build


def test_the_library_loads_without_the_binding(tmp_path):
    """No binding, and no compiler for one: the verification's entry points are
    there, the cache's say what is missing."""
    code = """
import speculative_decoding_verification_69_gb300 as sv
from speculative_decoding_verification_69_gb300 import _build
_build.native_path = lambda: %r
_build._binding_cmd = lambda: ["a-compiler-that-is-not-there"]
assert sv.load_library().spec_tree_attention_workspace_bytes(1, 1, 1, 1, 64) > 0
try:
    sv.cache_resize(None, None, None, None, 16)
except sv.SpecVerifyError as e:
    assert "binding" in str(e)
    print("refused")
""" % str(tmp_path / "_native.so")
    from speculative_decoding_verification_69_gb300 import _build
    _build.build_library()
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    assert r.stdout.strip() == "refused"
    assert not os.listdir(tmp_path)


def test_the_binding_belongs_to_one_torch_and_python(build, monkeypatch):
    import sysconfig

    import torch
    here = build.native_path()
    assert here.endswith(".so") and os.path.dirname(here) == build.OUT_DIR
    names = {here}
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", "2.99.0+other")
        names.add(build.native_path())
        assert build.binding_stale()
    with monkeypatch.context() as m:
        m.setattr(torch._C, "_GLIBCXX_USE_CXX11_ABI", not torch._C._GLIBCXX_USE_CXX11_ABI)
        names.add(build.native_path())
    with monkeypatch.context() as m:
        m.setattr(sysconfig, "get_config_var", lambda name: "cpython-399-other")
        names.add(build.native_path())
    assert len(names) == 4 and build.native_path() == here


def test_both_are_built_by_build(build, monkeypatch):
    ran = []
    monkeypatch.setattr(build, "_run", lambda cmd, out, verbose: ran.append(out))
    build.build(force=True)
    assert ran == [build.LIB, build.native_path()]
