"""What is built and loaded without what it does not need."""
import os
import subprocess
import sys

import pytest

from draft_selection_gb300 import build as dbuild


def test_the_library_loads_without_torch_or_the_extension(tmp_path):
    """Without torch, and without the extension that only the cache and tree calls need, the
    package is imported and the library loaded; a call that needs the extension says so."""
    code = """
import sys
sys.modules["torch"] = None                     # an import of torch raises ImportError
import draft_selection_gb300 as dfl2
from draft_selection_gb300 import build
build.CALLS += ".none"
assert dfl2.dfl2_version() and dfl2.load().dfl2_topk_workspace_size(0, 1, 16) == 0
try:
    dfl2.dfl2_cache_free(None, None)
except RuntimeError as e:
    assert "is missing" in str(e)
else:
    raise SystemExit("no error")
"""
    dbuild.build()
    r = subprocess.run([sys.executable, "-c", code], cwd=dbuild.ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


@pytest.fixture
def elsewhere(tmp_path, monkeypatch):
    """The build's results in a folder of their own; its commands are listed, and make empty files."""
    for name, file in (("LIB", "libdfl2.so"), ("CALLS", "_calls.so"), ("BUILD", "_build")):
        monkeypatch.setattr(dbuild, name, str(tmp_path / file))
    ran = []

    def run(cmd, **kw):
        ran.append([os.path.basename(x) for x in cmd])
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(dbuild.subprocess, "run", run)
    return ran


def test_without_torch_the_library_is_built(elsewhere, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)
    dbuild.build()
    assert os.path.exists(dbuild.LIB) and not os.path.exists(dbuild.CALLS)
    assert not any("calls.cpp" in cmd for cmd in elsewhere) and dbuild.is_fresh()


def test_without_a_host_compiler_the_library_is_built(elsewhere, monkeypatch):
    def no_compiler(*a):
        raise RuntimeError("g++ not found")

    monkeypatch.setattr(dbuild, "calls_cmds", no_compiler)
    with pytest.raises(RuntimeError, match="not found"):
        dbuild.build()
    assert os.path.exists(dbuild.LIB) and not os.path.exists(dbuild.CALLS)


def test_each_library_is_rebuilt_for_its_own_sources(elsewhere, monkeypatch):
    dbuild.build()
    assert sum("calls.cpp" in cmd for cmd in elsewhere) == 1 and dbuild.is_fresh()
    os.remove(dbuild.CALLS)
    elsewhere.clear()
    dbuild.build()
    assert dbuild.is_fresh() and [("calls.cpp" in cmd) for cmd in elsewhere] == [True, False]


def test_the_extension_is_rebuilt_for_another_torch_or_python(elsewhere, monkeypatch):
    dbuild.build()
    version = dbuild.importlib.metadata.version
    assert dbuild.is_fresh()
    monkeypatch.setattr(dbuild.importlib.metadata, "version", lambda name: version(name) + ".1")
    assert dbuild.lib_fresh() and not dbuild.is_fresh()
    elsewhere.clear()
    dbuild.build()
    assert dbuild.is_fresh() and [("calls.cpp" in cmd) for cmd in elsewhere] == [True, False]
    var = dbuild.sysconfig.get_config_var
    monkeypatch.setattr(dbuild.sysconfig, "get_config_var", lambda name: var(name) + "-other")
    assert not dbuild.is_fresh()
