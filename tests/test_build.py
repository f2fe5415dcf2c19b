"""What is built and loaded without what it does not need."""
import subprocess
import sys

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
