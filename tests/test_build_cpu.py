"""The library builds where there is no torch, or one without CUDA; only the binding needs it."""
import os
import shutil
import subprocess
import sys

import pytest

from conftest import ROOT

PACKAGE = "expert_dispatch_planning_gb300"


@pytest.fixture(scope="module")
def built():
    from expert_dispatch_planning_gb300 import build as b
    b.build()
    return b


@pytest.mark.parametrize("torch", ["missing", "without CUDA"])
def test_library_without_torch(built, tmp_path, torch):
    """A copy of the tree with its compiled objects (so that only linking is left), neither .so in it."""
    ignore = shutil.ignore_patterns("*.so", "__pycache__", "torch_binding.o")
    shutil.copytree(os.path.join(ROOT, PACKAGE), tmp_path / PACKAGE, ignore=ignore)
    shutil.copytree(os.path.join(ROOT, "include"), tmp_path / "include")
    if torch == "missing":
        fake = "sys.modules['torch'] = None"
    else:
        (tmp_path / "torch").mkdir()
        (tmp_path / "torch" / "__init__.py").write_text("")
        fake = "sys.path.insert(0, %r)" % str(tmp_path)
    code = "import sys; %s; sys.path.insert(0, %r); import build; print(build.build())" % (fake, str(tmp_path / PACKAGE))
    res = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=600)
    assert res.returncode == 0, res.stderr[-2000:]
    assert (tmp_path / PACKAGE / "libmoe_dispatch.so").exists()
    assert not (tmp_path / PACKAGE / "_torch_binding.so").exists()
