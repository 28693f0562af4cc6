"""The binding where the compiled module of the operators' calls is missing, was built for another PyTorch or
cannot be built (the library is usable, and ctypes takes every call), and what it refuses."""
import os
import shutil
import subprocess
import sys

import pytest

USE = """
import warnings
with warnings.catch_warnings(record=True) as seen:
    warnings.simplefilter("always")
    from lazy_optimizers_embedding_gb300 import binding as so
import torch
print("warned" if any("ctypes" in str(w.message) for w in seen) else "quiet")
f, m, e = torch.zeros(4, 8), torch.zeros(4), torch.zeros(1, dtype=torch.int32)
assert so._pycall.layer_norm(f, 4, 8, None, 4, None, None, 1e-5, f, m, m, e, None) is None
try:                                        # the table step's call and an operator's: tensors of the host
    so.sparse_read_rows(f, 4, 8, None, 4, f, e)
except ValueError:
    pass
try:
    so.sparse_layer_norm(f, 4, 8, None, 4, None, None, 1e-5, f, m, m, e)
except ValueError as x:
    assert "CUDA" in str(x)
else:
    raise AssertionError
assert so.sparse_workspace_size(10, 4, 100) > 0 and so.sparse_muon_workspace_size(1, 8, 8, 3) > 0
"""


@pytest.fixture
def package(tmp_path):
    """A copy of the built package, without the module."""
    from lazy_optimizers_embedding_gb300 import build
    build.build()
    to = tmp_path / "lazy_optimizers_embedding_gb300"
    shutil.copytree(build.PKG, to, ignore=shutil.ignore_patterns("__pycache__", "*.o"))
    os.remove(to / os.path.basename(build.PYCALL))
    return to


def _run(package, code, **env):
    r = subprocess.run([sys.executable, "-c", code], cwd=package.parent, capture_output=True, text=True,
                       env={**os.environ, "PYTHONPATH": str(package.parent), **env})
    assert r.returncode == 0, r.stderr
    return r.stdout


def test_the_module_is_missing(package):
    assert _run(package, USE).split() == ["warned"]


def test_the_module_is_another_pytorchs(package):
    from lazy_optimizers_embedding_gb300 import build
    shutil.copy(build.PYCALL, package)
    assert _run(package, USE).split() == ["quiet"]
    stamp = package / "_build" / os.path.basename(build.PYCALL_STAMP)
    stamp.write_text(build.pycall_key() + "0")
    assert _run(package, USE).split() == ["warned"]


def test_the_module_cannot_be_built(package):
    shutil.copytree(os.path.join(os.path.dirname(os.path.dirname(__file__)), "include"), package.parent / "include")
    for f in ("libsparseopt.so", "_build/defines.txt"):      # as new as their sources' copies
        os.utime(package / f)
    code = """
import sys
from lazy_optimizers_embedding_gb300 import build as b
b.build()
assert not b._pycall_stale() and not b.pycall_usable()       # not tried again until something changes
"""
    _run(package, code, CXX="/bin/false")
    assert _run(package, USE).split() == ["warned"]


def test_another_pytorch_makes_the_module_stale(monkeypatch):
    from lazy_optimizers_embedding_gb300 import build
    build.build()
    assert not build._pycall_stale()
    monkeypatch.setattr(build, "pycall_key", lambda: "another")
    assert build._pycall_stale() and not build.pycall_usable()


def test_a_pointer_where_a_tensor_says_the_type():
    """An array whose type the call takes from it cannot come as an integer."""
    import torch

    from lazy_optimizers_embedding_gb300 import binding as so
    e = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(TypeError, match="x: must be a tensor"):
        so.sparse_layer_norm(256, 4, 8, None, 4, None, None, 1e-5, 256, None, None, e)
    with pytest.raises(TypeError, match="u: must be a tensor"):
        so.sparse_orthogonalize(256, 1, 4, 8, so.NsConfig(), 256, None, e)
