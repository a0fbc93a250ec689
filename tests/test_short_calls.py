"""The binding's compiled checks are a shorter way to calls that the library and the
binding make without them: they are not needed to load, nor to build (no GPU needed)."""
import os
import shutil
import subprocess
import sys
import warnings

import pytest
import torch

from paged_kv_cache_20_gb300 import _build
from tests.test_abi import lib  # noqa: F401  (fixture)

PROBE = """
import warnings
with warnings.catch_warnings(record=True) as seen:
    warnings.simplefilter("always")
    import paged_kv_cache_20_gb300 as pa
    print(pa.pa_decode_workspace_size(2, 8, 1, 128, 4), pa.status_string(-1), pa._fast)
    print([str(w.message) for w in seen if issubclass(w.category, RuntimeWarning)])
"""


def probe(root):
    r = subprocess.run([sys.executable, "-c", PROBE], cwd=root, capture_output=True, text=True, timeout=300)
    return r.returncode, r.stdout, r.stderr


@pytest.fixture
def copy(lib, tmp_path):  # noqa: F811
    """The package without its compiled checks."""
    at = tmp_path / "paged_kv_cache_20_gb300"
    at.mkdir()
    for name in ("__init__.py", "_build.py", "libpagedattn.so"):
        shutil.copy2(os.path.join(_build.HERE, name), at / name)
    return at


@pytest.mark.parametrize("calls", ["absent", "not a library", "of another torch"])
def test_loads_without_them(copy, calls):
    if calls == "not a library":
        (copy / "_calls.so").write_bytes(b"x" * 4096)
    elif calls == "of another torch":
        (copy / "_calls.py").write_text("torch_version = '1.0'\n")
    rc, out, err = probe(copy.parent)
    assert rc == 0, err
    lines = out.splitlines()
    assert lines[0] == f"{(2 * 4 * 8) * (128 + 2) * 4} PA_ERR_INVALID_ARG None"
    assert "_calls" in lines[1] and "_build.build()" in lines[1]


def test_loads_with_them(lib):  # noqa: F811
    import paged_kv_cache_20_gb300 as pa
    assert pa._fast.torch_version == torch.__version__


def test_a_missing_library_says_how_to_build_it(copy):
    os.remove(copy / "libpagedattn.so")
    rc, out, err = probe(copy.parent)
    assert rc != 0 and "RuntimeError" in err and "_build.build()" in err


@pytest.fixture
def elsewhere(monkeypatch, tmp_path):
    for name, at in (("CALLS", "_calls.so"), ("LIBRARY", "libpagedattn.so"), ("BUILD_DIR", "")):
        monkeypatch.setattr(_build, name, str(tmp_path / at))
    (tmp_path / "libpagedattn.so").write_bytes(b"")
    return tmp_path


@pytest.mark.parametrize("command", [["false"], ["/nowhere/g++"]])
def test_a_build_without_their_headers_warns(elsewhere, monkeypatch, command):
    (elsewhere / "_calls.so").write_bytes(b"stale")
    monkeypatch.setattr(_build, "calls_command", lambda out: command)
    with pytest.warns(RuntimeWarning, match="_calls"):
        _build.build_calls()
    assert not os.path.exists(_build.CALLS)      # (a stale one is not left to be loaded)
    assert not _build.needs_build()              # nothing to gain by trying again with this torch


def test_built_again_for_another_torch(elsewhere, monkeypatch):
    monkeypatch.setattr(_build, "calls_command", lambda out: ["touch", out])
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        _build.build_calls()
    assert os.path.exists(_build.CALLS) and not _build.needs_build()
    monkeypatch.setattr(torch, "__version__", "1.0")
    assert _build.needs_build()


def test_built_again_where_they_are_gone(elsewhere, monkeypatch):
    monkeypatch.setattr(_build, "calls_command", lambda out: ["touch", out])
    _build.build_calls()
    os.remove(_build.CALLS)
    assert _build.needs_build()
