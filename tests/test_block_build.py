"""The build and the import of the block calls' binding (no GPU)."""
import os
import shutil
import subprocess
import sys
import sysconfig

import pytest

import __graft_entry__ as entry


@pytest.fixture()
def build():
    entry.build_library()
    return entry._build_script()


def test_the_binding_is_named_for_its_interpreter(build, monkeypatch):
    """Another interpreter's binding is not taken for this one's: it is missing,
    which the build sees."""
    import paged_kv_cache_136_gb300 as pa
    suffix = sysconfig.get_config_var("EXT_SUFFIX")
    assert os.path.basename(build.BLOCK_CALLS) == "pa_block_calls" + suffix
    assert pa._block_calls.bind and pa._load_block_calls().__file__ == build.BLOCK_CALLS
    assert not build._stale()
    monkeypatch.setattr(build, "BLOCK_CALLS", build.BLOCK_CALLS.replace(suffix, ".other.so"))
    assert build._stale()


def test_the_other_calls_do_not_need_the_binding(build, tmp_path):
    """Without it the package is imported and its other calls work; the block
    calls say what is missing."""
    here = os.path.dirname(build.__file__)
    package = tmp_path / os.path.basename(here)
    (package / "_lib").mkdir(parents=True)
    shutil.copy(os.path.join(here, "__init__.py"), package)
    shutil.copy(build.LIB, package / "_lib")
    code = f"""
import {package.name} as pa
assert pa.pa_version() > 0 and pa.lib_path().startswith({str(tmp_path)!r})
assert pa.pa_block_decode_workspace_size(32, 8, 128) > 0
for _ in range(2):
    try:
        pa.pa_select_blocks(*[None] * 10)
    except ImportError as e:
        assert "pa_block_calls" in str(e)
    else:
        raise AssertionError("the call was made")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=tmp_path, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_a_build_without_headers_leaves_the_binding_out(build, tmp_path, monkeypatch, capfd):
    monkeypatch.setattr(build, "_python_headers", lambda: None)
    monkeypatch.setattr(build, "BLOCK_CALLS", str(tmp_path / "pa_block_calls.so"))
    assert not build._stale()                           # nothing that could be built is missing
    build._build_block_calls()
    assert not os.path.exists(build.BLOCK_CALLS) and "Python.h" in capfd.readouterr().err


def test_a_binding_that_does_not_compile_is_an_error(build, tmp_path, monkeypatch):
    monkeypatch.setattr(build, "BLOCK_CALLS", str(tmp_path / "pa_block_calls.so"))
    monkeypatch.setattr(build, "CSRC", str(tmp_path))
    with pytest.raises(RuntimeError, match="gcc failed"):
        build._build_block_calls()
