"""The build and the import of the block calls' binding (no GPU)."""
import os
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
