"""The binding's compiled module belongs to one torch and one Python: it is built again for another, and not loaded."""
import os
import time

import pytest

from mxfp8_block_scaled_07_b200 import build as mxbuild


@pytest.fixture(scope="module")
def mx():
    mxbuild.build()
    from mxfp8_block_scaled_07_b200 import mx

    return mx


def test_the_module_carries_what_it_was_built_for(mx):
    import torch

    assert torch.__version__ in mxbuild.call_tag()
    assert mxbuild.built_for() == mxbuild.call_tag() and not mxbuild.call_needs_build()


def test_another_torch_asks_for_a_build_and_is_not_loaded(mx, monkeypatch):
    import torch

    monkeypatch.setattr(torch, "__version__", "0.0.1")
    assert mxbuild.call_needs_build()
    monkeypatch.setattr(mx, "_mxcall", None)
    with pytest.raises(ImportError, match="built for torch .*, this is torch 0.0.1 .*run python -m"):
        mx.route(None, 1)


def test_a_module_without_a_tag_is_built_again(mx, monkeypatch, tmp_path):
    old = tmp_path / "_mxcall.so"
    old.write_bytes(b"\x7fELF of a build before it carried one")
    os.utime(old, (time.time() + 60,) * 2)
    assert mxbuild.built_for(str(old)) is None
    monkeypatch.setattr(mxbuild, "CALL_LIB", str(old))
    monkeypatch.setattr(mxbuild, "built_for", lambda lib=str(old), f=mxbuild.built_for: f(lib))
    assert mxbuild.call_needs_build()
