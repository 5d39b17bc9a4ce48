"""The build on the host: the C library does not need torch."""
import os

import pytest

from helpers import build_lib


@pytest.mark.parametrize("torch", ["absent", "without CUDA"])
def test_library_builds_without_torch(torch, monkeypatch, tmp_path):
    """No torch, or one without CUDA: the library is built, the binding left out."""
    from lossless_lookahead_decoding_gb300 import build as B
    build_lib()  # (its objects are there)
    (tmp_path / "torch").mkdir()
    spec = None
    if torch != "absent":
        spec = type("Spec", (), {"origin": str(tmp_path / "torch" / "__init__.py")})
    monkeypatch.setattr(B.importlib.util, "find_spec", lambda name: spec)
    monkeypatch.setattr(B, "BINDING", str(tmp_path / "_kv4.so"))
    monkeypatch.setattr(B, "LIB", str(tmp_path / "liblookahead.so"))
    assert B.build() == B.LIB and os.path.exists(B.LIB)
    assert not os.path.exists(B.BINDING)
