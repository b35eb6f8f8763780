"""What the build runs, with and without torch (nothing is compiled here)."""
import os

import pytest

from vector_compression_b200 import build as b


@pytest.mark.parametrize("torch", [True, False])
def test_the_library_is_built_without_torch(torch, tmp_path, monkeypatch):
    ran = []

    class Done:
        returncode = 0

        def __init__(self, cmd, **_):
            ran.append(cmd)
            open(cmd[cmd.index("-o") + 1], "w").close()

        def communicate(self):
            return b"", None

    monkeypatch.setattr(b, "HERE", str(tmp_path))
    monkeypatch.setattr(b, "LIB", str(tmp_path / "libtq.so"))
    monkeypatch.setattr(b, "BINDING", str(tmp_path / "_torch_binding.so"))
    monkeypatch.setattr(b.subprocess, "Popen", Done)
    monkeypatch.setattr(b.subprocess, "run", Done)
    if not torch:
        find = b.importlib.util.find_spec
        monkeypatch.setattr(b.importlib.util, "find_spec", lambda n, *a: None if n == "torch" else find(n, *a))
        monkeypatch.setattr(b, "binding_commands", lambda *a: pytest.fail("needs torch"))
    assert b.needs_build()
    assert b.build() == b.LIB and os.path.exists(b.LIB)
    assert os.path.exists(b.BINDING) == torch
    assert len(ran) == len(b.sources()) + 1 + 2 * torch
    assert not b.needs_build()
    os.utime(b.LIB, (1, 1))
    assert b.needs_build()
