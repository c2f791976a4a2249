"""The build where the Python module's needs are absent."""
import os

import pytest

from conv_bn_silu_amd import build

pytestmark = pytest.mark.cpu


def test_the_library_needs_no_torch(monkeypatch, tmp_path, capsys):
    """Without g++, PyTorch's or Python's headers the module is left out, and one of another build removed; the
    library's own steps have succeeded by then and build() returns it."""
    for missing in ("g++", "torch", "headers"):
        module = tmp_path / "_block8.so"
        module.write_text("of another build")
        with monkeypatch.context() as m:
            m.setattr(build, "MODULE", str(module))
            if missing == "g++":
                m.setattr(build.shutil, "which", lambda name: None)
            elif missing == "torch":
                m.setattr(build.importlib.util, "find_spec", lambda name: None)
            else:
                m.setattr(build.sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
            ran = []
            m.setattr(build.subprocess, "run", lambda *a, **k: ran.append(a))
            assert build.build_module() is None
        assert not ran and not os.path.exists(module)
        assert "_block8.so is not built" in capsys.readouterr().err


def test_nothing_is_missing_here():
    assert build._module_needs()[1] == []
