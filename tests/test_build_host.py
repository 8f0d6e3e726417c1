"""What build() does in which order, when the torch-side module counts as current and what loading an older library
says (CPU)."""
import os
import subprocess

import pytest

from feed_forward_view_vggt_b200 import attn
from feed_forward_view_vggt_b200 import build as vbuild


@pytest.fixture
def commands(tmp_path, monkeypatch):
    """The compiler calls of a build into an empty folder; each writes a file with its command line."""
    ran = []

    def run(cmd, check):
        ran.append(cmd)
        out = cmd[cmd.index("-o") + 1]
        with open(out, "w") as f:
            f.write("\n".join(cmd))

    monkeypatch.setattr(vbuild.subprocess, "run", run)
    for name in ("LIB", "DEBUG_LIB", "BINDING"):
        monkeypatch.setattr(vbuild, name, str(tmp_path / os.path.basename(getattr(vbuild, name))))
    return ran


def test_the_library_is_built_where_the_module_cannot_be(commands, monkeypatch):
    def no_torch(*a, **k):
        raise ImportError("no torch here")

    monkeypatch.setattr(vbuild, "build_binding", no_torch)
    with pytest.raises(ImportError):
        vbuild.build()
    assert len(commands) == 1 and os.path.exists(vbuild.LIB)


def test_a_build_does_what_is_missing(commands):
    assert vbuild.build() == vbuild.LIB and len(commands) == 2
    assert vbuild.build() == vbuild.LIB and len(commands) == 2
    assert vbuild.build(debug=True) == vbuild.DEBUG_LIB and len(commands) == 3
    vbuild.build(force=True)
    assert len(commands) == 5


def test_the_module_is_rebuilt_for_another_torch(commands, monkeypatch):
    import torch

    vbuild.build()
    monkeypatch.setattr(torch, "__version__", "99.0")
    vbuild.build()
    assert len(commands) == 3 and "99.0" in " ".join(commands[2])
    vbuild.build()
    assert len(commands) == 3


def test_the_built_module_says_what_it_is_for():
    vbuild.build()
    import torch  # noqa: F401
    from feed_forward_view_vggt_b200 import _streaming

    assert _streaming.built_for == vbuild.binding_is_for()


def test_a_library_of_the_same_version_without_an_entry_point_is_refused(tmp_path):
    lib = str(tmp_path / "old.so")
    older = [n for n in attn.declared_symbols() if n != "vggt_attn_cached"]
    code = "".join(f"int {n}(void) {{ return {attn.ABI_VERSION}; }}\n" for n in older)
    subprocess.run([os.environ.get("CC", "gcc"), "-shared", "-fPIC", "-x", "c", "-", "-o", lib], input=code.encode(),
                   check=True)
    with pytest.raises(RuntimeError, match="no vggt_attn_cached; rebuild"):
        attn.load_library(lib)
