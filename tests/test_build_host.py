"""What build() makes and when it makes it again, with the compilers replaced by a recorder."""
import os
import types

import pytest


@pytest.fixture
def bl(monkeypatch, tmp_path):
    """build_lib with its outputs under tmp_path; bl.ran holds the commands it gave."""
    import __graft_entry__
    m = __graft_entry__._load_build_lib()
    m.BUILD, m.LIBDIR = str(tmp_path / "build"), str(tmp_path / "lib")
    m.LIB, m.BINDING = os.path.join(m.LIBDIR, "lib.so"), os.path.join(m.LIBDIR, "_moe_binding.so")
    m.BINDING_FOR = os.path.join(m.BUILD, "moe_binding.txt")
    m.ran = []

    def run(cmd, **kw):
        m.ran.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")
    monkeypatch.setattr(m, "subprocess", types.SimpleNamespace(run=run))
    torch = tmp_path / "torch"
    (torch / "lib").mkdir(parents=True)
    (torch / "lib" / "libc10_cuda.so").touch()
    (torch / "version.py").write_text("__version__ = '1'\n")
    m.torch = torch
    find = m.importlib.util.find_spec

    def spec(name):
        if name != "torch":
            return find(name)
        return types.SimpleNamespace(submodule_search_locations=[str(m.torch)]) if m.torch is not None else None
    monkeypatch.setattr(m, "importlib", types.SimpleNamespace(util=types.SimpleNamespace(find_spec=spec)))
    return m


def _units(m):
    return len(m.sources())


def test_library_and_binding_then_nothing(bl):
    assert not bl.up_to_date()
    assert bl.build() == bl.LIB
    assert len(bl.ran) == _units(bl) + 1 + 2 and os.path.exists(bl.BINDING) and bl.up_to_date()
    bl.ran.clear()
    bl.build()
    assert bl.ran == []
    bl.build(force=True)
    assert len(bl.ran) == _units(bl) + 1 + 2


def test_another_torch_makes_the_binding_again(bl):
    bl.build()
    bl.ran.clear()
    (bl.torch / "version.py").write_text("__version__ = '2'\n")
    os.utime(bl.torch / "version.py", (1, 1))           # older than what was built, as an installed file is
    assert not bl.up_to_date()
    bl.build()
    assert [c[0].rsplit("/", 1)[-1] for c in bl.ran] == ["g++", "g++"] and bl.up_to_date()


def test_the_library_builds_without_torch(bl, capfd):
    bl.torch = None
    bl.build()
    assert len(bl.ran) == _units(bl) + 1 and os.path.exists(bl.LIB) and not os.path.exists(bl.BINDING)
    assert "not built" in capfd.readouterr().err and bl.up_to_date()


def test_a_torch_without_cuda_counts_as_none(bl):
    os.remove(bl.torch / "lib" / "libc10_cuda.so")
    bl.build()
    assert os.path.exists(bl.LIB) and not os.path.exists(bl.BINDING)
