"""The build's order and the Python calls' stamp, with the compilers replaced by
a function that writes its output file (CPU)."""

import os

import pytest

from online_softmax_tiled_gb300 import _binding, _build


class Compilers:
    def __init__(self, fail=()):
        self.fail, self.made = tuple(fail), []

    def __call__(self, cmd):
        out = cmd[cmd.index("-o") + 1]
        name = os.path.basename(out)
        if any(name.startswith(f) for f in self.fail):
            raise RuntimeError("command failed: " + name)
        if "-shared" in cmd and "-l:libattn_gb300.so" in cmd:
            assert os.path.exists(_build.LIB_PATH)          # linked against it
        with open(out, "w") as f:
            f.write("built")
        self.made.append(name)
        return ""


@pytest.fixture
def tree(tmp_path, monkeypatch):
    lib = tmp_path / "_lib"
    monkeypatch.setattr(_build, "BUILD_DIR", str(tmp_path / "_build"))
    monkeypatch.setattr(_build, "LIB_DIR", str(lib))
    monkeypatch.setattr(_build, "LIB_PATH", str(lib / "libattn_gb300.so"))
    monkeypatch.setattr(_build, "CALLS_PATH", str(lib / "_cache_calls.so"))
    monkeypatch.setattr(_build, "STAMP_PATH", str(lib / "_cache_calls.so.stamp"))
    return lib


def _build_with(monkeypatch, **kw):
    run = Compilers(**kw)
    monkeypatch.setattr(_build, "_run", run)
    try:
        _build.build()
    except RuntimeError:
        run.made.append("error")
    return run.made


@pytest.mark.parametrize("fail", ["py_cache.o", "_cache_calls.so"])
def test_library_is_linked_where_the_calls_cannot_be_built(tree, monkeypatch, fail):
    made = _build_with(monkeypatch, fail=[fail])
    assert "libattn_gb300.so.tmp" in made and made[-1] == "error"
    assert (tree / "libattn_gb300.so").exists() and not (tree / "_cache_calls.so").exists()
    made = _build_with(monkeypatch)                         # the calls alone are left
    assert made == ["py_cache.o", "_cache_calls.so.tmp"]


def test_calls_are_rebuilt_for_another_torch(tree, monkeypatch):
    made = _build_with(monkeypatch)
    assert len(made) == len(_build.SOURCES) + 3
    assert _build_with(monkeypatch) == [] and _build.calls_current()
    monkeypatch.setattr(_build, "calls_stamp", lambda: "another python and torch")
    assert not _build.calls_current()
    assert _build_with(monkeypatch) == ["py_cache.o", "_cache_calls.so.tmp"]
    assert _build_with(monkeypatch) == [] and _build.calls_current()


def test_calls_of_another_torch_are_not_loaded(monkeypatch):
    import __graft_entry__
    __graft_entry__.build()
    monkeypatch.setattr(_binding, "_CALLS", None)
    monkeypatch.setattr(_build, "calls_stamp", lambda: "another python and torch")
    with pytest.raises(RuntimeError, match="another Python or torch"):
        _binding._calls()
