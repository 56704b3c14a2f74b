"""What build() makes when something that the Python module needs is missing (compilers
stand in for the real ones: they only write their output file)."""
import os
import stat
import sys

import pytest

from speculative_decoding_rejection_02_gb300 import _build

FAKE = """#!{python}
import sys
assert {ok}, "no compiler"
open(sys.argv[sys.argv.index("-o") + 1], "w").write("built")
"""


@pytest.fixture
def place(tmp_path, monkeypatch):
    """An empty output folder, and compilers that write "built"."""
    def tool(name, ok=True):
        path = tmp_path / "bin" / name
        path.parent.mkdir(exist_ok=True)
        path.write_text(FAKE.format(python=sys.executable, ok=ok))
        path.chmod(path.stat().st_mode | stat.S_IXUSR)
        return str(path)
    lib = tmp_path / "_lib"
    monkeypatch.setattr(_build, "LIB_DIR", str(lib))
    monkeypatch.setattr(_build, "LIB_PATH", str(lib / "libspecverify.so"))
    monkeypatch.setattr(_build, "BINDING_PATH", str(lib / "_cache_binding.so"))
    monkeypatch.setattr(_build, "_nvcc", lambda: tool("nvcc"))
    tool("g++")
    monkeypatch.setenv("PATH", str(tmp_path / "bin"))
    return tool


def both():
    return os.path.exists(_build.LIB_PATH), os.path.exists(_build.BINDING_PATH)


def test_all_there(place):
    assert _build.build() == _build.LIB_PATH
    assert both() == (True, True)
    assert not [f for f in os.listdir(_build.LIB_DIR) if ".tmp" in f]


def test_without_torch(place, monkeypatch):
    find = _build.importlib.util.find_spec
    monkeypatch.setattr(_build.importlib.util, "find_spec",
                        lambda name, *a: None if name == "torch" else find(name, *a))
    with pytest.warns(UserWarning, match="torch"):
        assert _build.build() == _build.LIB_PATH
    assert both() == (True, False)
    with pytest.warns(UserWarning, match="torch"):  # and again, with nothing to compile
        _build.build()


def test_without_a_host_compiler(place, monkeypatch):
    os.remove(os.path.join(os.environ["PATH"], "g++"))
    with pytest.warns(UserWarning, match=r"g\+\+"):
        _build.build()
    assert both() == (True, False)


def test_failing_host_compiler(place):
    place("g++", ok=False)
    with pytest.raises(RuntimeError, match="cache_binding.cpp"):
        _build.build()
    assert both() == (True, False)  # the verifier's library does not need it


def test_failing_nvcc(place, monkeypatch):
    bad = place("nvcc", ok=False)
    monkeypatch.setattr(_build, "_nvcc", lambda: bad)
    with pytest.raises(RuntimeError, match="spec_verify.cu"):
        _build.build()
    assert not both()[0]
    assert not [f for f in os.listdir(_build.LIB_DIR) if ".tmp" in f]


def rebuilt(path):
    with open(path, "w") as f:
        f.write("kept")
    _build.build()
    return open(path).read() == "built"


def test_another_torch_rebuilds_the_module(place, monkeypatch):
    _build.build()
    assert not rebuilt(_build.BINDING_PATH)
    monkeypatch.setattr(_build, "torch_version", lambda: "1.0+other")
    assert rebuilt(_build.BINDING_PATH)
    _build.build()
    assert open(_build.LIB_PATH).read() == "built"


def test_a_module_for_another_torch_is_not_loaded(place, monkeypatch):
    import torch

    import speculative_decoding_rejection_02_gb300 as sv
    from speculative_decoding_rejection_02_gb300 import cache
    assert _build.torch_version() == str(torch.__version__)
    _build.build()
    _build.build(force=True)
    monkeypatch.setattr(torch, "__version__", "1.0+other")
    monkeypatch.setattr(sv, "lib", lambda: None)
    with pytest.raises(ImportError, match="1.0.other"):
        cache._Native().step
