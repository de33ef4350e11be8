"""The build's parts (no GPU): the library needs neither PyTorch nor the call
module, and what is out of date or does not fit is not used in silence."""
import os
import time

import pytest

import conv2d_backward_implicit_dgrad_gb300.binding as binding
import conv2d_backward_implicit_dgrad_gb300.build as build

SMALL = 'extern "C" int answer() { return 42; }\n'


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A library of one small source and a call module that does not compile, in a folder of their own."""
    (tmp_path / "csrc").mkdir()
    (tmp_path / "csrc" / "one.cu").write_text(SMALL)
    (tmp_path / "bind.cpp").write_text("this is not C++\n")
    out = tmp_path / "out"
    for name, value in dict(CSRC=tmp_path / "csrc", BUILD=out, LIB=out / "libsmall.so", BIND=out / "_bind.so",
                            BIND_SRC=tmp_path / "bind.cpp").items():
        monkeypatch.setattr(build, name, str(value))
    return tmp_path


def test_library_builds_without_pytorch(tree, monkeypatch):
    real = build.importlib.util.find_spec
    monkeypatch.setattr(build.importlib.util, "find_spec", lambda name, *a: None if name == "torch" else real(name, *a))
    assert not build.up_to_date()
    build.build()
    assert os.path.exists(build.LIB) and build.up_to_date()
    with pytest.raises(RuntimeError, match="PyTorch not found"):
        build.build_bind()


def test_library_stands_when_the_call_module_does_not_compile(tree):
    build.build()
    assert build.up_to_date()
    os.remove(build.LIB)
    with pytest.raises(RuntimeError, match="g\\+\\+ on bind.cpp"):
        build.build_all()
    assert build.up_to_date() and not build.bind_fits()


def test_an_error_in_the_library_is_raised(tree):
    (tree / "csrc" / "one.cu").write_text("int x = ;\n")
    with pytest.raises(RuntimeError, match="one.cu"):
        build.build()
    assert not os.path.exists(build.LIB)


def test_a_call_module_of_another_pytorch_does_not_fit(tree, monkeypatch):
    os.makedirs(build.BUILD)
    for name, text in ((build.BIND, ""), (build.BIND + ".for", build._bind_key())):
        with open(name, "w") as f:
            f.write(text)
    assert build.bind_fits() and build.bind_up_to_date()
    later = time.time() + 10
    os.utime(build.BIND_SRC, (later, later))
    assert build.bind_fits() and not build.bind_up_to_date()
    other = tree / "torch"
    other.mkdir()
    (other / "version.py").write_text("__version__ = '0.0'\n")
    monkeypatch.setattr(build, "_torch_dir", lambda: str(other))
    assert not build.bind_fits() and not build.bind_up_to_date()


def test_an_older_library_is_used_with_a_warning(tree, monkeypatch):
    build.build()
    later = time.time() + 10
    os.utime(tree / "csrc" / "one.cu", (later, later))
    (tree / "csrc" / "one.cu").write_text("int x = ;\n")
    os.utime(tree / "csrc" / "one.cu", (later, later))
    assert not build.up_to_date()

    class Found(Exception):
        pass

    def load(path):
        raise Found(path)

    monkeypatch.setattr(binding, "_LIB", None)
    monkeypatch.setattr(binding.ctypes, "CDLL", load)
    with pytest.warns(RuntimeWarning, match="older than its sources"):
        with pytest.raises(Found):
            binding.load_library()
    os.remove(build.LIB)
    with pytest.raises(RuntimeError, match="missing and could not be built"):
        binding.load_library()


def test_warnings_are_not_switched_off():
    with open(build.__file__) as f:
        text = f.read()
    assert "-diag-suppress" not in text and '"-w"' not in text
