"""The Python extension of the feed-forward forms as a part that the library is whole without
(no GPU): what does not compile warns and leaves the Python forms, once for each torch and
Python; another torch than the one it was built for has it built again."""
import os
import warnings

import pytest

from dense_fp16_tensor_gemm_gb300 import _build


@pytest.fixture
def place(monkeypatch, tmp_path):
    """The extension's file elsewhere, the library's as it is; `made`: what is run."""
    _build.build()
    made = []
    monkeypatch.setattr(_build, "CALLS", str(tmp_path / "_tensor_calls.so"))
    monkeypatch.setattr(_build, "CALLS_FOR", str(tmp_path / "_tensor_calls.so.for"), raising=False)

    def use(*command):
        def one(out):
            if out.endswith(str(os.getpid())):
                made.append(out)
            return [a.replace("OUT", out) for a in command] or None
        monkeypatch.setattr(_build, "_calls_command", one)
    return use, made


@pytest.mark.parametrize("command", [("g++", "-x", "c++", "-c", os.devnull, "--no-such-option"), ("/nonexistent/g++",)])
def test_what_does_not_compile_is_a_warning(place, command):
    use, made = place
    use(*command)
    with open(_build.CALLS, "w") as f:
        f.write("of another torch")
    with pytest.warns(UserWarning, match="does not compile"):
        assert _build.build() == _build.LIB
    assert not os.path.exists(_build.CALLS) and len(made) == 1
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        assert _build.build() == _build.LIB  # and is not tried again
    assert len(made) == 1


def test_built_once_for_each_torch(place, monkeypatch):
    use, made = place
    use("cp", os.devnull, "OUT")
    for _ in range(2):
        _build.build()
        assert os.path.exists(_build.CALLS) and len(made) == 1
    version = _build.importlib.metadata.version
    monkeypatch.setattr(_build.importlib.metadata, "version", lambda name: "2.0.1" if name == "torch" else version(name))
    _build.build()
    assert len(made) == 2
    _build.build()
    assert len(made) == 2
    os.remove(_build.CALLS)
    _build.build()
    assert len(made) == 3


def test_a_machine_without_what_it_needs_builds_nothing(place):
    use, made = place
    use()
    assert _build.build() == _build.LIB
    assert not made[1:] and not os.path.exists(_build.CALLS_FOR)


def test_a_folder_that_cannot_be_written_is_left_alone(place, monkeypatch):
    use, made = place
    use("cp", os.devnull, "OUT")
    monkeypatch.setattr(_build.os, "access", lambda path, mode: path != _build.OUT_DIR)
    assert _build.build() == _build.LIB and not made


def test_no_toolkit_no_extension(monkeypatch):
    def missing():
        raise RuntimeError("nvcc not found")
    monkeypatch.setattr(_build, "nvcc", missing)
    assert _build._calls_command("x") is None
