"""Building the objectives' binding: what it lacks does not keep the optimizer step's library
from being built, and a binding of another torch or Python is built again.  The compiler is
not run here: the calls that would run it are recorded or fail."""
import os

import pytest

torch = pytest.importorskip("torch")

from loss_scaled_adamw_gb300 import _build


@pytest.fixture()
def binding(tmp_path, monkeypatch):
    """Binding and key in a temporary folder, the library taken to be up to date."""
    bind, calls = str(tmp_path / "_loss_bind.so"), []
    monkeypatch.setattr(_build, "BIND", bind)
    monkeypatch.setattr(_build, "BUILD", str(tmp_path))
    monkeypatch.setattr(_build, "_build_library", lambda srcs, verbose: calls.append("library"))

    def run(cmd, *args, **kw):
        calls.append(cmd[0])
        open(cmd[cmd.index("-o") + 1], "w").close()

    monkeypatch.setattr(_build, "_run", run)
    return bind, calls


@pytest.mark.parametrize("error", [FileNotFoundError(2, "g++"), RuntimeError("g++ failed: Python.h: No such file")])
def test_a_binding_that_cannot_be_built_is_a_warning(binding, monkeypatch, error):
    bind, _ = binding
    open(bind, "w").close()                # of before: other structures, perhaps

    def run(*args, **kw):
        raise error

    monkeypatch.setattr(_build, "_run", run)
    with pytest.warns(RuntimeWarning, match="g\\+\\+"):
        assert _build.build(force=True) == _build.LIB
    assert not os.path.exists(bind)        # nothing is left that could be loaded in its place
    with pytest.warns(RuntimeWarning):     # and the next build tries again
        _build.build()


def test_another_torch_builds_the_binding_again(binding, monkeypatch):
    bind, calls = binding
    _build.build()
    assert os.path.exists(bind) and calls.count("g++") == 1
    _build.build()
    assert calls.count("g++") == 1
    key = _build._binding_key()
    monkeypatch.setattr(_build, "_binding_key", lambda: key + " of another day")
    _build.build()
    _build.build()
    assert calls.count("g++") == 2
