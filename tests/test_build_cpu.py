"""What `python -m bit_matmul_lowbit_amd.build` makes, with the compilers
replaced by a record of their calls."""
import os
import sys

import pytest

from bit_matmul_lowbit_amd import build


@pytest.fixture
def made(monkeypatch):
    outs = []
    monkeypatch.setattr(build, "_run", lambda cmd, out, verbose: outs.append(os.path.basename(out)))
    return outs


def test_the_library_and_then_the_binding(made):
    assert build.build() == build.LIB
    assert made == ["liblowbit.so", "_marshal.so"]


def test_the_library_needs_no_torch(made, monkeypatch, capsys):
    """A user of the C interface has hipcc and no torch."""
    monkeypatch.setitem(sys.modules, "torch", None)
    assert build.build() == build.LIB
    assert made == ["liblowbit.so"]
    assert "_marshal.so" in capsys.readouterr().err


def test_the_library_is_there_when_the_binding_fails(monkeypatch):
    outs = []

    def run(cmd, out, verbose):
        if out == build.MARSHAL:
            raise RuntimeError("no Python headers")
        outs.append(out)

    monkeypatch.setattr(build, "_run", run)
    with pytest.raises(RuntimeError, match="no Python headers"):
        build.build()
    assert outs == [build.LIB]
