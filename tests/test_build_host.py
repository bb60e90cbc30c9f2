"""The build's order of work (host only, no compiler run): the C library needs hipcc alone."""
import os
import sys

import pytest

from gated_delta_rule_prologue_amd import build as B


@pytest.fixture
def made(monkeypatch, tmp_path):
    """The commands that a build runs, each leaving its output file; fail[word] raises for them."""
    cmds, fail = [], set()

    def run(cmd, verbose):
        cmds.append(cmd)
        if any(w in " ".join(cmd) for w in fail):
            raise RuntimeError("command failed: " + " ".join(cmd))
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("\n")

    monkeypatch.setattr(B, "_run", run)
    monkeypatch.setattr(B, "BUILD", str(tmp_path / "obj"))
    monkeypatch.setattr(B, "LIB", str(tmp_path / "libprism.so"))
    monkeypatch.setattr(B, "CALLS", str(tmp_path / "_calls.so"))
    return cmds, fail


def test_both_are_built(made):
    cmds, _ = made
    assert B.build() == B.LIB
    assert os.path.exists(B.LIB) and os.path.exists(B.CALLS)
    assert sum("torch_calls.cpp" in " ".join(c) for c in cmds) == 1
    assert not [f for f in os.listdir(os.path.dirname(B.LIB)) if ".tmp" in f]


def test_the_library_needs_no_torch(made, monkeypatch, capsys):
    cmds, _ = made
    monkeypatch.setitem(sys.modules, "torch", None)          # import torch raises
    open(B.CALLS, "w").close()
    assert B.build() == B.LIB and os.path.exists(B.LIB)
    assert not any("torch_calls" in " ".join(c) for c in cmds)
    assert not os.path.exists(B.CALLS)                       # none of an earlier build beside a newer library
    assert "_calls.so" in capsys.readouterr().out


@pytest.mark.parametrize("word", ["torch_calls.cpp", "-ltorch_python"])
def test_a_failure_of_the_calls_leaves_the_library(made, word):
    _, fail = made
    fail.add(word)
    open(B.CALLS, "w").close()
    with pytest.raises(RuntimeError, match="command failed"):
        B.build()
    assert os.path.exists(B.LIB) and not os.path.exists(B.CALLS)


def test_a_failure_of_the_library_is_raised(made):
    _, fail = made
    fail.add("decode.hip")
    open(B.CALLS, "w").close()
    with pytest.raises(RuntimeError, match="decode.hip"):
        B.build()
    assert not os.path.exists(B.LIB) and os.path.exists(B.CALLS)       # nothing was replaced
