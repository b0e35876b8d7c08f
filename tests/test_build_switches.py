"""A source whose extra compiler switch is not known is built without it; other errors stay errors."""
import os
import stat

import pytest

from bit_quantized_moe_dequant_amd import build

SCRIPT = """#!/bin/sh
case "$*" in
  *-some-switch*) echo "clang: Unknown command line argument '-some-switch'." >&2; exit 1;;
  *broken.hip*) echo "error: expected ';'" >&2; exit 1;;
esac
while [ $# -gt 0 ]; do [ "$1" = -o ] && echo "object" > "$2"; shift; done
"""


@pytest.fixture
def compiler(tmp_path, monkeypatch):
    exe = tmp_path / "hipcc"
    exe.write_text(SCRIPT)
    exe.chmod(exe.stat().st_mode | stat.S_IXUSR)
    monkeypatch.setattr(build, "HIPCC", str(exe))
    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    monkeypatch.setattr(build, "EXTRA", {"a.hip": ["-mllvm", "-some-switch=1"], "broken.hip": ["-mllvm", "-other"]})


def test_a_switch_that_is_not_known(compiler, capsys):
    assert os.path.exists(build._compile("a.hip"))
    assert "-some-switch=1" in capsys.readouterr().err
    assert os.path.exists(build._compile("plain.hip"))
    assert capsys.readouterr().err == ""


def test_other_errors_are_errors(compiler):
    with pytest.raises(RuntimeError, match="broken.hip"):
        build._compile("broken.hip")
