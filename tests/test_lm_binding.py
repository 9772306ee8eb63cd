"""pp_bind, the C half of the lm module: who needs it, and under which
interpreter a built one counts."""
import os
import shutil
import subprocess
import sys
import sysconfig

import pytest

from dfa_parsing_delimiter_gb300 import build as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_the_parser_does_not_need_it(tmp_path):
    """Without the file the library loads, and the lm calls say what is missing."""
    package = os.path.join(ROOT, "dfa_parsing_delimiter_gb300")
    shutil.copytree(package, tmp_path / "dfa_parsing_delimiter_gb300",
                    ignore=shutil.ignore_patterns("pp_bind*", "_build", "csrc", "__pycache__"))
    code = """
import torch
import dfa_parsing_delimiter_gb300 as pp
assert pp.__file__.startswith(%r)
assert pp.desc_csv().n_states == 5 and pp.tile_bytes() > 0
try:
    pp.embed(torch.zeros(3, dtype=torch.int64), torch.zeros(4, 8))
except RuntimeError as e:
    assert "pp_bind" in str(e) and "build" in str(e), e
else:
    raise AssertionError("no error")
""" % str(tmp_path)
    r = subprocess.run([sys.executable, "-c", code], cwd=tmp_path, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_a_build_without_pythons_headers_has_the_library(monkeypatch, tmp_path, capsys):
    monkeypatch.setattr(B, "BIND", str(tmp_path / "pp_bind.so"))
    monkeypatch.setattr(sysconfig, "get_path", lambda *a, **k: str(tmp_path))
    monkeypatch.setattr(sysconfig, "get_paths", lambda *a, **k: {"include": str(tmp_path)})
    assert B.build() == B.LIB
    assert os.path.exists(B.LIB) and not os.path.exists(B.BIND)
    assert "Python.h" in capsys.readouterr().err


def test_its_name_carries_the_interpreter():
    assert os.path.basename(B.BIND) == "pp_bind" + sysconfig.get_config_var("EXT_SUFFIX")
    if os.path.exists(os.path.join(sysconfig.get_path("include"), "Python.h")):
        B.build()
        assert os.path.exists(B.BIND)
