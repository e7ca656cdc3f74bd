"""The build and smoke script, run as one: everything that it calls is defined when it runs."""
import os
import runpy
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ENTRY = os.path.join(ROOT, "__graft_entry__.py")


def test_nothing_is_defined_behind_the_script_part():
    import ast
    with open(ENTRY) as f:
        body = ast.parse(f.read()).body
    script = [i for i, x in enumerate(body) if isinstance(x, ast.If) and "__main__" in ast.dump(x.test)]
    assert script == [len(body) - 1]


def test_the_build_part_runs(monkeypatch):
    monkeypatch.setattr(sys, "argv", [ENTRY])
    monkeypatch.setattr(sys, "path", list(sys.path))
    runpy.run_path(ENTRY, run_name="__main__")


@pytest.mark.gpu
def test_the_smoke_part_runs():
    r = subprocess.run([sys.executable, ENTRY, "smoke"], cwd=ROOT, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and "smoke ok" in r.stdout, r.stdout + r.stderr
