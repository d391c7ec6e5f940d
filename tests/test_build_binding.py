"""The marshalling of the paged calls holds for one Python and one torch: the
package works without it, and the build makes it anew for another."""

from __future__ import annotations

import importlib.util
import os
import subprocess
import sys
from pathlib import Path

import pytest
import torch

ROOT = Path(__file__).resolve().parents[1]
PACKAGE = ROOT / "causal_self_attention_flash_b200"


@pytest.fixture
def build():
    spec = importlib.util.spec_from_file_location("cattn_build", PACKAGE / "build.py")
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def package_without(tmp_path, name, contents=None):
    """A copy of the package with every file but the marshalling (or with
    `contents` in its place)."""
    to = tmp_path / PACKAGE.name
    to.mkdir()
    for f in PACKAGE.iterdir():
        if f.suffix in (".py", ".so") and f.name != name:
            os.symlink(f, to / f.name)
    if contents is not None:
        (to / name).write_bytes(contents)


USE = """
import warnings
with warnings.catch_warnings(record=True) as seen:
    warnings.simplefilter("always")
    import causal_self_attention_flash_b200 as cattn
print(len([w for w in seen if "_torch_calls" in str(w.message)]))
import torch
print(cattn.cattn_version() > 0)
t = torch.zeros(2, 4, 1, 64, dtype=torch.bfloat16)
try:
    cattn.attn_decode_paged(t, t, t, t, t, 1.0, t, t, t)
except ValueError as e:
    print(e)
"""


@pytest.mark.parametrize("contents", [None, b"no library"])
def test_the_package_works_without_the_marshalling(build, tmp_path, contents):
    package_without(tmp_path, os.path.basename(build.binding_path()), contents)
    r = subprocess.run([sys.executable, "-c", USE], capture_output=True, text=True, cwd=tmp_path,
                       env=dict(os.environ, PYTHONPATH=str(tmp_path)))
    assert r.returncode == 0, r.stderr[-2000:]
    assert r.stdout.split("\n")[:3] == ["1", "True", "expected CUDA tensors"]


def test_the_built_marshalling_is_loaded(build):
    import causal_self_attention_flash_b200 as cattn
    assert cattn.TORCH_CALLS.__spec__.origin == build.binding_path()


@pytest.mark.parametrize("what", ["torch", "python"])
def test_another_torch_or_python_builds_anew(build, monkeypatch, what):
    assert os.path.exists(build.binding_path())
    ran = []
    monkeypatch.setattr(build.os.path, "getmtime", lambda f: 0.0)     # all of one age
    monkeypatch.setattr(build.subprocess, "run", lambda cmd, check: ran.append(cmd))
    monkeypatch.setattr(build.os, "replace", lambda a, b: ran.append((a, b)))
    old = build.build_binding()
    assert not ran, "the one that is there is up to date"
    if what == "torch":
        monkeypatch.setattr(torch, "__version__", "99.1+cu999")
    else:
        monkeypatch.setattr(build.sys.implementation, "cache_tag", "cpython-999")
    new = build.build_binding()
    assert new != old and ("99.1+cu999" if what == "torch" else "cpython-999") in new
    cmd, move = ran
    assert cmd[-1] == new + ".tmp" and move == (new + ".tmp", new)
