"""The compiled binding is optional: the package loads, and calls through ctypes, wherever the binding cannot be made or
used.  Each case loads a copy of the package in a process of its own."""
import os
import pathlib
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = "gated_deltanet_decode_gb300"

LOAD = """
import os, shutil, sys
hidden = sys.argv[1].split(",")
which, exists = shutil.which, os.path.exists
shutil.which = lambda name, *a, **k: None if name in hidden else which(name, *a, **k)
os.path.exists = lambda p: not ("nvcc" in hidden and str(p).endswith("bin/nvcc")) and exists(p)
from gated_deltanet_decode_gb300 import _lib
assert _lib.load().paged_attention
print("binding" if _lib.fast() else "ctypes")
"""


@pytest.fixture
def package(tmp_path):
    """A copy of the package with its library, up to date, and no binding."""
    from gated_deltanet_decode_gb300 import build
    build.build()
    shutil.copytree(os.path.join(ROOT, PKG), tmp_path / PKG,
                    ignore=shutil.ignore_patterns("_fast_binding*", "__pycache__", "_build"))
    shutil.copytree(os.path.join(ROOT, "include"), tmp_path / "include")
    return tmp_path


def give_binding(package):
    """The binding that was built here, put into the copy."""
    from gated_deltanet_decode_gb300 import build
    name = os.path.basename(build.binding_path())
    if not os.path.exists(build.binding_path()):
        pytest.skip("no compiler for the binding")
    return pathlib.Path(shutil.copy2(build.binding_path(), package / PKG / name))


def load(package, without="", path=None):
    """How the copy makes its calls, where the programs of `without` are missing."""
    env = dict(os.environ, PYTHONPATH=str(package))
    if path:
        env["PATH"] = f"{path}{os.pathsep}{env['PATH']}"
    r = subprocess.run([sys.executable, "-c", LOAD, without], cwd=package, env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    return r.stdout.split()[-1]


def test_without_a_toolkit_the_built_library_loads(package):
    assert load(package, without="nvcc") == "ctypes"
    assert load(package, without="g++") == "ctypes"


def test_a_binding_that_cannot_be_loaded_is_left_alone(package):
    binding = give_binding(package)
    assert load(package) == "binding"
    binding.write_bytes(b"not a shared library")
    assert load(package) == "ctypes"


def test_a_binding_belongs_to_one_interpreter_and_one_pytorch(monkeypatch):
    import sysconfig

    import torch

    from gated_deltanet_decode_gb300 import build
    here = build.binding_path()
    monkeypatch.setattr(torch, "__version__", torch.__version__.split("+")[0] + "+cu999")
    other = build.binding_path()
    assert other != here
    monkeypatch.setattr(sysconfig, "get_config_var", lambda name: ".cpython-399-other.so" if name == "EXT_SUFFIX" else None)
    assert build.binding_path() not in (here, other)


def test_a_binding_older_than_its_sources_is_not_used(package):
    binding = give_binding(package)
    assert load(package, without="g++") == "binding"
    os.utime(binding, (1, 1))
    assert load(package, without="g++") == "ctypes"


def test_a_binding_that_does_not_compile_is_tried_once(package):
    """The compiler is asked again only when a source has changed since."""
    tools, log = package / "tools", package / "asked"
    tools.mkdir()
    (tools / "g++").write_text(f"#!/bin/sh\necho asked >> {log}\nexit 1\n")
    (tools / "g++").chmod(0o755)
    assert load(package, path=tools) == "ctypes"
    assert load(package, path=tools) == "ctypes"
    assert log.read_text().count("asked") == 1
    source = package / PKG / "csrc" / "fast_binding.cpp"
    later = os.path.getmtime(log) + 10
    os.utime(source, (later, later))
    assert load(package, path=tools) == "ctypes"
    assert log.read_text().count("asked") == 2
