"""When the library and the short way into the layer operators are built, loaded
and bound: on copies of the package in processes of their own (no GPU)."""
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NAME = "linear_attention_sequence_falcon_b200"


@pytest.fixture
def copy(tmp_path):
    """A copy of the built tree with its times; runs Python code in it."""
    from linear_attention_sequence_falcon_b200 import build
    build.build()
    for d in (NAME, "include", "_build"):
        shutil.copytree(os.path.join(ROOT, d), tmp_path / d, ignore=shutil.ignore_patterns("__pycache__", "*.o"))

    def run(code, **env):
        env = {**os.environ, "PYTHONDONTWRITEBYTECODE": "1", **env}
        return subprocess.run([sys.executable, "-c", HEAD + code], cwd=tmp_path, env=env, capture_output=True, text=True,
                              timeout=600)
    run.path = tmp_path
    return run


def quick():
    from linear_attention_sequence_falcon_b200 import build
    return os.path.basename(build.QUICK)


HEAD = """
import os, sys
sys.path.insert(0, os.getcwd())
import linear_attention_sequence_falcon_b200 as F
from linear_attention_sequence_falcon_b200 import build, layer
mapped = lambda: {p for p in (build.LIB, build.QUICK) for l in open("/proc/self/maps") if l.rstrip().endswith(p)}
"""


def test_import_maps_no_library(copy):
    """A build between import and load() is what load() takes."""
    r = copy("""
assert not mapped(), mapped()
build.build()
assert not mapped(), mapped()
F.load()
assert mapped() == {build.LIB, build.QUICK} and layer._quick is not None
build.build()  # nothing to do
""")
    assert r.returncode == 0, r.stderr[-2000:]


def test_short_way_built_after_the_import_is_bound(copy):
    """A clean tree's first process takes the short way too."""
    os.rename(copy.path / NAME / quick(), copy.path / "away")
    r = copy("""
assert layer._quick is None
os.rename("away", build.QUICK)
F.load()
assert layer._quick is not None
""")
    assert r.returncode == 0, r.stderr[-2000:]


def test_build_refuses_to_replace_a_loaded_library(copy):
    for target, source in (("libfalcon.so", "common.cuh"), (quick(), "quick_layer.cpp")):
        before = os.stat(copy.path / NAME / target)  # (an import changes the access time)
        r = copy("""
F.load()
new = os.path.getmtime(build.LIB) + 100
os.utime(os.path.join(build.CSRC, "%s"), (new, new))
build.build()
""" % source, NVCC="/bin/false")
        assert r.returncode != 0 and "RuntimeError: %s is out of date, and loaded" % target in r.stderr, r.stderr[-2000:]
        after = os.stat(copy.path / NAME / target)
        assert (after.st_ino, after.st_mtime_ns) == (before.st_ino, before.st_mtime_ns)
        os.utime(copy.path / NAME / "csrc" / source, (before.st_mtime - 100,) * 2)


@pytest.mark.parametrize("objects", [True, False])
def test_short_way_for_another_torch_is_neither_bound_nor_kept(copy, objects):
    """A module made for another torch is not imported, and the one for this torch
    is built beside it, also in a copy of the tree without _build/."""
    if not objects:
        shutil.rmtree(copy.path / "_build")
    made = copy.path / NAME / quick()
    code = """
F.load()
assert (layer._quick is not None) == %s
def refuse(*args, **kw):
    raise LookupError("built again")
build.subprocess.run = refuse
build.build_quick()
"""
    r = copy(code % True)
    assert r.returncode == 0, r.stderr[-2000:]
    import torch
    assert torch.__version__ in quick() and sys.implementation.cache_tag in quick()
    made.rename(made.with_name(quick().replace(torch.__version__, "1.0")))
    r = copy(code % False)
    assert "LookupError: built again" in r.stderr, r.stderr[-2000:]


def test_short_way_that_does_not_load_leaves_the_long_one(copy):
    (copy.path / NAME / quick()).write_bytes(b"not a library")
    r = copy("F.load(); assert layer._quick is None")
    assert r.returncode == 0, r.stderr[-2000:]
