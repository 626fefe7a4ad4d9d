"""What the build makes, and from what, with compilers that only record their calls."""
import os
import stat
import subprocess
import sys

import pytest

BUILD_PY = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                        "paged_gqa_decode_kv_gb300", "build.py")

COMPILER = """#!%s
import sys
a = sys.argv[1:]
with open(%r, "a") as f:
    f.write(" ".join(a) + "\\n")
if %r and any(%r in x for x in a):
    sys.exit(1)
open(a[a.index("-o") + 1], "w").close()
"""

RUN = """
import importlib.util, os, sys
if %(no_torch)r:
    sys.modules["torch"] = None  # (an import of it fails)
spec = importlib.util.spec_from_file_location("build", %(build)r)
b = importlib.util.module_from_spec(spec)
spec.loader.exec_module(b)
b.BUILD = %(out)r
b.LIB = os.path.join(b.BUILD, "libpgd.so")
for step in %(steps)r:
    if step:
        os.utime(os.path.join(b.BUILD, step), (0, 0))
    try:
        print(os.path.basename(b.build()))
    except RuntimeError as e:
        print("failed", str(e).split("\\n")[0][:60])
"""


def _run(tmp_path, no_torch=False, steps=("",), fails=""):
    """Runs build() once for each step, before which the named file is made old; returns what each
    printed and the names of the files compiled or linked in each, in order."""
    log = tmp_path / "calls"
    for name in ("nvcc", "cxx"):
        c = tmp_path / name
        c.write_text(COMPILER % (sys.executable, str(log), fails, fails))
        c.chmod(c.stat().st_mode | stat.S_IXUSR)
    env = dict(os.environ, NVCC=str(tmp_path / "nvcc"), CXX=str(tmp_path / "cxx"))
    script = RUN % dict(no_torch=no_torch, build=BUILD_PY, out=str(tmp_path / "out"),
                        steps=list(steps))
    r = subprocess.run([sys.executable, "-c", script], env=env, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    outs = [x.split()[x.split().index("-o") + 1] for x in log.read_text().splitlines()]
    return r.stdout.split("\n")[:-1], [os.path.basename(x).split(".tmp")[0] for x in outs]


def test_the_library_is_built_without_torch(tmp_path):
    said, made = _run(tmp_path, no_torch=True, steps=("", ""))
    assert said == ["libpgd.so"] * 2
    assert made[-1] == "libpgd.so" and made.count("libpgd.so") == 1  # (the second call: built)
    assert "api.cu.o" in made and not any("tensors" in x for x in made)


def test_the_extension_is_built_with_torch(tmp_path):
    pytest.importorskip("torch")
    said, made = _run(tmp_path, steps=("", "", "libpgd.so"))
    assert said == ["libpgd.so"] * 3
    assert made.count("libpgd.so") == 2 and made.count("tensors.cpp.o") == 1
    assert sum(x.startswith("_pgd_tensors_torch_") for x in made) == 1


def test_the_library_stands_where_the_extension_fails(tmp_path):
    pytest.importorskip("torch")
    said, made = _run(tmp_path, fails="tensors.cpp")
    assert said[0].startswith("failed compile failed") and "libpgd.so" in made
    assert os.path.exists(tmp_path / "out" / "libpgd.so")
