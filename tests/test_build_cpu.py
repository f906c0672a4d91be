"""What the build and the package need: nvcc alone for the library, allocator, decode and prefill;
torch and its headers only for the helper of the drafted step's binding."""
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NAME = "paged_kv_cache_465_b200"


@pytest.fixture
def tree(tmp_path):
    """A copy of the sources, with compilers that only make their output file and say so."""
    shutil.copytree(os.path.join(ROOT, NAME), tmp_path / NAME,
                    ignore=shutil.ignore_patterns("*.so", "__pycache__"))
    shutil.copytree(os.path.join(ROOT, "include"), tmp_path / "include")
    tool = tmp_path / "tool"
    tool.write_text('#!/bin/sh\nwhile [ $# -gt 0 ]; do\n  [ "$1" = -o ] && echo "$2" >> "$TOOL_LOG" '
                    '&& : > "$2"\n  shift\ndone\n')
    tool.chmod(0o755)
    return tmp_path


def run(tree, code, **env):
    log = tree / "log"
    log.write_text("")
    e = dict(os.environ, NVCC=str(tree / "tool"), CXX=str(tree / "tool"), TOOL_LOG=str(log),
             PYTHONPATH=str(tree), **env)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, env=e, cwd=tree)
    made = [os.path.basename(x) for x in log.read_text().split()]
    return r, made


LOAD = f"""
import importlib.util
spec = importlib.util.spec_from_file_location("b", "{NAME}/build.py")
b = importlib.util.module_from_spec(spec)
spec.loader.exec_module(b)
"""


def fake_torch(tree, version, headers=True):
    d = tree / "torch"
    (d / "include" / "torch" / "csrc").mkdir(parents=True, exist_ok=True)
    if headers:
        (d / "include" / "torch" / "csrc" / "Dtype.h").write_text("")
    (d / "__init__.py").write_text(f"__version__ = '{version}'\nclass _C: _GLIBCXX_USE_CXX11_ABI = True\n")


def test_the_library_builds_without_torch(tree):
    r, made = run(tree, "import sys; sys.modules['torch'] = None\n" + LOAD + "b.build()")
    assert r.returncode == 0, r.stderr
    assert "libpagedattn.so.tmp" in made and not any("_tensors" in m for m in made)
    assert (tree / NAME / "libpagedattn.so").exists()
    r, made = run(tree, "import sys; sys.modules['torch'] = None\n" + LOAD + "b.build()")
    assert r.returncode == 0 and not made     # nothing is stale


def test_the_library_builds_without_torch_headers(tree):
    fake_torch(tree, "9.1.0", headers=False)
    r, made = run(tree, LOAD + "b.build()")
    assert r.returncode == 0, r.stderr
    assert (tree / NAME / "libpagedattn.so").exists() and not any("_tensors" in m for m in made)


def test_the_helper_is_built_anew_for_another_torch(tree):
    fake_torch(tree, "9.1.0")
    r, made = run(tree, LOAD + "b.build()")
    assert r.returncode == 0 and any("torch9.1.0" in m for m in made), (r.stderr, made)
    r, made = run(tree, LOAD + "b.build()")
    assert r.returncode == 0 and not made
    fake_torch(tree, "9.2.0")
    shutil.rmtree(tree / "torch" / "__pycache__", ignore_errors=True)
    r, made = run(tree, LOAD + "b.build()")
    assert r.returncode == 0 and len(made) == 1 and "torch9.2.0" in made[0], (r.stderr, made)


def test_the_package_needs_the_helper_for_drafted_calls_only(tree):
    """The allocator works without it; a drafted call says what is missing. A helper for another
    torch does not count."""
    from tests.test_lib_cpu import ROOT as r0
    os.symlink(os.path.join(r0, NAME, "libpagedattn.so"), tree / NAME / "libpagedattn.so")
    (tree / NAME / "_tensors.so").write_text("not loaded")
    (tree / NAME / "_tensors-torch0.1-abi1.so").write_text("not loaded")
    r, _ = run(tree, f"""
import {NAME} as pa, torch
a = pa.BlockAllocator(8, 16)
print(len(a.free_queue()))
assert pa.paged_attn_decode and pa.paged_attn_prefill
i = torch.zeros(2, dtype=torch.int32)
class Cuda:     # of which the call asks the device first
    def get_device(self): return 0
    shape = (2,)
c = Cuda()
try:
    pa.release_blocks(c, c, c, c, c, block_size=16, blocks_held_out=c, queue_state_out=c)
except ImportError as e:
    print("missing" in str(e) and "build.py" in str(e))
""")
    assert r.returncode == 0, r.stderr
    assert r.stdout.split() == ["8", "True"]
