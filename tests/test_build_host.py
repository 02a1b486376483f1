"""What the build needs and when it is done again: the C library without
PyTorch, the Python binding with the PyTorch that is installed."""
import os
import shutil
import subprocess
import sys

from paged_kv_cache_xs_gb300 import build as xsbuild

ROOT = xsbuild.ROOT


def copy_of(tmp_path):
    """The package's build module and sources, with what is built here."""
    shutil.copytree(xsbuild.PKG, tmp_path / "paged_kv_cache_xs_gb300",
                    ignore=shutil.ignore_patterns("__pycache__", "_build_debug"))
    shutil.copytree(xsbuild.INCLUDE, tmp_path / "include")
    return tmp_path


def run(path, code, *flags):
    r = subprocess.run([sys.executable, *flags, "-c", code], cwd=path, capture_output=True, text=True,
                       env={**os.environ, "PYTHONPATH": str(path)})
    assert r.returncode == 0, r.stderr
    return r.stdout.strip()


def test_library_builds_without_pytorch(tmp_path):
    # An interpreter without site packages: no torch.  The compiler is a stand-in
    # that writes its output file.
    root = copy_of(tmp_path)
    shutil.rmtree(root / "paged_kv_cache_xs_gb300" / "_build", ignore_errors=True)
    fake = tmp_path / "bin"
    fake.mkdir()
    (fake / "nvcc").write_text('#!/bin/sh\nwhile [ $# -gt 1 ]; do [ "$1" = -o ] && echo x > "$2"; shift; done\n')
    (fake / "nvcc").chmod(0o755)
    code = ("import os, importlib.util\n"
            "assert importlib.util.find_spec('torch') is None\n"
            f"os.environ['PATH'] = {str(fake)!r} + ':' + os.environ['PATH']\n"
            "from paged_kv_cache_xs_gb300 import build as b\n"
            "assert not b.up_to_date()\n"
            "print(os.path.exists(b.build()), b.up_to_date(), os.path.exists(b.BIND_PATH))")
    assert run(root, code, "-S") == "True True False"


def test_binding_is_built_again_for_another_pytorch(tmp_path):
    xsbuild.build()
    root = copy_of(tmp_path)
    built = root / "paged_kv_cache_xs_gb300" / "_build"
    (built / "xs_bind.so.against").write_text("another\n")
    code = ("from paged_kv_cache_xs_gb300 import build as b\n"
            "def bind():\n"
            "    open(b.BIND_PATH, 'w').write('new')\n"
            "    open(b.BIND_PATH + '.against', 'w').write(b._bind_against())\n"
            "b.build_bind = bind\n"
            "old = b.up_to_date(), b._newer(b.LIB_PATH, b._deps())\n"
            "b.nvcc = lambda: 1 / 0 if not old[1] else 'nvcc'\n"
            "b.build()\n"
            "print(old, open(b.BIND_PATH).read(), b.up_to_date())")
    assert run(root, code) == "(False, True) new True"
