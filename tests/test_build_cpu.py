"""How the libraries are built and loaded, without a GPU: compilers and torch
are stood in for where a case needs them to be missing or to fail."""
import importlib.util
import os
import shutil
import stat
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PACKAGE = os.path.join(ROOT, "long_context_genomics_b200")


def _script(path, text):
    path.write_text("#!/bin/sh\n" + text)
    path.chmod(path.stat().st_mode | stat.S_IXUSR)
    return str(path)


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """build.py in a tree of its own, with compilers that only leave a file."""
    pkg = tmp_path / "pkg"
    (pkg / "csrc").mkdir(parents=True)
    (tmp_path / "include").mkdir()
    (tmp_path / "include" / "ag.h").write_text("")
    shutil.copy(os.path.join(PACKAGE, "build.py"), pkg / "build.py")
    out = 'while [ $# -gt 0 ]; do [ "$1" = -o ] && echo built > "$2"; shift; done\n'
    monkeypatch.setenv("NVCC", _script(tmp_path / "nvcc", out))
    monkeypatch.setenv("CXX", _script(tmp_path / "cxx", out))
    spec = importlib.util.spec_from_file_location("build_of_a_test", pkg / "build.py")
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    for name in mod.SOURCES + mod.HEADERS + ["layers_binding.cpp"]:
        (pkg / "csrc" / name).write_text("")
    return mod


def test_builds_both(tree):
    assert tree.needs_build()
    assert tree.build() == tree.LIB
    assert os.path.exists(tree.LIB) and os.path.exists(tree.LAYERS)
    assert not tree.needs_build()


def test_builds_the_library_without_torch(tree, monkeypatch):
    """The C ABI needs nvcc alone."""
    real = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec",
                        lambda name, *a: None if name == "torch" else real(name, *a))
    assert tree.build() == tree.LIB
    assert os.path.exists(tree.LIB) and not os.path.exists(tree.LAYERS)
    assert not tree.needs_build()


def test_builds_the_library_where_the_binding_fails(tree, tmp_path):
    tree.CXX = _script(tmp_path / "bad", "echo no compiler here >&2; exit 3\n")
    with pytest.raises(RuntimeError, match="_layers build failed(.|\n)*no compiler here"):
        tree.build()
    assert os.path.exists(tree.LIB) and tree.needs_build()
    tree.CXX = str(tmp_path / "missing")
    with pytest.raises(OSError):
        tree.build()


def test_reports_a_library_that_does_not_build(tree, tmp_path):
    tree.NVCC = _script(tmp_path / "bad", "echo no kernel today; exit 1\n")
    with pytest.raises(RuntimeError, match="libag build failed(.|\n)*no kernel today"):
        tree.build()


def _import(tmp_path, name, code, layers=None, before=""):
    """Runs `code` with a copy of the package that has the library and, unless
    it is None, `layers` for the compiled binding."""
    pkg = tmp_path / name
    pkg.mkdir()
    shutil.copy(os.path.join(PACKAGE, "__init__.py"), pkg)
    os.symlink(os.path.join(PACKAGE, "libag.so"), pkg / "libag.so")
    if layers is not None:
        layers(pkg / "_layers.so")
    return subprocess.run([sys.executable, "-c", f"{before}\nimport {name} as ag\n{code}"],
                          cwd=tmp_path, capture_output=True, text=True, timeout=300)


ATTENTION = """
import torch
assert ag.ag_version() > 0 and ag.ag_attn_bwd_launch_count() > 0
for call in (lambda: ag.ag_linear_fwd(torch.zeros(1, 8), torch.zeros(8, 8)),
             lambda: ag.ag_grad_clip([torch.zeros(3)], 1.0),
             lambda: ag.ag_qk_norm_rope_fwd(torch.zeros(1, 2, 3, 4), None)):
    try:
        call()
    except ImportError as e:
        print(e)
    else:
        raise SystemExit("no ImportError")
"""


def test_attention_needs_no_compiled_binding(tmp_path):
    res = _import(tmp_path, "ag_without", ATTENTION)
    assert res.returncode == 0, res.stdout + res.stderr
    assert res.stdout.count("_layers.so is missing: build it with") == 3


def test_a_binding_that_does_not_load_is_named(tmp_path):
    res = _import(tmp_path, "ag_broken", ATTENTION, lambda p: p.write_text("not a library"))
    assert res.returncode == 0, res.stdout + res.stderr
    assert res.stdout.count("_layers.so does not load") == 3 and "build.py" in res.stdout


def test_another_torch_builds_the_binding_anew(tree, tmp_path, monkeypatch):
    tree.build()
    assert not tree.needs_build()
    now = tree.built_for(tree.torch_dir())
    other = tmp_path / "torch"
    other.mkdir()
    (other / "version.py").write_text("__version__ = '2.12.1+cu130'\n")
    monkeypatch.setattr(tree, "torch_dir", lambda: str(other))
    assert tree.built_for(str(other)).startswith("torch 2.12.1+cu130 ") and now.startswith("torch ")
    assert tree.needs_build()
    monkeypatch.undo()
    os.remove(tree.LAYERS_BUILT_FOR)
    assert tree.needs_build()


def test_the_binding_is_compiled_for_the_abi_of_torch(tree):
    torch = pytest.importorskip("torch")
    assert (f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}"
            in tree._layers_command(tree.torch_dir()))


def test_a_binding_for_another_torch_is_refused(tmp_path):
    """(Where its symbols happen to be there: the version tells.)"""
    res = _import(tmp_path, "ag_other", ATTENTION, before="import torch\ntorch.__version__ = '2.10.0'",
                  layers=lambda p: os.symlink(os.path.join(PACKAGE, "_layers.so"), p))
    assert res.returncode == 0, res.stdout + res.stderr
    assert res.stdout.count("this is torch 2.10.0") == 3 and "was built for torch" in res.stdout
