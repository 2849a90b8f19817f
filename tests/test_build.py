"""Build of the C library beside the torch binding, with stand-ins for the
compilers (no GPU, nothing is compiled)."""
import os
import stat
import warnings

import pytest

from exact_attention_57_gb300 import build

# Writes what -o names, after half a second, so that a build that does not wait
# for its compilers leaves files unwritten.
COMPILER = """#!/bin/sh
while [ $# -gt 0 ]; do [ "$1" = -o ] && out="$2"; shift; done
sleep 0.5
echo done > "$out"
"""


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A package of two kernel sources and a binding, built in tmp_path."""
    csrc, tools = tmp_path / "csrc", tmp_path / "tools"
    (csrc / "bind").mkdir(parents=True)
    tools.mkdir()
    for name in ("a.cu", "b.cu", "bind/x.cpp"):
        (csrc / name).write_text("// nothing\n")
    paths = dict(CSRC=csrc, BUILD=tmp_path / "_build", LIB=tmp_path / "libx.so",
                 BIND=csrc / "bind" / "x.cpp", LIB_BIND=tmp_path / "_x.so",
                 INCLUDE=tmp_path / "include")
    (tmp_path / "include").mkdir()
    (tmp_path / "include" / "fa.h").write_text("")
    for k, v in paths.items():
        monkeypatch.setattr(build, k, str(v))

    def tool(name, text):
        p = tools / name
        p.write_text(text)
        p.chmod(p.stat().st_mode | stat.S_IXUSR)

    tool("nvcc", COMPILER)
    tool("g++", COMPILER)
    monkeypatch.setattr(build, "nvcc", lambda: str(tools / "nvcc"))
    monkeypatch.setenv("PATH", f"{tools}:{os.environ['PATH']}")
    return tmp_path, tool


def built(path):
    return sorted(n for n in ("libx.so", "_x.so") if os.path.exists(path / n))


def test_library_and_binding(tree):
    path, _ = tree
    build.build_library()
    assert built(path) == ["_x.so", "libx.so"]


def test_a_binding_that_does_not_compile_leaves_the_library(tree):
    path, tool = tree
    tool("g++", "#!/bin/sh\necho it does not compile\nexit 1\n")
    with pytest.raises(RuntimeError, match="it does not compile"):
        build.build_library()
    assert built(path) == ["libx.so"]
    assert sorted(os.listdir(path / "_build")) == ["a.o", "a.o.log", "b.o", "b.o.log", "ptxas.log"]
    tool("g++", COMPILER)  # and the next build makes it
    build.build_library()
    assert built(path) == ["_x.so", "libx.so"]


def test_kernels_that_do_not_compile_are_named(tree):
    path, tool = tree
    tool("nvcc", "#!/bin/sh\necho no kernel\nexit 1\n")
    with pytest.raises(RuntimeError, match="no kernel"):
        build.build_library()
    assert not os.path.exists(path / "libx.so")
    assert not [n for n in os.listdir(path) if ".tmp" in n]


def test_without_the_binding_s_compiler_or_a_torch_with_cuda(tree, monkeypatch):
    import torch
    path, _ = tree
    popen = build.subprocess.Popen

    def none(cmd, *a, **k):
        if cmd[0] == "g++":
            raise FileNotFoundError("g++")
        return popen(cmd, *a, **k)

    monkeypatch.setattr(build.subprocess, "Popen", none)
    with pytest.warns(UserWarning, match="no g\\+\\+"):
        build.build_library()
    assert built(path) == ["libx.so"]
    monkeypatch.setattr(torch.version, "cuda", None)
    with warnings.catch_warnings():
        warnings.simplefilter("error", UserWarning)
        build.build_library(force=True)
    assert built(path) == ["libx.so"]
