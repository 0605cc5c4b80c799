"""What a build compiles and links again, with stub compilers in place of nvcc and g++."""
import os
import stat
import sys
import time

import pytest

STUB = """#!{python} -SE
import os, sys
here, args = os.path.dirname(os.path.abspath(__file__)), sys.argv[1:]
out = args[args.index("-o") + 1]
inputs = [a for i, a in enumerate(args) if a.endswith((".cu", ".cpp", ".o")) and args[i - 1] != "-o"]
open(os.path.join(here, "log"), "a").write(" ".join(os.path.basename(i) for i in inputs) + "\\n")
failing = open(os.path.join(here, "failing")).read().split()
what = "link" if "-shared" in args and not any(a.startswith("-l:") for a in args) else "extension link" if "-shared" in args else ""
if any(os.path.basename(i) in failing for i in inputs if not i.endswith(".o")) or what.replace(" ", "_") in failing:
    sys.exit(1)
if "-shared" in args:
    text = "".join(open(i).read() for i in inputs)
else:
    text = os.path.basename(inputs[0]) + open(os.path.join(here, "version")).read() + "\\n"
open(out, "w").write(text)
"""


class Tree:
    def __init__(self, tmp, monkeypatch):
        from attention_backward_gb300 import build

        self.build, self.bin = build, tmp / "bin"
        self.bin.mkdir()
        for name in ("nvcc", "g++"):
            path = self.bin / name
            path.write_text(STUB.format(python=sys.executable))
            path.chmod(path.stat().st_mode | stat.S_IXUSR)
        monkeypatch.setenv("PATH", f"{self.bin}{os.pathsep}{os.environ['PATH']}")
        out = tmp / "_build"
        monkeypatch.setattr(build, "BUILD", str(out))
        monkeypatch.setattr(build, "LIB", str(out / "lib.so"))
        monkeypatch.setattr(build, "TORCH_LIB", str(out / "torch.so"))
        csrc, include = tmp / "csrc", tmp / "include"
        csrc.mkdir(), include.mkdir()
        self.header = include / "a.h"
        self.sources = [csrc / s for s in ("one.cu", "two.cu", build.TORCH_SOURCE)]
        monkeypatch.setattr(build, "SOURCES", ["one.cu", "two.cu"])
        monkeypatch.setattr(build, "CSRC", str(csrc))
        monkeypatch.setattr(build, "ROOT", str(tmp))
        self.at = time.time() - 1000
        for f in (*self.sources, self.header):
            self.edit(f)
        self.set()

    def edit(self, path):  # (a second later each time, well before the objects)
        self.at += 1
        path.write_text("")
        os.utime(path, (self.at, self.at))

    def touch_all(self):
        """An edit of a header that everything includes: newer than all that was built."""
        for f in os.listdir(self.build.BUILD):
            old = time.time() - 2000
            os.utime(os.path.join(self.build.BUILD, f), (old, old))

    def set(self, version="1", failing=""):
        (self.bin / "version").write_text(version)
        (self.bin / "failing").write_text(failing)
        (self.bin / "log").write_text("")

    def run(self):
        return self.build.build()

    def log(self):
        return sorted((self.bin / "log").read_text().split("\n")[:-1])

    def libraries(self):
        return [open(p).read() if os.path.exists(p) else None for p in (self.build.LIB, self.build.TORCH_LIB)]


@pytest.fixture
def tree(tmp_path, monkeypatch):
    return Tree(tmp_path, monkeypatch)


def whole(v):
    return [f"one.cu{v}\ntwo.cu{v}\n", f"torch_latent.cpp{v}\n"]


def test_nothing_is_done_twice(tree):
    tree.run()
    assert tree.libraries() == whole("1") and len(tree.log()) == 5
    tree.set("2")
    tree.run()
    assert tree.log() == [] and tree.libraries() == whole("1")
    tree.sources[0].write_text("")  # one source, now: its object and the library
    os.utime(tree.sources[0], (time.time() + 5, time.time() + 5))
    tree.run()
    assert tree.log() == ["one.cu", "one.o two.o"]
    assert tree.libraries() == ["one.cu2\ntwo.cu1\n", whole("1")[1]]


@pytest.mark.parametrize("failing", ["torch_latent.cpp", "one.cu", "two.cu", "link", "extension_link", "one.cu torch_latent.cpp"])
def test_a_build_that_failed_is_taken_up(tree, failing):
    """All is stale and one step fails; once that is mended, both libraries are new."""
    tree.run()
    tree.touch_all()
    tree.set("2", failing)
    with pytest.raises(RuntimeError):
        tree.run()
    tree.set("2")
    tree.run()
    assert tree.libraries() == whole("2")
    tree.set("3")
    tree.run()
    assert tree.log() == [] and tree.libraries() == whole("2")


def test_a_build_that_was_cut_off_is_taken_up(tree, monkeypatch):
    """Compiled and not linked: the objects are newer than the libraries."""
    tree.run()
    tree.touch_all()
    tree.set("2", "link extension_link")
    with pytest.raises(RuntimeError):
        tree.run()
    tree.set("3")  # (no source has changed)
    tree.run()
    assert tree.libraries() == whole("2") and tree.log() == ["one.o two.o", "torch_latent.o"]


@pytest.mark.parametrize("failing", ["torch_latent.cpp", "extension_link", "flags"])
def test_the_library_does_not_wait_for_the_extension(tree, monkeypatch, failing):
    """Without Python's headers, or without torch, the library is built all the same; the
    build says what failed."""
    tree.set("1", failing)
    if failing == "flags":
        def none(cc):
            raise ImportError("No module named 'torch'")

        monkeypatch.setattr(tree.build, "_torch_flags", none)
    with pytest.raises((RuntimeError, ImportError)):
        tree.run()
    assert tree.libraries() == [whole("1")[0], None]


def test_the_extension_belongs_to_one_interpreter_and_torch(tree, monkeypatch):
    """Another torch, interpreter or set of flags compiles and links it anew; the library
    stays."""
    import torch

    tree.run()
    plain = tree.build._torch_flags
    for i, (where, name, value) in enumerate([(torch, "__version__", "9.9"), (sys, "version", "4.0 (other)"),
                                              (tree.build, "_torch_flags", lambda cc: (plain(cc)[0] + ["-DX"], plain(cc)[1])),
                                              (tree.build, "_torch_flags", lambda cc: (plain(cc)[0], plain(cc)[1] + ["-lx"]))]):
        with monkeypatch.context() as m:
            m.setattr(where, name, value)
            tree.set(f"{i + 2}")
            tree.run()
            assert tree.libraries() == [whole("1")[0], whole(f"{i + 2}")[1]]
            assert tree.log() == ["torch_latent.cpp", "torch_latent.o"]
            tree.set("x")
            tree.run()
            assert tree.log() == []
    tree.set("7", "torch_latent.cpp")  # back again, and the compiler fails: the old one is not kept for good
    with pytest.raises(RuntimeError):
        tree.run()
    tree.set("8")
    tree.run()
    assert tree.libraries()[1] == whole("8")[1]
