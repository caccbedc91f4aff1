"""The incremental build, with a compiler that records its calls in place of nvcc."""
import os
import subprocess
import sys
import time

import pytest

from banded_log_domain_b200 import build as b

# -c: the "object" is the text of the source and of what it includes; -shared: all objects
FAKE = r"""#!{python}
import os, sys, time
a = sys.argv[1:]
out = a[a.index("-o") + 1]
with open(os.environ["FAKE_LOG"], "a") as f:
    f.write(("link" if "-shared" in a else os.path.basename(a[a.index("-c") + 1])) + "\n")
if "-shared" in a:
    text = "".join(open(x).read() for x in a if x.endswith(".o"))
else:
    src = a[a.index("-c") + 1]
    text, files = "", [src]
    for line in open(src):
        if line.startswith("#include "):
            files.append(os.path.join(os.path.dirname(src), line.split()[1]))
            line = open(files[-1]).read()
        text += line
    open(a[a.index("-MF") + 1], "w").write(out + ": " + " ".join(files) + "\n")
    if os.environ.get("FAKE_FAIL", "-") in text:
        open(out, "w").write(text[:3])
        sys.exit(1)
    if os.environ.get("FAKE_HANG", "-") in text:
        open(out, "w").write(text[:3])
        time.sleep(600)
open(out, "w").write(text)
"""


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A tree of two sources and a header; run() builds it and returns the compiler's calls."""
    src = tmp_path / "csrc"
    src.mkdir()
    (src / "x.cuh").write_text("header\n")
    (src / "one.cu").write_text("#include x.cuh\none\n")
    (src / "two.cu").write_text("two\n")
    nvcc, log = tmp_path / "nvcc", tmp_path / "log"
    nvcc.write_text(FAKE.replace("{python}", sys.executable))
    nvcc.chmod(0o755)
    monkeypatch.setenv("FAKE_LOG", str(log))
    for name, value in dict(NVCC=nvcc, CSRC=src, OBJ=tmp_path / "build", LIB=tmp_path / "lib.so",
                            DEBUG_LIB=tmp_path / "debug.so").items():
        monkeypatch.setattr(b, name, str(value))
    past = time.time() - 100
    for f in src.iterdir():
        os.utime(f, (past, past))

    def run(**kw):
        log.write_text("")
        b.build(**kw)
        return sorted(log.read_text().split())

    run.path, run.src, run.monkeypatch = tmp_path, src, monkeypatch
    return run


ALL = ["link"] * 2 + ["one.cu"] * 2 + ["two.cu"] * 2


def text(run, lib="lib.so"):
    return (run.path / lib).read_text()


def test_only_what_changed_is_compiled(tree):
    assert tree() == ALL and text(tree) == text(tree, "debug.so") == "header\none\ntwo\n"
    assert tree() == []
    (tree.src / "x.cuh").write_text("HEADER\n")
    assert tree() == ["link"] * 2 + ["one.cu"] * 2 and text(tree) == "HEADER\none\ntwo\n"
    (tree.path / "lib.so").unlink()
    assert tree() == ["link"]
    assert tree(force=True) == ALL and tree() == []


def test_flags_and_sources_count(tree):
    tree()
    tree.monkeypatch.setattr(b, "FLAGS", b.FLAGS + ["-DX"])
    assert tree() == ALL and tree() == []
    (tree.src / "two.cu").unlink()
    assert tree() == ["link"] * 2 and text(tree) == "header\none\n"
    (tree.src / "three.cu").write_text("three\n")
    assert tree() == ["link"] * 2 + ["three.cu"] * 2 and text(tree) == "header\none\nthree\n"


def test_a_failed_compilation_leaves_nothing(tree):
    tree()
    (tree.src / "two.cu").write_text("broken\n")
    tree.monkeypatch.setenv("FAKE_FAIL", "broken")
    with pytest.raises(subprocess.CalledProcessError):
        tree()
    assert text(tree) == "header\none\ntwo\n"
    assert not [f for f in (tree.path / "build").rglob("*") if ".tmp" in f.name]
    tree.monkeypatch.delenv("FAKE_FAIL")
    assert tree() == ["link"] * 2 + ["two.cu"] * 2 and text(tree) == "header\none\nbroken\n"


def test_a_source_written_while_it_was_compiled_is_compiled_again(tree):
    tree()
    (tree.src / "two.cu").write_text("2\n")
    real = subprocess.Popen

    def popen(cmd, *a, **kw):  # the compiler has read the source; then it changes
        p = real(cmd, *a, **kw)
        p.wait()
        if "two.cu" in cmd[cmd.index("-c") + 1] if "-c" in cmd else False:
            (tree.src / "two.cu").write_text("zwei\n")
        return p

    with tree.monkeypatch.context() as m:
        m.setattr(b.subprocess, "Popen", popen)
        tree()
    tree()
    assert text(tree) == text(tree, "debug.so") == "header\none\nzwei\n"


def test_a_build_killed_part_way_is_not_taken_for_current(tree):
    tree()
    (tree.src / "two.cu").write_text("slow\n")
    code = "import sys; from banded_log_domain_b200 import build as b\n" + "".join(
        f"b.{n} = {getattr(b, n)!r}\n" for n in ("NVCC", "CSRC", "OBJ", "LIB", "DEBUG_LIB")) + "b.build()\n"
    p = subprocess.Popen([sys.executable, "-c", code], cwd=b.ROOT, start_new_session=True,
                         env=dict(os.environ, FAKE_HANG="slow"))
    try:
        for _ in range(300):  # until both compilers have written their half objects
            if len([f for f in (tree.path / "build").rglob("two.o*.tmp*") if ".d." not in f.name]) == 2:
                break
            time.sleep(0.1)
        assert text(tree) == "header\none\ntwo\n"
    finally:
        os.killpg(p.pid, 9)
        p.wait()
    assert tree() == ["link"] * 2 + ["two.cu"] * 2
    assert text(tree) == text(tree, "debug.so") == "header\none\nslow\n"
