"""Which objects a build compiles and links, with a compiler that writes down its
flags in place of code."""
import os
import stat
import sys

import pytest

FAKE = '''#!{python}
import sys
args = sys.argv[1:]
out = args[args.index("-o") + 1]
if "-c" in args:
    text = " ".join(a for a in args if a.startswith("-D")) + " " + open(args[-1]).read() + "\\n"
else:
    text = "".join(open(a).read() for a in args if a.endswith(".o"))
open(out, "w").write(text)
'''


@pytest.fixture
def build(monkeypatch, tmp_path):
    from linear_attention_recurrent_lq_b200 import build as b
    nvcc = tmp_path / "nvcc"
    nvcc.write_text(FAKE.format(python=sys.executable))
    nvcc.chmod(nvcc.stat().st_mode | stat.S_IXUSR)
    monkeypatch.setenv("NVCC", str(nvcc))
    (tmp_path / "csrc").mkdir()
    for name in ("a", "b"):
        (tmp_path / "csrc" / f"{name}.cu").write_text(name)
    monkeypatch.setattr(b, "HERE", str(tmp_path))
    monkeypatch.setattr(b, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(b, "OBJ", str(tmp_path / "_build"))
    monkeypatch.setattr(b, "_headers_of", lambda src: [])
    monkeypatch.setattr(b, "_deps", b._sources)
    for p in b._sources():
        os.utime(p, (1, 1))
    return b


def lib(b):
    return sorted(line.split() for line in open(b.LIB).read().splitlines())


def touch(b, name, text):
    path = os.path.join(b.HERE, "csrc", name)
    with open(path, "w") as f:
        f.write(text)
    t = os.path.getmtime(b.LIB) + 10
    os.utime(path, (t, t))


def test_flags_of_one_build_do_not_stay_in_the_next(build):
    build.build()
    assert lib(build) == [["a"], ["b"]]
    build.build(force=True, extra=["-DX=1"])
    assert lib(build) == [["-DX=1", "a"], ["-DX=1", "b"]]
    touch(build, "a.cu", "a2")
    build.build()
    assert lib(build) == [["a2"], ["b"]]


def test_a_library_with_other_flags_is_built_anew(build):
    build.build(extra=["-DX=1"])
    assert lib(build) == [["-DX=1", "a"], ["-DX=1", "b"]]
    assert build.needs_build() and not build.needs_build(["-DX=1"])
    build.build()
    assert lib(build) == [["a"], ["b"]]
    assert not build.needs_build()
    build.build(extra=["-DY=1"])
    assert lib(build) == [["-DY=1", "a"], ["-DY=1", "b"]]


def test_only_older_objects_are_compiled(build):
    build.build()
    obj = os.path.join(build.OBJ, "b.o")
    before = os.path.getmtime(obj)
    touch(build, "a.cu", "a2")
    build.build()
    assert lib(build) == [["a2"], ["b"]] and os.path.getmtime(obj) == before


def test_a_library_without_a_record_counts_as_built_without_flags(build):
    build.build()
    os.remove(os.path.join(build.OBJ, "extra_flags"))
    assert not build.needs_build()
