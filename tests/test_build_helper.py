"""The build helper: what makes the library stale, and builds at the same
time.  With a stand-in for the compiler; no GPU."""
import importlib.util
import os
import sys
import threading
import time

import pytest

PKG = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "speculative_decoding_draft_column_gb300")


@pytest.fixture
def helper(tmp_path, monkeypatch):
    """The helper with sources and library of its own, all of one age."""
    spec = importlib.util.spec_from_file_location("_build_under_test", os.path.join(PKG, "_build.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    src = tmp_path / "csrc"
    src.mkdir()
    old = os.path.getmtime(os.path.join(PKG, "_build.py")) - 100
    for name in ("specsel.cu", "paged.cu", "common.cuh", "host.h", "specsel.h"):
        (src / name).write_text(name)
        os.utime(src / name, (old, old))
    monkeypatch.setattr(m, "CSRC", str(src))
    monkeypatch.setattr(m, "SRCS", [str(src / "specsel.cu"), str(src / "paged.cu")])
    monkeypatch.setattr(m, "HDR", str(src / "specsel.h"))
    monkeypatch.setattr(m, "LIB", str(tmp_path / "libspecsel.so"))
    return m


@pytest.mark.parametrize("name", ["specsel.cu", "paged.cu", "common.cuh", "host.h", "specsel.h"])
def test_every_source_and_header_counts(helper, name):
    now = time.time() + 10
    out = helper.LIB
    open(out, "w").close()
    os.utime(out, (now, now))
    assert not helper.stale(out)
    path = os.path.join(helper.CSRC, name)
    os.utime(path, (now + 10, now + 10))
    assert helper.stale(out)


def test_the_helper_itself_counts(helper):
    """Its flags are part of the library."""
    then = os.path.getmtime(os.path.join(PKG, "_build.py")) - 50
    open(helper.LIB, "w").close()
    os.utime(helper.LIB, (then, then))
    assert helper.stale(helper.LIB)


def test_builds_at_the_same_time_do_not_mix(helper, monkeypatch):
    """Two builds, one a little later: each links its own objects, and the
    library is never there in part."""
    compile_ = "import sys, time; f = open(sys.argv[1], 'w'); time.sleep(float(sys.argv[3])); f.write(sys.argv[2] + chr(10)); f.close()"
    link = ("import sys, time; x = ''.join(open(p).read() for p in sys.argv[3:]); f = open(sys.argv[1], 'w'); f.write(x[:3]); f.flush(); "
            "time.sleep(0.3); f.write(x[3:]); f.close()")

    def command(out, srcs, extra=()):
        if "-shared" in extra:
            return [sys.executable, "-c", link, out, "", *srcs]
        return [sys.executable, "-c", compile_, out, threading.current_thread().name, "0.1" if "specsel" in srcs[0] else "0.8"]

    monkeypatch.setattr(helper, "command", command)
    seen, done = [], threading.Event()

    def watch():
        while not done.is_set():
            try:
                seen.append(open(helper.LIB).read())
            except FileNotFoundError:
                pass
            time.sleep(0.01)

    watcher = threading.Thread(target=watch)
    watcher.start()
    builds = [threading.Thread(target=helper.build, args=(True,), name=n) for n in ("one", "two")]
    for b in builds:
        b.start()
        time.sleep(0.4)
    for b in builds:
        b.join()
    done.set()
    watcher.join()
    assert set(seen + [open(helper.LIB).read()]) <= {"one\none\n", "two\ntwo\n"}
    assert sorted(os.listdir(os.path.dirname(helper.LIB))) == ["csrc", "libspecsel.so"]
    assert sorted(os.listdir(helper.CSRC)) == ["common.cuh", "host.h", "paged.cu", "specsel.cu", "specsel.h"]
