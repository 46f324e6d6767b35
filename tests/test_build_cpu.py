"""How the compiled parts come to be: whole files or none, the CPython module for this Python and this
torch, and the CUDA library without either."""
import os
import stat
import sys
import threading

import pytest

from gated_linear_attention_relu_b200 import build

COMPILER = """#!/bin/sh
while [ "$1" != "-o" ]; do shift; done
printf half > "$2"
sleep 0.4
[ -e "{stop}" ] && exit 1
printf whole > "$2"
"""


@pytest.fixture
def slow(tmp_path, monkeypatch):
    """A compiler that takes its time over its output; (folder, the file that makes it fail)."""
    stop, cc = tmp_path / "stop", tmp_path / "cc"
    cc.write_text(COMPILER.format(stop=stop))
    cc.chmod(cc.stat().st_mode | stat.S_IXUSR)
    folder = tmp_path / "out"
    folder.mkdir()
    monkeypatch.setenv("CXX", str(cc))
    monkeypatch.setenv("NVCC", str(cc))
    monkeypatch.setattr(build, "HERE", str(folder))
    monkeypatch.setattr(build, "LIB", str(folder / "liblinattn.so"))
    return folder, stop


@pytest.mark.parametrize("what", ["marshal", "library"])
def test_processes_that_build_together_see_whole_files(slow, what):
    make = build.build_marshal if what == "marshal" else build.build_library
    out = build.marshal_path() if what == "marshal" else build.LIB
    workers = [threading.Thread(target=make, args=(True,)) for _ in range(3)]
    seen = set()
    for w in workers:
        w.start()
    while any(w.is_alive() for w in workers):
        if os.path.exists(out):
            with open(out) as f:
                seen.add(f.read())
    with open(out) as f:
        seen.add(f.read())
    assert seen == {"whole"}
    assert os.listdir(slow[0]) == [os.path.basename(out)]


def test_a_failed_build_leaves_nothing(slow):
    folder, stop = slow
    stop.touch()
    for make in (build.build_marshal, build.build_library):
        with pytest.raises(RuntimeError, match="failed building"):
            make(True)
    assert os.listdir(folder) == []


def test_module_belongs_to_its_python_torch_and_sources(monkeypatch, tmp_path):
    import sysconfig

    import torch

    names = {build.marshal_path()}
    assert build.marshal_path() in names
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", "0.0")
        names.add(build.marshal_path())
    with monkeypatch.context() as m:
        m.setattr(sysconfig, "get_config_var", lambda name: "other")
        names.add(build.marshal_path())
    with monkeypatch.context() as m:
        source = tmp_path / "marshal.cpp"
        source.write_text("// another one")
        m.setattr(build, "MARSHAL_SOURCE", str(source))
        names.add(build.marshal_path())
    assert len(names) == 4


def test_cuda_library_is_built_without_torch(slow, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)
    assert build.build_library(True) == build.LIB and os.path.exists(build.LIB)


def test_module_that_is_there_is_not_built_again(slow):
    out = build.build_marshal()
    os.utime(out, (0, 0))
    assert build.build_marshal() == out and os.path.getmtime(out) == 0
