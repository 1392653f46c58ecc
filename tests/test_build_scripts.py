"""The build scripts that take the library's compiler call, each into a place of its own."""
import ctypes
import importlib.util
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def script(rel):
    spec = importlib.util.spec_from_file_location("_built_" + rel.replace("/", "_")[:-3], os.path.join(ROOT, rel))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("rel", ["bench_probe/build.py", "tests/devmath/build.py"])
def test_builds(rel, tmp_path):
    mod = script(rel)
    mod.LIB = str(tmp_path / "built.so")
    assert mod.build() == mod.LIB
    ctypes.CDLL(mod.LIB)


def test_the_librarys_compiler_call_takes_sources_and_objects(tmp_path):
    """Sources compiled and objects linked in one call, as the other scripts make it."""
    lib = script("sharded_mixed_precision_rank_amd/build.py")
    (tmp_path / "a.hip").write_text('extern "C" __attribute__((visibility("default"))) int a() { return 1; }\n')
    lib._hipcc([str(tmp_path / "a.hip")], [], str(tmp_path / "a.so"), [], False)
    assert ctypes.CDLL(str(tmp_path / "a.so")).a() == 1


def test_extra_flags_reach_every_compile_and_the_link(monkeypatch, tmp_path):
    lib = script("sharded_mixed_precision_rank_amd/build.py")
    calls = []
    monkeypatch.setattr(lib, "_run", lambda cmd, verbose: calls.append(cmd))
    monkeypatch.setattr(lib.subprocess, "run", lambda *args, **kw: None)
    lib.build(out=str(tmp_path / "built.so"), extra=("-lextra",))
    assert len(calls) == len(lib.SOURCES) + 1 and calls[-1][-1] == str(tmp_path / "built.so")
    assert all("-lextra" in cmd for cmd in calls)
