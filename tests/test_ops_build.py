"""The build of the GEMM library and of the operators' extension beside it (CPU; in a folder of its own)."""
import os
import subprocess

import pytest

from bit_exact_fp8_gb300 import build


@pytest.fixture
def small(monkeypatch, tmp_path):
    """The build on sources that compile in a moment, with its outputs in tmp_path."""
    src = tmp_path / "small.cu"
    src.write_text('extern "C" int answer() { return 42; }\n')
    for lib, sources, deps in (("LIB", "SOURCES", "DEPS"), ("PEAKS_LIB", "PEAKS_SOURCES", "PEAKS_DEPS")):
        monkeypatch.setattr(build, lib, str(tmp_path / (lib.lower() + ".so")))
        monkeypatch.setattr(build, sources, [str(src)])
        monkeypatch.setattr(build, deps, [str(src)])
    monkeypatch.setattr(build, "OPS_LIB", str(tmp_path / "ops.so"))
    return tmp_path


def no_torch(out):
    raise ImportError("no module named torch")


@pytest.mark.parametrize("commands", [lambda out: (["false"], ["false"]), lambda out: (["true"], ["false"]),
                                      lambda out: (["no-such-compiler"], []), no_torch])
def test_the_libraries_need_no_host_extension(small, monkeypatch, commands):
    monkeypatch.setattr(build, "ops_commands", commands)
    with pytest.raises(subprocess.CalledProcessError, match="ops.so"):
        build.build()
    assert os.path.exists(build.LIB) and os.path.exists(build.PEAKS_LIB) and not os.path.exists(build.OPS_LIB)
    assert not [f for f in os.listdir(small) if ".tmp" in f]


def test_the_extension_does_not_hide_a_failed_library(small, monkeypatch):
    (small / "small.cu").write_text("not C++")
    monkeypatch.setattr(build, "ops_commands", lambda out: (["true"], ["touch", out]))
    with pytest.raises(subprocess.CalledProcessError, match="lib.so"):
        build.build()
    assert not os.path.exists(build.LIB) and not os.path.exists(build.OPS_LIB)


def test_an_extension_of_another_torch_is_made_anew(monkeypatch):
    from bit_exact_fp8_gb300 import _lib
    build.build()
    assert build.up_to_date() and build.ops_built_for(build.OPS_LIB) == build.built_for()
    assert _lib.load_ops().built_for == build.OPS_MARK + build.built_for()
    for module in (build, _lib):
        monkeypatch.setattr(module, "built_for", lambda: "torch 0.0, another")
    assert not build.up_to_date()
    with pytest.raises(OSError, match="another torch|built for"):
        _lib.load_ops()
