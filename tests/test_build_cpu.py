"""The library is built where the binding's native module cannot be: without the host compiler, PyTorch's headers or its
GPU libraries the build says so and goes on, and no module of an earlier build stays."""
import os

import pytest

from bit_unstructured_sparse_amd import build


@pytest.fixture
def places(tmp_path, monkeypatch):
    """The build's results in a folder of their own; commands are noted, and make what they are asked for."""
    for name, file in (("LIB", "lib.so"), ("PROBE_LIB", "probe.so"), ("BINDING", "_binding.so")):
        monkeypatch.setattr(build, name, str(tmp_path / file))
    ran = []

    def run(cmd, verbose):
        ran.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("made")

    monkeypatch.setattr(build, "_run", run)
    monkeypatch.setattr(build, "binding_command", lambda out: ["host-compiler", "-o", out])
    return tmp_path, ran


def test_everything(places):
    folder, ran = places
    assert build.build() == build.LIB
    assert sorted(os.listdir(folder)) == ["_binding.so", "lib.so", "probe.so"] and any(c[0] == "host-compiler" for c in ran)


@pytest.mark.parametrize("how", [RuntimeError("g++ failed:\nno torch/csrc/Dtype.h"), FileNotFoundError("g++")])
@pytest.mark.parametrize("stale", [False, True])
def test_without_the_native_module(how, stale, places, monkeypatch, capfd):
    folder, _ = places
    if stale:
        (folder / "_binding.so").write_text("of other sources")
    library = build._run

    def run(cmd, verbose):
        if cmd[0] == "host-compiler":
            raise how
        library(cmd, verbose)

    monkeypatch.setattr(build, "_run", run)
    assert build.build() == build.LIB
    assert sorted(os.listdir(folder)) == ["lib.so", "probe.so"]
    said = capfd.readouterr()
    assert "_binding.so" in said.err and str(how).splitlines()[-1] in said.err


def test_a_library_that_does_not_build_is_an_error(places, monkeypatch):
    def run(cmd, verbose):
        raise RuntimeError("hipcc failed")

    monkeypatch.setattr(build, "_run", run)
    with pytest.raises(RuntimeError):
        build.build()


def test_without_pytorch(places, monkeypatch):
    folder, _ = places
    monkeypatch.setattr(build, "binding_command", lambda out: None)
    build.build()
    assert sorted(os.listdir(folder)) == ["lib.so", "probe.so"]
