"""The compiled binding belongs to one torch and one Python: another's is rebuilt, and not loaded."""
import os

import pytest

import phase_disaggregated_quantized_b200 as nvq
from phase_disaggregated_quantized_b200 import build_lib


@pytest.fixture(scope="module", autouse=True)
def _built():
    build_lib.build()


def _compiles(monkeypatch, tmp_path):
    """Whether build_binding compiles, with a compiler that only writes the file that it is asked for."""
    runs = []

    def run(cmd, check):
        runs.append(cmd)
        open(cmd[cmd.index("-o") + 1], "wb").close()

    monkeypatch.setattr(build_lib.subprocess, "run", run)
    copy = tmp_path / "_binding.so"
    copy.write_bytes(open(nvq.BINDING_PATH, "rb").read())
    monkeypatch.setattr(build_lib, "BINDING", str(copy))
    build_lib.build_binding()
    return len(runs) > 0


def test_a_binding_of_this_torch_is_kept(monkeypatch, tmp_path):
    assert not _compiles(monkeypatch, tmp_path)


def test_a_binding_of_another_torch_is_rebuilt(monkeypatch, tmp_path):
    monkeypatch.setattr("torch.__version__", "99.0.0")
    assert _compiles(monkeypatch, tmp_path)


def test_a_binding_older_than_its_source_is_rebuilt(monkeypatch, tmp_path):
    newer = tmp_path / "binding.cpp"
    newer.write_text("")
    os.utime(newer, (4e9, 4e9))
    monkeypatch.setattr(build_lib, "BINDING_SOURCE", str(newer))
    assert _compiles(monkeypatch, tmp_path)


def test_a_binding_of_another_torch_is_not_loaded(monkeypatch):
    monkeypatch.setattr(nvq, "_fast", None)
    monkeypatch.setattr("torch.__version__", "99.0.0")
    with pytest.raises(RuntimeError, match="another torch"):
        nvq._load_binding()


def test_the_loaded_binding_names_what_it_was_built_for():
    assert nvq._load_binding().built_for == build_lib.binding_tag()
