"""CPU checks of the binding's loading: a library that is not this source's says
so and asks to be rebuilt, whatever it lacks."""

import shutil
import subprocess

import pytest

CC = shutil.which("gcc") or shutil.which("cc")


@pytest.mark.skipif(CC is None, reason="no C compiler")
@pytest.mark.parametrize("code", [
    "int sbl_abi_version(void) { return 10; }",            # another version, with or without the functions
    "int sbl_abi_version(void) { return 11; }",            # this version, older than its newest functions
    "int nothing(void) { return 0; }",
])
def test_a_library_of_another_source_is_refused(tmp_path, monkeypatch, code):
    from sparse_linear_layers_absmean_amd import sbl
    (tmp_path / "old.c").write_text(code)
    subprocess.run([CC, "-shared", "-fPIC", "old.c", "-o", "old.so"], cwd=tmp_path, check=True)
    monkeypatch.setattr(sbl, "LIB_PATH", str(tmp_path / "old.so"))
    monkeypatch.setattr(sbl, "_lib", None)
    with pytest.raises(RuntimeError, match="rebuild it"):
        sbl.load()
    assert sbl._lib is None


@pytest.mark.parametrize("private", [True, False])
def test_current_stream_with_and_without_torchs_own_function(monkeypatch, private):
    import torch
    from sparse_linear_layers_absmean_amd import sbl
    # stands in for a torch whose module has, or lacks, the function
    monkeypatch.setattr(sbl, "_raw_stream", (lambda device: 4096 + device) if private else None)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 2)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: type("Stream", (), {"cuda_stream": 8192}))
    assert sbl._stream(None) == (4098 if private else 8192)
    assert sbl._stream(64) == 64
