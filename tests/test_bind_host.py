"""The compiled module of the short calls is an option: what it is not there for runs without it.
CPU only."""
import os
import shutil
import subprocess
import sys
import warnings

import pytest
import torch

from paged_kv_cache_09_gb300 import _build


@pytest.fixture
def pa():
    if shutil.which("nvcc") is None:
        pytest.skip("nvcc not available")
    import paged_kv_cache_09_gb300
    paged_kv_cache_09_gb300.build()
    return paged_kv_cache_09_gb300


@pytest.mark.parametrize("there", [False, True])
def test_calls_without_the_module(pa, monkeypatch, tmp_path, there):
    # Not there, or no module of this interpreter: the library's other calls do not look at it, and those
    # that would take the short way check their arguments in Python, as they do for unusual ones.
    path = tmp_path / "pa_bind.so"
    if there:
        path.write_bytes(b"no module")
    monkeypatch.setattr(_build, "BIND", str(path))
    monkeypatch.setattr(pa, "_lib", None)
    monkeypatch.setattr(pa, "_bind", None)
    with warnings.catch_warnings():
        warnings.simplefilter("error")  # (no word before a call that wants it)
        assert isinstance(pa.prefill_workspace_size(10, 0, True, 24, 4, 256, 832), int)
        assert pa.q8_cache_shapes(1, 16, 1)[1] == (1, 1, 1)
    x = torch.zeros(3, 1, 256, dtype=torch.bfloat16)
    codes = torch.zeros(1, 16, 1, 256, dtype=torch.uint8).view(torch.float8_e4m3fn)
    args = (x, x, codes, codes, x[:1, :, :1].to(torch.uint8), x[:1, :, :1].to(torch.uint8), torch.arange(3))
    with pytest.warns(RuntimeWarning, match="pa_bind"), pytest.raises(TypeError, match="must be a CUDA tensor"):
        pa.reshape_and_cache_q8(*args)
    with warnings.catch_warnings():
        warnings.simplefilter("error")  # (said once)
        with pytest.raises(TypeError, match="must be a CUDA tensor"):
            pa.decode_q8(x, *args[2:6], torch.zeros(3, 1, dtype=torch.int32), torch.zeros(3, dtype=torch.int32), 1.0, 16)
        with pytest.raises(TypeError, match="must be a CUDA tensor"):
            pa.gather_cache_q8(*args[2:])


@pytest.mark.parametrize("compiler", ["none", "fails"])
def test_build_without_a_compiler_for_the_module(pa, monkeypatch, tmp_path, compiler):
    # The library is built all the same, and no module of other sources than its own stays beside it.
    stale, tools = tmp_path / "pa_bind.so", tmp_path / "bin"
    stale.write_bytes(b"")
    os.utime(stale, (0, 0))
    tools.mkdir()
    if compiler == "fails":
        (tools / "g++").write_text("#!/bin/sh\necho no headers >&2\nexit 1\n")
        (tools / "g++").chmod(0o755)
    monkeypatch.setattr(_build, "BIND", str(stale))
    monkeypatch.setenv("PATH", str(tools))
    with pytest.warns(RuntimeWarning, match="pa_bind" if compiler == "none" else "no headers"):
        assert _build.build() == _build.LIB
    assert not stale.exists()


def _imported(code):
    """The package imported by a fresh interpreter after `code`: what it says the module's file is."""
    run = subprocess.run([sys.executable, "-c", code + "\nfrom paged_kv_cache_09_gb300 import _build\n"
                          "print(_build.BIND)"], cwd=_build.ROOT, capture_output=True, text=True)
    assert run.returncode == 0, run.stderr
    return run.stdout.strip()


def test_import_needs_no_metadata_of_torch():
    # (A torch that is used from where it was built has none.)
    path = _imported("""
import importlib.metadata as m, torch
def version(name):
    raise m.PackageNotFoundError(name)
m.version = version""")
    assert path == _build.BIND and torch.__version__ in path


def test_another_python_looks_for_a_module_of_its_own():
    path = _imported("""
import torch, sysconfig
was = sysconfig.get_config_var
sysconfig.get_config_var = lambda name: '.cpython-399-another.so' if name == 'EXT_SUFFIX' else was(name)""")
    assert path.endswith(".cpython-399-another.so") and path != _build.BIND
