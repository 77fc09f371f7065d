"""The binding's extension module is optional: the library is built and used
without it, and never with one that was built for another torch (CPU)."""
import os
import subprocess
import sys
import textwrap
import warnings

import pytest
import torch

from hybrid_linear_attention_packed_gb300 import build as spanla_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def small_tree(tmp_path, monkeypatch):
    """A library of one empty translation unit, in a folder of its own."""
    src = tmp_path / "one.cu"
    src.write_text("extern \"C\" int one() { return 1; }\n")
    monkeypatch.setattr(spanla_build, "_sources", lambda: [str(src)])
    monkeypatch.setattr(spanla_build, "BUILD", str(tmp_path / "objects"))
    monkeypatch.setattr(spanla_build, "LIB", str(tmp_path / "libone.so"))
    monkeypatch.setattr(spanla_build, "EXT", str(tmp_path / "_ext.so"))
    return tmp_path


def _missing(*_):
    raise RuntimeError("no host compiler")


def test_library_is_built_where_the_extension_cannot_be(small_tree, monkeypatch):
    monkeypatch.setattr(spanla_build, "_compile_ext", _missing)
    with pytest.warns(UserWarning, match="no host compiler"):
        lib = spanla_build.build()
    assert os.path.exists(lib) and not os.path.exists(spanla_build.EXT)
    made = os.path.getmtime(lib)
    with pytest.warns(UserWarning, match="no host compiler"):
        spanla_build.build()
    assert os.path.getmtime(lib) == made          # the library itself is not stale


def test_an_older_extension_goes_when_it_cannot_be_rebuilt(small_tree, monkeypatch):
    """(It could hold structures of another header.)"""
    with open(spanla_build.EXT, "w"):
        pass
    os.utime(spanla_build.EXT, (1, 1))
    monkeypatch.setattr(spanla_build, "_compile_ext", _missing)
    with pytest.warns(UserWarning):
        spanla_build.build()
    assert not os.path.exists(spanla_build.EXT)


def test_extension_is_rebuilt_for_another_torch(small_tree, monkeypatch):
    made = []

    def compile_ext():
        made.append(torch.__version__)
        tmp = spanla_build.EXT + ".tmp"
        with open(tmp, "w"):
            pass
        return tmp

    monkeypatch.setattr(spanla_build, "_compile_ext", compile_ext)
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        spanla_build.build()
        lib = os.path.getmtime(spanla_build.LIB)
        spanla_build.build()
        assert len(made) == 1
        monkeypatch.setattr(torch, "__version__", "0.0.1+other")
        spanla_build.build()
        spanla_build.build()
    assert len(made) == 2 and os.path.getmtime(spanla_build.LIB) == lib


def _child(code):
    r = subprocess.run([sys.executable, "-c", textwrap.dedent(code)], capture_output=True, text=True, cwd=ROOT, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    return r.stdout.strip().splitlines()[-1]


def test_extension_is_used_with_the_torch_it_was_built_for_only():
    spanla_build.build()
    load = """
        import torch
        from hybrid_linear_attention_packed_gb300 import spanla
        %s
        spanla.load_library()
        print(spanla._fast is not None)
    """
    assert _child(load % "") == "True"
    assert _child(load % "torch.__version__ = '0.0.1+other'") == "False"


REPORT = """ptxas info    : Compiling entry function '_ZN6spanla18paged_chunk_kernelILb0ELb%dEEEv' for 'sm_103a'
ptxas info    : Function properties for _ZN6spanla18paged_chunk_kernelILb0ELb%dEEEv
    48 bytes stack frame, 388 bytes spill stores, 540 bytes spill loads
ptxas info    : Used %d registers, used 1 barriers
"""


def test_registers_of_the_chunk_kernel_are_checked_by_the_build():
    """Its warps share out the block's registers: with fewer than they ask for one would wait for ever."""
    other = REPORT.replace("ILb0E", "ILb1E")
    good = REPORT % (0, 0, 168) + REPORT % (1, 1, 168) + other % (0, 0, 128) + other % (1, 1, 128)
    spanla_build._check_registers("csrc/k_paged_chunk.cu", good)
    spanla_build._check_registers("csrc/k_scan.cu", "")
    for bad in (good.replace("Used 128", "Used 120"), good.replace("Used 168 registers", "Used 160 registers", 1), REPORT % (0, 0, 168), ""):
        with pytest.raises(RuntimeError, match="registers a thread"):
            spanla_build._check_registers("csrc/k_paged_chunk.cu", bad)
