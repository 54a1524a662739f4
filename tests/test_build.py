"""The build on the CPU: libfp8fg.so, which needs neither torch nor Python's
headers, is linked also where the Python module cannot be built."""

import ctypes
import os

import pytest

from fp8_fine_grained_x1_amd import build


def test_the_c_library_is_linked_without_the_python_module(tmp_path, monkeypatch):
    if not os.path.exists(build.HIPCC):
        pytest.skip("hipcc not available")

    def no_torch():
        raise ImportError("no torch here")

    def small(src, outdir=None, extra=()):
        # one tiny source in place of the library's
        import subprocess
        obj = str(tmp_path / (src + ".o"))
        code = "extern \"C\" int built_%s() { return 7; }" % src.split(".")[0]
        subprocess.run(["g++", "-fPIC", "-x", "c++", "-c", "-o", obj, "-"], input=code, text=True, check=True)
        return obj

    lib, native = str(tmp_path / "lib.so"), str(tmp_path / "native.so")
    for name, value in (("BUILD", str(tmp_path)), ("LIB", lib), ("NATIVE", native), ("SOURCES", ["one.cpp"]),
                        ("_compile", small), ("_compile_native", no_torch)):
        monkeypatch.setattr(build, name, value)
    with pytest.raises(ImportError):
        build.build(verbose=False)
    assert ctypes.CDLL(lib).built_one() == 7 and not os.path.exists(native)
