"""The host side of the experts' products, the beam selection and the cache reordering under AddressSanitizer and
UndefinedBehaviorSanitizer (see test_sanitize.py, whose build of the library this uses).  No GPU."""
import os

import pytest

sanitize = pytest.importorskip("test_sanitize")  # a checkout for GPU runs may leave the sanitizers' files out
CLANG, ROOT, SAN, SAN_FLAGS = sanitize.CLANG, sanitize.ROOT, sanitize.SAN, sanitize.SAN_FLAGS


@pytest.mark.skipif(not os.path.exists(CLANG), reason="ROCm clang not installed")
def test_search_host_side_under_asan_ubsan(tmp_path):
    lib = sanitize._sanitized_library()
    exe = str(tmp_path / "search_driver")
    res = sanitize._run([CLANG, *SAN_FLAGS, "-I", os.path.join(ROOT, "include"), os.path.join(SAN, "search_driver.c"), "-o",
                exe, lib, f"-Wl,-rpath,{os.path.dirname(lib)}", "-L/opt/rocm/lib", "-lamdhip64",
                "-Wl,-rpath,/opt/rocm/lib", "-lstdc++", "-lm"])
    assert res.returncode == 0, res.stderr
    # leak checking is off: the HIP runtime keeps allocations until exit
    res = sanitize._run([exe], {"ASAN_OPTIONS": "detect_leaks=0:halt_on_error=1"})
    assert res.returncode == 0, res.stdout + res.stderr
    assert "all checks passed" in res.stdout
    assert "runtime error" not in res.stderr
