"""The host-side checks of the calls around the dense projections (tests/test_dense_host.py) against the library build
whose host code carries AddressSanitizer and UndefinedBehaviorSanitizer. No GPU is used."""
import glob

import pytest

from tests.test_sanitizers import _child


def test_dense_host_checks_under_asan_ubsan():
    from gemm_nvfp4_amd import build
    lib = build.build_host_sanitized()
    rt = sorted(glob.glob("/opt/rocm/llvm/lib/clang/*/lib/linux/libclang_rt.asan-x86_64.so"))
    if not rt:
        pytest.skip("clang's ASan runtime is not installed")
    out = _child({"LD_PRELOAD": rt[-1], "NVFP4_TEST_LIB": lib}, ["tests/test_dense_host.py"])
    assert " passed" in out
