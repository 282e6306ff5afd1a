"""AddressSanitizer and UndefinedBehaviorSanitizer over the host code of the operators on dense
rows, on the CPU: the library's host side built with the sanitizers (GPU code is not
instrumented) and driven by tests/sanitize/dense_abi_main.c through the C ABI, every call of
which returns before any device work."""
import os

import pytest

from sparse_embedding_exact_amd import _build

# the toolchain's flags and helpers; a copy of the tree for GPU runs may lack that file
ts = pytest.importorskip("test_sanitizers")


def test_dense_operators_host_code_clean(tmp_path):
    ts._need(ts.HIPCC)
    ts._need(ts.CLANG)
    d = str(tmp_path)
    include = ["-I", os.path.join(ts.ROOT, "include"), "-I", ts.CSRC]
    ts._build([ts.HIPCC] + ts.HIP_FLAGS + ts.HIP_HOST_SAN + include + ["-o", "libsps_san.so"]
              + _build.SOURCES, d)
    ts._build([ts.CLANG, "-std=c11"] + ts.C_SAN + include[:2]
              + [os.path.join(ts.SAN, "dense_abi_main.c"), "-L.", "-lsps_san", "-Wl,-rpath," + d,
                 "-o", "dsan"], d)
    r = ts._run(["./dsan"], d, ts.ENV)
    assert r.returncode == 0 and "clean" in r.stdout, r.stdout
