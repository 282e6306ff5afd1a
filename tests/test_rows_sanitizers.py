"""AddressSanitizer and UndefinedBehaviorSanitizer over the host code of the
operators on rows of scores, on the CPU: the library's host side built with the
sanitizers (GPU code is not instrumented) and driven by
tests/sanitize/rows_abi_main.c through the C ABI, every call of which returns
before any device work."""
import os

import pytest

# the toolchain's flags and helpers; a copy of the tree for GPU runs may lack that file
ts = pytest.importorskip("test_sanitizers")

SOURCES = ("sps_prepare.hip", "sps_score.hip", "sps_bsc.hip", "sps_select.hip", "sps_distill.hip",
           "sps_grad.hip", "sps_api.hip")


def test_row_operators_host_code_clean(tmp_path):
    ts._need(ts.HIPCC)
    ts._need(ts.CLANG)
    d = str(tmp_path)
    include = ["-I", os.path.join(ts.ROOT, "include"), "-I", ts.CSRC]
    ts._build([ts.HIPCC] + ts.HIP_FLAGS + ts.HIP_HOST_SAN + include + ["-o", "libsps_san.so"]
              + [os.path.join(ts.CSRC, f) for f in SOURCES], d)
    ts._build([ts.CLANG, "-std=c11"] + ts.C_SAN + include[:2]
              + [os.path.join(ts.SAN, "rows_abi_main.c"), "-L.", "-lsps_san", "-Wl,-rpath," + d,
                 "-o", "rsan"], d)
    r = ts._run(["./rsan"], d, ts.ENV)
    assert r.returncode == 0 and "clean" in r.stdout, r.stdout
