"""The key/value cache calls' argument checks under the host address and
undefined-behaviour sanitizers (no GPU needed): every size of the structs at its
extremes, alone and in pairs."""

import concurrent.futures
import glob
import os
import shutil

import pytest

from int8_quantized_matmul_absmax_amd import build as B

# (skipped where the host-only files are absent)
H = pytest.importorskip("tests.test_host_sanitizers")

DRIVER = os.path.join(H.HERE, "kv_sanitizer_driver.cpp")


def test_kv_checks_under_host_sanitizers(tmp_path):
    if not (shutil.which("hipcc") or os.path.exists(os.path.join(H.ROCM, "bin", "hipcc"))):
        pytest.skip("hipcc not available")
    if not os.path.exists(H.CLANG):
        pytest.skip("ROCm clang++ not available")
    hipcc = B._hipcc()
    srcs = sorted(glob.glob(os.path.join(B.CSRC, "*.hip")))

    def compile_one(src):
        obj = str(tmp_path / (os.path.basename(src) + ".o"))
        rc, out = H._run([hipcc] + H._hipcc_flags() + ["-c", src, "-o", obj])
        assert rc == 0, "compile %s:\n%s" % (src, out)
        return obj

    with concurrent.futures.ThreadPoolExecutor(min(len(srcs), 8)) as ex:
        objs = list(ex.map(compile_one, srcs))
    exe, drv = str(tmp_path / "driver"), str(tmp_path / "driver.o")
    san = ["-fsanitize=address,undefined", "-fno-sanitize-recover=all"]
    rc, out = H._run([H.CLANG, "-std=c++17", "-O1", "-g"] + san
                     + ["-I", os.path.join(B.ROOT, "include"), "-c", DRIVER, "-o", drv])
    assert rc == 0, out
    lib = os.path.join(H.ROCM, "lib")
    rc, out = H._run([H.CLANG] + san + [drv] + objs
                     + ["-L" + lib, "-lamdhip64", "-Wl,-rpath," + lib, "-o", exe])
    assert rc == 0, out
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0", UBSAN_OPTIONS="print_stacktrace=1")
    rc, out = H._run([exe], env=env, timeout=300)
    assert rc == 0 and "ALL OK" in out, out
