"""host_validation/driver_block.c on the library's host code under the sanitizers, built as test_host_sanitizers.py
builds its driver: the calls around experts of the caller's own."""
import concurrent.futures
import os
import subprocess

import pytest


@pytest.mark.timeout(600)
def test_block_host_code_under_the_sanitizers(tmp_path):
    hs = pytest.importorskip("test_host_sanitizers")
    if not (os.path.exists(hs.HIPCC) and os.path.exists(hs.CLANG)):
        pytest.skip("ROCm compilers not present")
    b = hs._build_module()
    flags = [f for f in b.FLAGS if f != "-O3"] + ["-O1", "-g", "-fno-omit-frame-pointer"] + hs.SAN

    def compile_one(src):
        obj = str(tmp_path / (src + ".o"))
        lang = ["-x", "hip"] if src.endswith(".hip") else []
        hs._run([hs.HIPCC] + flags + lang + ["-c", os.path.join(b.CSRC, src), "-o", obj])
        return obj

    with concurrent.futures.ThreadPoolExecutor(max_workers=8) as ex:
        objs = list(ex.map(compile_one, b.SOURCES))
    drv = str(tmp_path / "driver.o")
    san = [f for f in hs.SAN if f != "-Xarch_host"]
    hs._run([hs.CLANG, "-std=c11", "-Wall", "-Werror", "-O1", "-g"] + san +
            ["-I", os.path.join(hs.ROOT, "include"), "-c",
             os.path.join(hs.ROOT, "tests", "host_validation", "driver_block.c"), "-o", drv])
    exe = str(tmp_path / "driver")
    hs._run([hs.HIPCC, "--offload-arch=gfx950"] + hs.SAN + [drv] + objs + ["-o", exe])
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:halt_on_error=1",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1", HIP_VISIBLE_DEVICES="-1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)
    print(r.stdout)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "runtime error" not in r.stderr and "AddressSanitizer" not in r.stderr, r.stderr
    assert "failures 0" in r.stdout
