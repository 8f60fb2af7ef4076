"""The argument checks of the operators around the layer built with
AddressSanitizer and UndefinedBehaviorSanitizer on the host side only, driven
by tests/abi_sanitize/rows_harness.cpp over extreme sizes.  Nothing there
reaches a launch, so this runs on the CPU."""
import os
import subprocess

import pytest

from test_abi_sanitize import CSRC, FLAGS, HIPCC, ROOT, SAN

SOURCES = ("rows_api", "norm", "act", "gemm_pick", "gemm_split", "gemm_tile")


@pytest.mark.slow
@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not found")
def test_rows_abi_under_asan_and_ubsan(tmp_path):
    import concurrent.futures as cf

    def compile_one(src):
        obj = os.path.join(tmp_path, os.path.basename(src) + ".o")
        lang = ["-x", "hip"] if src.endswith(".hip") else []
        r = subprocess.run([HIPCC, *FLAGS, *SAN, *lang, "-c", src, "-o", obj], capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-3000:]
        return obj

    srcs = [os.path.join(CSRC, s + ".hip") for s in SOURCES]
    srcs.append(os.path.join(ROOT, "tests", "abi_sanitize", "rows_harness.cpp"))
    with cf.ThreadPoolExecutor(min(8, os.cpu_count() or 1)) as ex:
        objs = list(ex.map(compile_one, srcs))
    exe = os.path.join(tmp_path, "rows_harness")
    r = subprocess.run([HIPCC, "--offload-arch=gfx950", *SAN, *objs, "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0:halt_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1", HIP_VISIBLE_DEVICES="")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=600)
    out = r.stdout + r.stderr
    assert r.returncode == 0 and "rows sanitize harness: ok" in out, out[-4000:]
    assert "runtime error" not in out and "AddressSanitizer" not in out, out[-4000:]
