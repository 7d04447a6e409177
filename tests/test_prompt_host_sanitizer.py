"""The host code of rotary positions, prompt attention, slots and pages under
AddressSanitizer and UndefinedBehaviorSanitizer, with sizes at and past every
limit (CPU only; the sanitizers are on the host side of the build, device code
is unchanged)."""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil

import pytest

from tests.test_host_sanitizer import CLANG, CSRC, HIPCC, HOST_SAN, INCLUDE, LINK_SAN, ROCM, ROOT, _run

import subprocess


@pytest.mark.skipif(not (os.path.exists(HIPCC) and os.path.exists(CLANG)), reason="ROCm toolchain not found")
def test_prompt_validation_under_host_sanitizers(tmp_path):
    out = str(tmp_path)
    common = ["-O1", "-g", "-fno-omit-frame-pointer", "-std=c++17", "-fPIC", "-I", INCLUDE]

    def compile_one(name):
        obj = os.path.join(out, name + ".o")
        _run([HIPCC, "--offload-arch=gfx950", *common, *HOST_SAN, "-Xclang", "-target-feature", "-Xclang",
              "-packed-fp32-ops", "-I", CSRC, "-c", os.path.join(CSRC, name + ".hip"), "-o", obj])
        return obj

    with cf.ThreadPoolExecutor(max_workers=4) as ex:
        objs = list(ex.map(compile_one, ["attn_prompt", "attn_prompt_bwd", "kv_slots", "rope", "status"]))
    drv, exe = os.path.join(out, "driver.o"), os.path.join(out, "prompt_driver")
    _run([CLANG, *common, *LINK_SAN, "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROCM, "include"), "-c",
          os.path.join(ROOT, "tests", "host_sanitizer", "prompt_driver.cpp"), "-o", drv])
    _run([CLANG, *LINK_SAN, "-o", exe, drv, *objs, "-L", os.path.join(ROCM, "lib"), "-lamdhip64",
          "-Wl,-rpath," + os.path.join(ROCM, "lib")])
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)
    if r.returncode == 77:
        pytest.skip("a GPU is visible: the driver checks host code only")
    log = r.stdout + r.stderr
    assert "runtime error" not in log and "AddressSanitizer" not in log, log
    assert r.returncode == 0 and " 0 failures" in log, log
    shutil.rmtree(out, ignore_errors=True)
