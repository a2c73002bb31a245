"""The argument validation of the 4-bit products with scales per group and of the
sampler under AddressSanitizer and UndefinedBehaviorSanitizer, built and run like
test_abi_sanitized.py (host code only, no GPU)."""
import os
import subprocess

import pytest

from tests.conftest import ROOT
from tests.test_abi_sanitized import SAN, _run
from ternary_weight_quantized_q2_amd import build_lib


def test_token_validation_under_sanitizers(tmp_path):
    if not os.path.exists(build_lib.HIPCC):
        pytest.fail("hipcc is needed to build the sanitized driver")
    csrc, objs = build_lib.CSRC, []
    for name in ("q2_linear.hip", "q2_a8.hip", "q2_pack.hip", "q4_matvec.hip", "q4_matvec32.hip", "q4_matvec64.hip",
                 "q4_matvec128.hip", "q2_sample.hip"):
        obj = os.path.join(build_lib.OBJ_DIR, name + ".o")
        if not os.path.exists(obj):                    # the library build leaves these behind
            build_lib._compile(os.path.join(csrc, name))
        objs.append(obj)
    for name in ("q2_api", "q2_token_api"):
        objs.append(str(tmp_path / f"{name}_san.o"))
        _run([build_lib.HIPCC, *build_lib.FLAGS, *SAN, "-c", os.path.join(csrc, name + ".hip"), "-o", objs[-1]])
    objs.append(str(tmp_path / "token_driver.o"))
    _run([build_lib.HIPCC, "-O1", "-std=c++17", "-I", build_lib.INCLUDE, *SAN, "-c",
          os.path.join(ROOT, "tests", "abi_sanitize", "token_driver.cpp"), "-o", objs[-1]])
    exe = str(tmp_path / "token_abi_driver")
    _run([build_lib.HIPCC, "--offload-arch=gfx950", *SAN, *objs, "-o", exe])
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1", HIP_VISIBLE_DEVICES="")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=120)
    assert r.returncode == 0 and "token abi driver ok" in r.stdout, r.stdout + r.stderr
