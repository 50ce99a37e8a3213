"""The host code of the 8-bit floating-point linear (fp8_api.cpp, its packer) under
AddressSanitizer and UndefinedBehaviorSanitizer, as tests/test_host_sanitized.py
does for the others.  CPU only."""
import os
import shutil
import subprocess

import pytest

from tests.test_host_sanitized import CSRC, HERE, ROCM_INCLUDE, ROOT, SAN, _run


@pytest.fixture(scope="module")
def driver(tmp_path_factory):
    if shutil.which("g++") is None or not os.path.isdir(ROCM_INCLUDE):
        pytest.skip("needs g++ and the HIP headers")
    out = str(tmp_path_factory.mktemp("san_fp8") / "fp8_driver")
    src = [os.path.join(CSRC, f) for f in ("api.cpp", "fp8_api.cpp", "packer.cpp")]
    src += [os.path.join(HERE, f) for f in ("fake_runtime.cpp", "fp8_fake.cpp", "fp8_driver.cpp")]
    cmd = ["g++", "-std=c++17", "-O1", "-g", *SAN, "-D__HIP_PLATFORM_AMD__", "-I", ROCM_INCLUDE,
           "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-I", HERE, *src, "-o", out, "-lpthread"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-4000:]
    return out


@pytest.mark.parametrize("mode,env", [("full", {}), ("arch-mismatch", dict(FAKE_GFX_ARCH="gfx942")),
                                      ("no-device", dict(FAKE_DEVICE_COUNT="0"))])
def test_host_code_clean_under_sanitizers(driver, mode, env):
    res = _run(driver, mode, **env)
    assert res.returncode == 0, res.stdout + res.stderr[-6000:]
    assert "host checks passed" in res.stdout
