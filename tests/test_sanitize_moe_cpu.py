"""The argument validation of the mixture-of-experts entries (moe_abi.cpp) under
AddressSanitizer and UndefinedBehaviorSanitizer: host code only, no GPU call.
A sanitizer report or an unexpected status fails the test."""

import os

import pytest

from test_sanitize_cpu import BUILD, DEVICE_OBJECTS, DRIVERS, ENV, HOST_SAN, ROOT, _hipcc, _run


def test_moe_abi_validation_under_asan_and_ubsan(tmp_path):
    hipcc = _hipcc()
    if hipcc is None:
        pytest.skip("hipcc not found")
    objs = [os.path.join(BUILD, o) for o in
            DEVICE_OBJECTS + ["abi.o", "moe_route.o", "moe_slots.o", "moe_combine.o", "gemv_w4.o"]]
    if not all(os.path.exists(o) for o in objs):
        pytest.skip("the library's objects are not built (computation_collective_amd/build.py)")
    flags = ["-x", "hip", "--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-fPIC",
             "-I", os.path.join(ROOT, "include"), "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops"]
    abi_o, drv_o, exe = str(tmp_path / "moe_abi.o"), str(tmp_path / "drv.o"), str(tmp_path / "moe_abi_driver")
    for src, obj in ((os.path.join(ROOT, "computation_collective_amd", "csrc", "moe_abi.cpp"), abi_o),
                     (os.path.join(DRIVERS, "moe_abi_driver.cpp"), drv_o)):
        rc, out = _run([hipcc] + flags + HOST_SAN + ["-c", src, "-o", obj])
        assert rc == 0, out
    rc, out = _run([hipcc, "--offload-arch=gfx950"] + HOST_SAN + [drv_o, abi_o] + objs + ["-o", exe])
    assert rc == 0, out
    # (leak checking off: the HIP runtime's own allocations live until exit; no GPU is shown to the program)
    rc, out = _run([exe], env=dict(ENV, ASAN_OPTIONS="halt_on_error=1:detect_leaks=0", HIP_VISIBLE_DEVICES=""))
    assert rc == 0 and " 0 failures" in out, out
    assert "Sanitizer" not in out and "runtime error" not in out, out
