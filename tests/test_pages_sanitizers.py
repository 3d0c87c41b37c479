"""Refusals and queries of packed and paged attention, page slots and writes
under AddressSanitizer and UndefinedBehaviorSanitizer, on the CPU: the library's
host code alone is built with both (an empty device image beside it: no device,
nothing that would load it) and tests/pages_abi_driver.c walks the entry points
with the largest and smallest arguments."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = "/opt/rocm/bin/hipcc"
CLANG = "/opt/rocm/llvm/bin/clang"
SAN = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined"]


def _device_visible() -> bool:
    try:
        import torch
    except ImportError:
        return True   # cannot tell: treat as visible
    return torch.cuda.device_count() > 0


def _run(*cmd, **kw):
    r = subprocess.run(cmd, capture_output=True, text=True, **kw)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-3000:]
    return r


@pytest.mark.skipif(not (os.path.exists(HIPCC) and os.path.exists(CLANG)), reason="ROCm compilers not found")
@pytest.mark.timeout(900)
def test_pages_abi_paths_under_asan_and_ubsan(tmp_path):
    if _device_visible():
        pytest.skip("a device is visible: the driver's fake-pointer calls are not made")
    src, include = os.path.join(ROOT, "test_layers_amd", "csrc"), os.path.join(ROOT, "include")
    obj, stub, lib, exe = (str(tmp_path / n) for n in ("host.o", "image.c", "liblact_san.so", "driver"))
    _run(HIPCC, "--offload-arch=gfx950", "--offload-host-only", "-O1", "-g", "-std=c++17", "-fPIC", "-w", *SAN,
         "-Xarch_host", "-fno-omit-frame-pointer", "-I", include, "-I", src, "-c", os.path.join(src, "liblact.hip"),
         "-o", obj)
    images = [x.split()[-1] for x in _run("nm", obj).stdout.splitlines() if " U __hip_fatbin" in x]
    with open(stub, "w") as f:
        f.writelines(f"const char {x}[4096] __attribute__((aligned(4096))) = {{0}};\n" for x in images)
    _run(CLANG, "-fPIC", "-c", stub, "-o", stub + ".o")
    _run(HIPCC, "-shared", "-fPIC", *SAN, obj, stub + ".o", "-o", lib)
    _run(CLANG, "-std=c11", "-g", "-O1", "-fsanitize=address,undefined", "-fno-omit-frame-pointer", "-I", include,
         os.path.join(ROOT, "tests", "pages_abi_driver.c"), "-L", str(tmp_path), "-llact_san", f"-Wl,-rpath,{tmp_path}",
         "-o", exe)
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1", UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1",
               HIP_VISIBLE_DEVICES="")
    r = _run(exe, env=env, timeout=300)
    assert " 0 failures" in r.stdout, r.stdout
    assert "runtime error" not in r.stderr and "AddressSanitizer" not in r.stderr, r.stderr[-3000:]
