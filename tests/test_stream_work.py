"""How paged attention counts and deals the work of its key streams: the kernels'
own whole numbers (lact_stream_work.hpp) in a host program, under
UndefinedBehaviorSanitizer, for offsets in order and for those that name the same
rows again and again, whose work would pass 2^31 many times over."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = "/opt/rocm/bin/hipcc"


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="ROCm compiler not found")
def test_work_stays_inside_for_any_offsets(tmp_path):
    exe = str(tmp_path / "stream_work")
    r = subprocess.run([HIPCC, "--offload-arch=gfx950", "--offload-host-only", "-O1", "-g", "-std=c++17", "-w", "-Xarch_host",
                        "-fsanitize=undefined", "-I", os.path.join(ROOT, "test_layers_amd", "csrc"),
                        os.path.join(ROOT, "tests", "stream_work.hip"), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "424 walks, 0 failures" in r.stdout, r.stdout[-2000:] + r.stderr[-2000:]
    assert "runtime error" not in r.stderr, r.stderr[-2000:]
