"""No launch of the optimizer and 4-bit calls exceeds what the runtime takes, at sizes up to the largest
accepted (CPU only): tests/launches/train_launches.cpp stands in for the runtime's launch."""
import os
import subprocess
import tempfile

import gradient_sync_amd as dps
from gradient_sync_amd import _build as B

HERE = os.path.dirname(os.path.abspath(__file__))


def test_every_launch_fits():
    dps.lib()
    with tempfile.TemporaryDirectory() as tmp:
        exe = os.path.join(tmp, "train_launches")
        cmd = ["/opt/rocm/llvm/bin/clang++", "-O1", "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I", "/opt/rocm/include",
               "-I", B.CSRC, "-I", os.path.join(B.ROOT, "include"), "-rdynamic",
               os.path.join(HERE, "launches", "train_launches.cpp"), "-ldl", "-o", exe]
        p = subprocess.run(cmd, capture_output=True, text=True)
        assert p.returncode == 0, p.stderr[-3000:]
        p = subprocess.run([exe, dps.LIB_PATH], capture_output=True, text=True, timeout=120)
        assert p.returncode == 0 and "0 failures" in p.stdout, (p.stdout[-2000:], p.stderr[-4000:])
