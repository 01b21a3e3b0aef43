"""The host side of the optimizer and 4-bit entry points under AddressSanitizer and
UndefinedBehaviorSanitizer (CPU only): tests/sanitize/train_driver.cpp stands in for the launches and
checks the tables they are given."""
import os
import subprocess
import tempfile

from gradient_sync_amd import _build as B

HERE = os.path.dirname(os.path.abspath(__file__))


def test_train_host_code_under_sanitizers():
    with tempfile.TemporaryDirectory() as tmp:
        exe = os.path.join(tmp, "train_driver")
        cmd = ["/opt/rocm/llvm/bin/clang++", "-O1", "-g", "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I", "/opt/rocm/include",
               "-I", B.CSRC, "-I", os.path.join(B.ROOT, "include"), "-fsanitize=address,undefined",
               "-fno-sanitize-recover=all", "-x", "c++", os.path.join(B.CSRC, "api_train.hip"),
               os.path.join(HERE, "sanitize", "train_driver.cpp"), "-o", exe]
        p = subprocess.run(cmd, capture_output=True, text=True)
        assert p.returncode == 0, p.stderr[-3000:]
        env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1", UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
        p = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=120)
        assert p.returncode == 0 and "0 failures" in p.stdout, (p.stdout[-2000:], p.stderr[-4000:])


def test_train_refusals_under_sanitizers():
    """Every refusal's status, and nothing launched for it (tests/sanitize/train_alias_driver.cpp)."""
    with tempfile.TemporaryDirectory() as tmp:
        exe = os.path.join(tmp, "train_alias_driver")
        cmd = ["/opt/rocm/llvm/bin/clang++", "-O1", "-g", "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I", "/opt/rocm/include",
               "-I", B.CSRC, "-I", os.path.join(B.ROOT, "include"), "-fsanitize=address,undefined",
               "-fno-sanitize-recover=all", "-x", "c++", os.path.join(B.CSRC, "api_train.hip"),
               os.path.join(HERE, "sanitize", "train_alias_driver.cpp"), "-o", exe]
        p = subprocess.run(cmd, capture_output=True, text=True)
        assert p.returncode == 0, p.stderr[-3000:]
        env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1", UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
        p = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=120)
        assert p.returncode == 0 and "0 failures" in p.stdout, (p.stdout[-2000:], p.stderr[-4000:])
