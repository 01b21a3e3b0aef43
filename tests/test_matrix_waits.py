"""The wait behind the matrix instructions whose results inline assembly writes (CPU only): at least as long as the one
that the compiler puts between the same instruction, written as a builtin, and the first use of its result."""
import os
import re
import subprocess
import tempfile

import pytest

from gradient_sync_amd import _build as B

KERNEL = """
#include <hip/hip_runtime.h>
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
__global__ void k(f32x4 *c, const i32x8 *a, const i32x8 *b)
{
    f32x4 x = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a[threadIdx.x], b[threadIdx.x], f32x4{}, %d, %d, 0, 1, 0, 1);
    x[0] += 1.0f;
    c[threadIdx.x] = x;
}
"""


def wait_states(lines):
    return sum(int(n) + 1 for n in re.findall(r"s_nop (\d+)", lines))


@pytest.fixture(scope="module")
def settle():
    text = open(os.path.join(B.CSRC, "mx_gemm_device.h")).read()
    return wait_states(re.search(r"void mx_settle\(\) \{ asm volatile\(\"([^)]*)\"", text).group(1))


@pytest.mark.parametrize("first,second", [(4, 4), (4, 0), (0, 0)])   # e2m1 and e4m3 operands
def test_settle_is_longer_than_the_compilers_wait(first, second, settle):
    with tempfile.TemporaryDirectory() as tmp:
        src, asm = os.path.join(tmp, "k.hip"), os.path.join(tmp, "k.s")
        open(src, "w").write(KERNEL % (first, second))
        subprocess.run([B.HIPCC, *B.FLAGS, "--cuda-device-only", "-S", src, "-o", asm], check=True, stdout=subprocess.DEVNULL,
                       stderr=subprocess.DEVNULL)
        body = open(asm).read()
    body = body[body.index("v_mfma_scale"):]
    own = wait_states(body[:body.index("v_add_f32")])
    assert 0 < own < settle, (own, settle)
