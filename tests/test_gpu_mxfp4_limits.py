"""4-bit calls of more workgroups than one launch has (2^24 - 1 of 256 threads)."""
import pytest
import torch

import gradient_sync_amd as dps
from tests.helpers import say

pytestmark = pytest.mark.gpu
DEV = "cuda"


def need(gib):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gib << 30:
        pytest.skip(f"needs {gib} GiB of GPU memory")


@pytest.fixture(autouse=True)
def leave_no_cache():
    yield
    torch.cuda.empty_cache()


def test_expansion_in_two_launches():
    """2^35 values and some: the last rows, which the second launch writes, and others."""
    rows, cols = (1 << 21) + 48, 1 << 14
    need(90)
    q = dps.Mxfp4(rows, cols)
    q.codes.view(-1).view(torch.int64).fill_(0x7654321076543210)
    q.scales.fill_(130)
    g = torch.Generator(device=DEV).manual_seed(1)
    q.codes[-96:].random_(generator=g)
    q.scales[-6:].random_(100, 150, generator=g)
    say("expansion in two launches")
    out = dps.dp_mxfp4_dequantize(q)
    part = dps.Mxfp4(96, cols, q.codes[-96:].clone(), q.scales[-6:].clone())
    assert torch.equal(out[-96:].view(torch.int16), dps.dp_mxfp4_dequantize(part).view(torch.int16))
    assert bool((out[:-96:4096].reshape(-1, 16) == 8 * torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, .5, 1, 1.5, 2, 3, 4, 6], device=DEV)).all())


def test_product_of_short_rows_in_two_launches():
    """Exactly one workgroup of 64 x 16 outputs more than a launch has, and 34 GB of C."""
    n = 1 << 17
    need(40)
    g = torch.Generator(device=DEV).manual_seed(2)
    a, b = (dps.dp_mxfp4_quantize(torch.randn(n, 64, generator=g, device=DEV)) for _ in range(2))
    say("product in two launches")
    c = torch.full((n, n), 5.0, dtype=torch.bfloat16, device=DEV)
    dps.dp_gemm_mxfp4(a, b, out=c)
    rows = lambda q, at, k: dps.Mxfp4(k, 64, q.codes[at:at + k].clone(), q.scales[at // 16:(at + k) // 16].clone())
    for at in (0, 1 << 16, n - 128):
        assert torch.equal(c[at:at + 128], dps.dp_gemm_mxfp4(rows(a, at, 128), b))
        assert torch.equal(c[:, at:at + 128], dps.dp_gemm_mxfp4(a, rows(b, at, 128)))
