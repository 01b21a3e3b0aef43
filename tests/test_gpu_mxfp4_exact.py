"""Large 4-bit products of small numbers, exact in any order of addition: both tile sizes, one tile a workgroup
and several in turn, edges, every remainder of k, and each kind of store of C."""
import pytest
import torch

import gradient_sync_amd as dps
from tests.helpers import say

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16


def small(rows, k, seed):
    """Multiples of 1/8 up to 12, each block at a scale of its own: what four bits hold exactly."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=DEV)
    x = grid[torch.randint(0, 16, (rows, k), generator=g, device=DEV)]
    e = torch.randint(-2, 2, (rows, -(-k // 32)), generator=g, device=DEV).float()
    return x * torch.exp2(e).repeat_interleave(32, 1)[:, :k]


@pytest.mark.parametrize("m,n,k", [
    (8192, 8192, 200), (8192, 8192, 1024), (8192, 8192, 1100), (8192, 8192, 1400),    # in turn, no edges
    (8001, 8200, 200), (8100, 8072, 1024), (7937, 8192, 1100), (8192, 7944, 1400),    # in turn, edges, 16-byte stores
    (8001, 8203, 200), (7941, 5099, 1400), (8190, 8191, 1100),                        # in turn, other stores
    (4096, 4096, 1024), (4001, 4090, 1100), (4090, 4096, 1300),                       # large tiles, one each
    (4096, 2560, 512), (3900, 2601, 640), (2561, 4090, 130), (1024, 1024, 1400)])     # tiles of 128
def test_large_products_are_exact(m, n, k):
    """Products are multiples of 1/64 up to 144, their sums below 144 * 1400 = 2^24 / 64 * 0.77: every partial
    sum is a number of fp32."""
    a, b = small(m, k, m + k), small(n, k, n + k + 1)
    qa, qb = dps.dp_mxfp4_quantize(a), dps.dp_mxfp4_quantize(b)
    assert torch.equal(dps.dp_mxfp4_dequantize(qa, dtype=F32), a) and torch.equal(dps.dp_mxfp4_dequantize(qb, dtype=F32), b)
    want = (a.double() @ b.double().t().contiguous()).float()
    say("exact product", m, n, k)
    for dtype in (F32, BF16):
        buf = torch.full((m * n + 64,), 5.0, dtype=dtype, device=DEV)
        out = buf[32:32 + m * n].view(m, n)
        dps.dp_gemm_mxfp4(qa, qb, out=out)
        assert torch.equal(out, want.to(dtype)), dtype
        if dtype == F32:
            dps.dp_gemm_mxfp4(qa, qb, out=out, accumulate=True)
            assert torch.equal(out, want + want)
        assert bool((buf[:32] == 5).all()) and bool((buf[-32:] == 5).all())
    # rows of C that start on 2 bytes
    buf = torch.full((m * n + 65,), 5.0, dtype=BF16, device=DEV)
    dps.dp_gemm_mxfp4(qa, qb, out=buf[33:33 + m * n].view(m, n))
    assert torch.equal(buf[33:33 + m * n].view(m, n), want.bfloat16()) and bool((buf[:33] == 5).all()) and bool((buf[-32:] == 5).all())
