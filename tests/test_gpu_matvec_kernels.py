"""The product of a few unrounded rows with a 4-bit weight through every kernel that its sizes lead to, against 64 bits,
and bit for bit where the sum has one term."""
import pytest
import torch

import gradient_sync_amd as dps
from tests.helpers import say

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16


def rand(shape, seed, dtype=F32):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(shape, generator=g, device=DEV)
    return (x * torch.exp2(torch.randint(-3, 4, (shape[0], 1), generator=g, device=DEV).float())).to(dtype)


def check(y, x, w):
    """Each of at most 3 k fp32 additions may lose 2^-23 of the sum of magnitudes; a bf16 output half a step, 2^-8."""
    x, w = x.double(), dps.dp_mxfp4_dequantize(w, dtype=F32).double()
    want, mag = x @ w.t().contiguous(), x.abs() @ w.abs().t().contiguous()
    tol = 3 * x.shape[1] * 2.0 ** -23 * mag + (2.0 ** -8 * want.abs() if y.dtype == BF16 else 0)
    off = (y.double() - want).abs()
    assert bool((off <= tol).all()), float((off - tol).max())


# around the number of rows up to which x goes through LDS (8 of bf16, 2 of fp32, fewer beyond 8192 columns), and every
# number of 16-row blocks a workgroup beyond 8192 columns
@pytest.mark.parametrize("x_dtype", [F32, BF16])
@pytest.mark.parametrize("m,n", [(m, n) for m in (2, 3, 6, 7, 8, 9) for n in (300, 8192, 8200)]
                         + [(m, n) for m in (17, 32, 33, 48, 49, 64) for n in (2100, 8200, 14336)])
def test_rows_around_the_limits(m, n, x_dtype):
    for k in (1030, 2047):
        x, w = rand((m, k), m, x_dtype), dps.dp_mxfp4_quantize(rand((n, k), 6))
        say("matvec", m, n, k, x_dtype)
        for t in (F32, BF16):
            buf = torch.full((m * n + 64,), 5.0, dtype=t, device=DEV)
            out = buf[32:32 + m * n].view(m, n)
            dps.dp_mxfp4_matvec(x, w, out=out)
            check(out, x, w)
            assert bool((buf[:32] == 5).all()) and bool((buf[-32:] == 5).all())


@pytest.mark.parametrize("m,n,k", [(1, 300, 4700), (2, 300, 4700), (2, 8200, 1030), (3, 300, 4700), (9, 1000, 1030), (3, 8192, 1030),
                                   (17, 2100, 1030), (3, 8200, 600), (33, 4096, 1030), (17, 8200, 1030), (64, 8192, 1030),
                                   (48, 8200, 1030), (49, 8200, 1030), (64, 14336, 2047)])
def test_all_24_bits_of_x_enter_every_kernel(m, n, k):
    """Rows with one value and weights that are powers of two: an output is a product of 24 bits and a power, and has a
    wrong bit wherever a part of x is lost, or a part, a row or a column is taken for another. The column with the
    value goes through all of K."""
    g = torch.Generator(device=DEV).manual_seed(m + n)
    pick = lambda lo, hi, shape: torch.randint(lo, hi, shape, generator=g, device=DEV)
    w = torch.exp2(pick(-1, 3, (n, k)).float() + pick(-20, 21, (n, -(-k // 32))).float().repeat_interleave(32, 1)[:, :k])
    w = torch.where(pick(0, 2, (n, k)) == 0, w, -w)
    q = dps.dp_mxfp4_quantize(w)
    assert torch.equal(dps.dp_mxfp4_dequantize(q, dtype=F32), w)
    r = torch.arange(m, device=DEV)
    say("matvec, 24 bits", m, n, k)
    for call in range(24):
        v = (pick(0, 1 << 23, (m,)) | 1 | pick(127 - 60, 127 + 61, (m,)) << 23).int().view(F32)
        v = torch.where(pick(0, 2, (m,)) == 0, v, -v)
        at = (torch.tensor([0, k - 1, k // 2], device=DEV)[r % 3] if call == 0 else pick(0, k, (m,)))
        x = torch.zeros(m, k, device=DEV)
        x[r, at] = v
        want = v.unsqueeze(1) * w[:, at].t()
        assert torch.equal(dps.dp_mxfp4_matvec(x, q, dtype=F32), want)


@pytest.mark.parametrize("m,n,k", [(1, 300, 1030), (2, 300, 4700), (9, 1000, 1030), (64, 8200, 1030)])
def test_small_values_of_x(m, n, k):
    """fp32 values from 2^-110 on enter with all their bits (the last of which is 2^-133, bf16's smallest number), smaller ones
    with those from 2^-133 on; zero and what is below that are nothing."""
    g = torch.Generator(device=DEV).manual_seed(m)
    w = torch.full((n, k), 2.0 ** 40, device=DEV)
    q = dps.dp_mxfp4_quantize(w)
    r = torch.arange(m, device=DEV)
    for e in (-108, -109, -110, -111, -118, -126, -127):         # -127: fp32's own subnormal numbers
        bits = torch.randint(0, 1 << 23, (m,), generator=g, device=DEV) | 1 | (e + 127) << 23
        v = bits.int().view(F32)
        x = torch.zeros(m, k, device=DEV)
        x[r, (r * 97 + 5) % k] = v
        say("matvec, small values", m, n, k, e)
        y = dps.dp_mxfp4_matvec(x, q, dtype=F32).double() * 2.0 ** -40
        kept = (v.double() * 2.0 ** 133).trunc() * 2.0 ** -133
        assert torch.equal(y, (v.double() if e >= -110 else kept).unsqueeze(1).expand(m, n))
